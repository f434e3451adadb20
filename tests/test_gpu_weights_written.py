"""Weights that this library has just written: the kernel that reads them next waits in full.

Linears read their weights before they wait for the launches ahead of them.  The dependency is
looked at in a captured graph (no kernel runs for that), and the values in calls queued back to back.
"""
import ctypes

import pytest
import torch

import gemv_dg_bf16_gb300 as dg

pytestmark = pytest.mark.gpu

FULL, PROGRAMMATIC = 0, 1                # CUgraphDependencyType


class _Edge(ctypes.Structure):
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte),
                ("reserved", ctypes.c_ubyte * 5)]


def _edges(calls):
    """Types of the dependencies between the launches that `calls` queues on a stream, in order."""
    cu = ctypes.CDLL("libcuda.so.1")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    handle, graph, n = ctypes.c_void_p(st.cuda_stream), ctypes.c_void_p(), ctypes.c_size_t()
    assert cu.cuStreamBeginCapture_v2(handle, 2) == 0                      # relaxed: this thread may allocate
    try:
        for c in calls:
            c(st)
    finally:
        assert cu.cuStreamEndCapture(handle, ctypes.byref(graph)) == 0
    try:
        assert cu.cuGraphGetEdges_v2(graph, None, None, None, ctypes.byref(n)) == 0
        a, b, data = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (_Edge * n.value)()
        assert cu.cuGraphGetEdges_v2(graph, a, b, data, ctypes.byref(n)) == 0
    finally:
        cu.cuGraphDestroy(graph)
    after = {a[i]: (b[i], data[i].type) for i in range(n.value)}
    assert len(after) == n.value                                           # a chain
    at, types = (set(after) - {v[0] for v in after.values()}).pop(), []
    while at in after:
        at, t = after[at]
        types.append(t)
    return types


@pytest.fixture(scope="module")
def bench(cuda_device):
    """Buffers of every call used here, made once (and every kernel loaded)."""
    N, K = 512, 1024
    g = torch.Generator("cuda").manual_seed(1)
    b = {"w": [(torch.randn((N, K), generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16) for _ in range(2)]}
    b["x"] = torch.randn((64, K), generator=g, device="cuda").to(torch.bfloat16)
    b["packed"] = [dg.dg_quant_fp4_blockscale(w, dg.DG_FP4_NV) for w in b["w"]]
    b["q"], b["s"] = (torch.empty_like(t) for t in b["packed"][0])
    b["dense"] = torch.empty_like(b["w"][0])
    b["y"] = {M: torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for M in (1, 4, 16, 64)}
    b["half"] = torch.empty((1, N // 2), dtype=torch.bfloat16, device="cuda")
    b["ws"] = dg.workspace(dg.DG_OP_GEMV_A4W4, 64, N, K)
    b["logits"] = torch.randn((4, 64), device="cuda")
    b["ids"], b["gate"] = dg.dg_moe_route(b["logits"], 4)
    torch.cuda.synchronize()
    return b


def _quant(b, i=0):
    return lambda st: dg.dg_quant_fp4_blockscale(b["w"][i], dg.DG_FP4_NV, q=b["q"], s=b["s"], stream=st)


def _dequant(b, i=0):
    return lambda st: dg.dg_dequant_fp4_blockscale(*b["packed"][i], dg.DG_FP4_NV, y=b["dense"], stream=st)


def _linear4(b, M):
    return lambda st: dg.dg_gemv_a4w4_blockscale(b["x"][:M], b["q"], b["s"], dg.DG_FP4_NV, y=b["y"][M], ws=b["ws"], stream=st)


def _linear16(b, M):
    return lambda st: dg.dg_gemv_bf16(b["x"][:M], b["dense"], y=b["y"][M], ws=b["ws"], stream=st)


def _gate_up(b):
    return lambda st: dg.dg_gate_up_silu(b["x"][:1], b["dense"], out=b["half"], ws=b["ws"], stream=st)


def _route(b):
    return lambda st: dg.dg_moe_route(b["logits"], 4, ids=b["ids"], w=b["gate"], stream=st)


def _readers(b):
    return [(_linear4(b, 1), 1), (_linear4(b, 64), 2)] + [(_linear16(b, M), 1) for M in (1, 4, 16)] + [(_gate_up(b), 1)]


@pytest.mark.parametrize("writer", [_quant, _dequant])
def test_reader_of_weights_behind_their_writer_waits_in_full(bench, writer):
    for read, launches in _readers(bench):
        assert len(_edges([read, read])) == 2 * launches - 1
        for calls in ([writer(bench), read], [writer(bench), _route(bench), read],
                      [writer(bench), writer(bench), read]):
            assert _edges(calls)[-1] == FULL                               # (a quantisation of activations reads none)
        assert _edges([writer(bench), read, read]) == [PROGRAMMATIC] * (launches - 1) + [FULL] + [PROGRAMMATIC] * launches


def test_launches_that_read_no_fresh_weights_still_overlap(bench):
    for read, launches in _readers(bench):
        assert set(_edges([read, read, _route(bench), read])) == {PROGRAMMATIC}
    assert _edges([_quant(bench), _dequant(bench), _route(bench)]) == [PROGRAMMATIC] * 2
    # the note belongs to the stream it was made on
    other = torch.cuda.Stream()
    _quant(bench)(other)
    assert set(_edges([_route(bench), _linear4(bench, 1)])) == {PROGRAMMATIC}
    torch.cuda.synchronize()


@pytest.mark.parametrize("M", [1, 4, 16])
def test_linears_read_the_weights_just_written(bench, M):
    """Quantised -> 4-bit linear and dequantised -> bf16 linear, on a stream and from a graph."""
    b, want4, want16 = bench, [], []
    for i in range(2):
        for call in (_quant(b, i), _dequant(b, i)):
            call(torch.cuda.current_stream())
        torch.cuda.synchronize()
        _linear4(b, M)(torch.cuda.current_stream())
        want4.append(b["y"][M].clone())
        _linear16(b, M)(torch.cuda.current_stream())
        want16.append(b["y"][M].clone())
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for i in range(40):
        for write, read, want in ((_quant, _linear4, want4), (_dequant, _linear16, want16)):
            write(b, i % 2)(st)
            read(b, M)(st)
            st.synchronize()
            assert torch.equal(b["y"][M].view(torch.int16), want[i % 2].view(torch.int16)), i
    graphs = []
    for write, read in ((_quant, _linear4), (_dequant, _linear16)):
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                write(b, i)(None)
                read(b, M)(None)
            graphs.append((g, (want4 if write is _quant else want16)[i]))
    for k in (0, 1, 2, 3, 1, 0, 3, 2):
        graphs[k][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(b["y"][M].view(torch.int16), graphs[k][1].view(torch.int16)), k


def test_linear_on_another_stream_behind_an_event(bench):
    """Written on one stream, read on another that is busy with linears of its own, in turn and from a graph."""
    b, t, s, want = bench, torch.cuda.Stream(), torch.cuda.Stream(), []
    for i in range(2):
        _quant(b, i)(t)
        _linear4(b, 4)(t)
        t.synchronize()
        want.append(b["y"][4].clone())

    def step(i):
        """Fork from t, write on s, join, read on t; linears of other weights around it."""
        dg.dg_gemv_bf16(b["x"][:1], b["w"][0], y=b["y"][1], ws=b["ws"], stream=t)
        s.wait_stream(t)
        _quant(b, i)(s)
        dg.dg_gemv_bf16(b["x"][:1], b["w"][0], y=b["y"][1], ws=b["ws"], stream=t)
        t.wait_stream(s)
        _linear4(b, 4)(t)
    for i in range(40):
        step(i % 2)
        t.synchronize()
        assert torch.equal(b["y"][4].view(torch.int16), want[i % 2].view(torch.int16)), i
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=t):
            step(i)
        graphs.append(g)
    for i in (0, 1, 0, 1, 1, 0) * 5:
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(b["y"][4].view(torch.int16), want[i].view(torch.int16))
