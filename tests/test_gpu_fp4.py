"""The microscaled 4-bit formats and their linear against plain references.

Codes and scales are decided in binary32 on both sides and must agree to the bit.  The
linear's bound, from its definition: one rounding to bf16 (8 significant bits, so 2^-8 of
the result, taken as 2^-7.9 for the scaling before it) plus the fp32 accumulation -- at most 12288 / 64 chained
64-element products, each with an error below 2^-21 of sum |x w| -- 2^-13 of that sum.
"""
import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg
from tests import _ref64 as R

pytestmark = pytest.mark.gpu

FMTS = [dg.DG_FP4_MX, dg.DG_FP4_NV]


def _x(M, K, seed, device="cuda", wide=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    if wide:                                   # blocks of many magnitudes, zero, subnormal, lone spikes
        x *= torch.exp2(torch.randint(-40, 30, (M, K // 16), generator=g).float()).repeat_interleave(16, 1)
        x[torch.rand((M, K), generator=g) < 0.05] = 0.0
        x[0, :32] = 0.0
        x[-1, K - 32:] *= 2.0 ** -120
        x[M // 2, K // 2] = -3.0e38
    return x.to(torch.bfloat16).to(device)


def _f32(t):
    return t.float().cpu().numpy()


def _codes(q):
    return R.unpack(q.cpu().numpy())


def _g(v):
    return None if v is None else torch.tensor([v], dtype=torch.float32, device="cuda")


def _ref_linear(x, code_w, byte_w, fmt, gx, gw):
    cx, bx = R.fp4_quant(_f32(x), fmt, 1.0 if gx is None else gx)
    a, w = R.fp4_values(cx, bx, fmt), R.fp4_values(code_w, byte_w, fmt)
    alpha = float(np.float32(1.0 if gx is None else gx) * np.float32(1.0 if gw is None else gw))
    return a @ w.T * alpha, np.abs(a) @ np.abs(w).T * abs(alpha)


def _check(y, ref, absdot):
    err = np.abs(y.float().cpu().double().numpy() - ref)
    lim = 2.0 ** -7.9 * np.abs(ref) + 2.0 ** -13 * absdot + 1e-30
    assert (err <= lim).all(), f"largest error / bound {np.max(err / lim):.3f} at {np.unravel_index((err / lim).argmax(), err.shape)}"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,seed,wide", [(1, 32, 1, False), (3, 96, 2, True), (16, 4096, 3, True), (127, 1056, 4, True),
                                           (128, 256, 5, False), (129, 544, 6, True), (300, 2080, 7, True),
                                           (1, 12288, 8, False)])
@pytest.mark.parametrize("g", [None, 117.5 / 2688, 3.7e-5])
def test_quant_codes_and_scales_bit_exact(cuda_device, fmt, M, K, seed, wide, g):
    if fmt == dg.DG_FP4_MX and g is not None:
        pytest.skip("MX has no tensor scale")
    x = _x(M, K, seed, wide=wide)
    s = torch.full(dg.fp4_scale_shape(M, K, fmt), 0xAB, dtype=torch.uint8, device="cuda")   # padding is written too
    q, s = dg.dg_quant_fp4_blockscale(x, fmt, g=_g(g), s=s)
    code, byte = R.fp4_quant(_f32(x), fmt, 1.0 if g is None else g)
    assert np.array_equal(s.cpu().numpy(), R.tile(byte))
    assert np.array_equal(_codes(q), code)
    assert dg.dg_fp4_scale_bytes(M, K, fmt) == s.numel()


@pytest.mark.parametrize("fmt", FMTS)
def test_quant_every_bf16_magnitude(cuda_device, fmt):
    """Each finite bf16 value as the largest of its block, with every value below it sampled."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    top = bits.to(torch.int16).view(torch.bfloat16).float()
    g = torch.Generator().manual_seed(9)
    x = top[:, None] * (torch.rand((len(top), 32), generator=g) * 2 - 1)
    x[:, ::16] = top[:, None]
    x[:, 1::16] = top[:, None] * torch.tensor([5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25])[torch.arange(len(top)) % 7][:, None] / 6
    x = x.to(torch.bfloat16).cuda()
    q, s = dg.dg_quant_fp4_blockscale(x, fmt)
    code, byte = R.fp4_quant(_f32(x), fmt)
    assert np.array_equal(s.cpu().numpy(), R.tile(byte))
    assert np.array_equal(_codes(q), code)


@pytest.mark.parametrize("fmt", FMTS)
def test_quant_non_finite_blocks(cuda_device, fmt):
    x = _x(4, 128, 3)
    x[0, 5], x[1, 40], x[2, 127] = float("nan"), float("inf"), -float("inf")
    q, s = dg.dg_quant_fp4_blockscale(x, fmt)
    code, byte = R.fp4_quant(_f32(x), fmt)
    assert np.array_equal(s.cpu().numpy(), R.tile(byte)) and np.array_equal(_codes(q), code)
    b = R.BLOCK[fmt]
    y = dg.dg_dequant_fp4_blockscale(q, s, fmt).cpu()
    nan = torch.zeros((4, 128), dtype=torch.bool)
    for r, c in ((0, 5), (1, 40), (2, 127)):
        nan[r, c // b * b:(c // b + 1) * b] = True
    assert torch.equal(torch.isnan(y), nan)


@pytest.mark.parametrize("fmt,g", [(dg.DG_FP4_MX, None), (dg.DG_FP4_NV, None), (dg.DG_FP4_NV, 0.013)])
@pytest.mark.parametrize("M,K", [(1, 32), (5, 288), (200, 1056)])
def test_dequant_bit_exact(cuda_device, fmt, g, M, K):
    x = _x(M, K, 11, wide=g is None)
    q, s = dg.dg_quant_fp4_blockscale(x, fmt, g=_g(g))
    y = dg.dg_dequant_fp4_blockscale(q, s, fmt, g=_g(g))
    code, byte = R.fp4_quant(_f32(x), fmt, 1.0 if g is None else g)
    sg = (R.fp4_scale_value(byte, fmt).astype(np.float32) * np.float32(1.0 if g is None else g)).astype(np.float32)
    v = (R.fp4_value(code).astype(np.float32).reshape(M, -1, R.BLOCK[fmt]) * sg[..., None]).reshape(M, K)
    assert torch.equal(y.cpu(), torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16))


def test_quant_offsets_past_32_bits(cuda_device):
    """More than 2^31 elements: the last rows equal the same rows on their own."""
    M, K = 140000, 16384
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(5))
    q, s = dg.dg_quant_fp4_blockscale(x, dg.DG_FP4_NV)
    t0 = M // 128 * 128
    q1, s1 = dg.dg_quant_fp4_blockscale(x[t0:].contiguous(), dg.DG_FP4_NV)
    assert torch.equal(q[t0:], q1) and torch.equal(s[t0 // 128:], s1)
    y = dg.dg_dequant_fp4_blockscale(q, s, dg.DG_FP4_NV)
    assert torch.equal(y[t0:], dg.dg_dequant_fp4_blockscale(q1, s1, dg.DG_FP4_NV))


def _weights(N, K, fmt, gw, seed):
    w = (torch.randn((N, K), generator=torch.Generator().manual_seed(seed)) * K ** -0.5).to(torch.bfloat16)
    code, byte = R.fp4_quant(w.float().numpy(), fmt, 1.0 if gw is None else gw)
    return (torch.from_numpy(R.pack(code)).cuda(), torch.from_numpy(R.tile(byte)).cuda(), code, byte)


SMALL = [(1, 128, 256), (2, 1, 32), (3, 130, 1056), (5, 77, 544), (8, 300, 2080), (9, 128, 64), (16, 96, 288),
         (17, 65, 160), (31, 640, 4096), (33, 129, 96), (64, 257, 1056), (77, 200, 12288), (100, 1000, 512),
         (128, 128, 8192), (129, 140, 1056), (200, 70, 320), (256, 384, 2048), (257, 129, 1056), (512, 100, 4096)]


@pytest.mark.parametrize("fmt,gx,gw", [(0, None, None), (1, None, None), (1, 0.044, 2.1e-4)])
@pytest.mark.parametrize("M,N,K", SMALL)
def test_linear_small_exhaustive(cuda_device, M, N, K, fmt, gx, gw):
    Wq, sw, code, byte = _weights(N, K, fmt, gw, N + K)
    x = _x(M, K, M + N)
    ws = dg.workspace(dg.DG_OP_GEMV_A4W4, M, N, K)
    y = dg.dg_gemv_a4w4_blockscale(x, Wq, sw, fmt, gx=_g(gx), gw=_g(gw), ws=ws)
    _check(y, *_ref_linear(x, code, byte, fmt, gx, gw))
    assert dg.dg_device_status(ws) == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 12288, 4096), (64, 4096, 12288), (512, 8192, 1024)])
def test_linear_model_shapes_sampled(cuda_device, M, N, K, fmt):
    w = (torch.randn((N, K), generator=torch.Generator("cuda").manual_seed(N), device="cuda") * K ** -0.5).to(torch.bfloat16)
    Wq, sw = dg.dg_quant_fp4_blockscale(w, fmt)
    x = _x(M, K, 5)
    y = dg.dg_gemv_a4w4_blockscale(x, Wq, sw, fmt)
    rows = np.unique(np.r_[0, N - 1, np.random.default_rng(N + M).choice(N, 96)])
    code, byte = R.fp4_quant(_f32(w[torch.as_tensor(rows, device="cuda")]), fmt)
    _check(y[:, torch.as_tensor(rows, device="cuda")], *_ref_linear(x, code, byte, fmt, None, None))


@pytest.mark.parametrize("fmt", FMTS)
def test_linear_one_hot_reads_every_weight(cuda_device, fmt):
    """x = 6 e_k gives column k of the dequantised weights times 6: every code, scale and
    position of both layouts shows."""
    N, K = 200, 512
    Wq, sw, code, byte = _weights(N, K, fmt, None, 4)
    w = R.fp4_values(code, byte, fmt)
    eye = torch.eye(K, device="cuda").mul_(6.0).to(torch.bfloat16)
    y = dg.dg_gemv_a4w4_blockscale(eye, Wq, sw, fmt).float().cpu().double().numpy()
    assert np.array_equal(y, torch.from_numpy((6.0 * w.T).astype(np.float32)).to(torch.bfloat16).double().numpy())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 8, 9, 40, 128, 130])
def test_linear_variants_bitwise_identical(cuda_device, fmt, M):
    N, K = 1000, 4096 + 96
    Wq, sw, _, _ = _weights(N, K, fmt, None, 8)
    x = _x(M, K, 2)
    for rule in (0, 1):
        ref = dg.dg_gemv_a4w4_blockscale(x, Wq, sw, fmt, choice=dg.Choice.make(dg.DG_VAR_TC, 0, rule))
        ran = 0
        for st in range(2, 9):
            try:
                y = dg.dg_gemv_a4w4_blockscale(x, Wq, sw, fmt, choice=dg.Choice.make(dg.DG_VAR_TC, st, rule))
            except dg.DGError as e:
                assert e.status in (3, 8)
                continue
            ran += 1
            assert torch.equal(y.view(torch.int16), ref.view(torch.int16)), (st, rule)
        assert ran >= 2


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,K", [(4096, 4096), (300, 1056)])
def test_linear_rows_independent_of_the_batch(cuda_device, fmt, N, K):
    """At every row count in the batch-invariant mode, whatever the groups and the quantisation's place."""
    Wq, sw, _, _ = _weights(N, K, fmt, None, 3)
    x = _x(300, K, 6)
    dg.dg_set_numerics(dg.DG_NUMERICS_BATCH_INVARIANT)
    try:
        every = dg.dg_gemv_a4w4_blockscale(x, Wq, sw, fmt)
        for M in (1, 2, 7, 8, 9, 16, 17, 33, 65, 127, 128, 129, 200, 257, 300):
            y = dg.dg_gemv_a4w4_blockscale(x[:M].contiguous(), Wq, sw, fmt)
            assert torch.equal(y.view(torch.int16), every[:M].view(torch.int16)), M
    finally:
        dg.dg_set_numerics(dg.DG_NUMERICS_FASTEST)
    full = dg.dg_gemv_a4w4_blockscale(x[:40].contiguous(), Wq, sw, fmt)
    x2 = x[:40].clone()
    x2[3] = float("nan")                                      # a poisoned token stays in its row
    y = dg.dg_gemv_a4w4_blockscale(x2, Wq, sw, fmt)
    assert torch.isnan(y[3]).all()
    keep = [i for i in range(40) if i != 3]
    assert torch.equal(y[keep].view(torch.int16), full[keep].view(torch.int16))


def test_linear_after_quantising_its_weights_and_in_a_graph(cuda_device):
    """A linear queued right behind the quantisation of its weights reads the new weights, on a
    stream of its own and replayed from a graph."""
    N, K, fmt = 4096, 4096, dg.DG_FP4_NV
    w = [(torch.randn((N, K), device="cuda") * K ** -0.5).to(torch.bfloat16) for _ in range(2)]
    x = _x(4, K, 1)
    want = []
    for v in w:
        q, s = dg.dg_quant_fp4_blockscale(v, fmt)
        torch.cuda.synchronize()
        want.append(dg.dg_gemv_a4w4_blockscale(x, q, s, fmt))
    torch.cuda.synchronize()
    q, s, y = torch.empty_like(q), torch.empty_like(s), torch.empty_like(want[0])
    ws = dg.workspace(dg.DG_OP_GEMV_A4W4, 4, N, K)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for i in range(40):
            dg.dg_quant_fp4_blockscale(w[i % 2], fmt, q=q, s=s)
            dg.dg_gemv_a4w4_blockscale(x, q, s, fmt, y=y, ws=ws)
            assert torch.equal(y.view(torch.int16), want[i % 2].view(torch.int16)), i
    st.synchronize()
    cur = w[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.dg_quant_fp4_blockscale(cur, fmt, q=q, s=s)
        dg.dg_gemv_a4w4_blockscale(x, q, s, fmt, y=y, ws=ws)
    for i in (0, 1, 1, 0):
        cur.copy_(w[i])
        graph.replay()
        assert torch.equal(y.view(torch.int16), want[i].view(torch.int16))


def test_linear_in_the_sweep_and_the_table(cuda_device, tmp_path):
    """The sweep measures pipeline depths for either format, the table it writes drives the call, same bits."""
    M, N, K = 16, 512, 1024
    path = str(tmp_path / "t.json")
    dg.dg_sweep([(dg.DG_OP_GEMV_A4W4, M, N, K, dg.DG_FP4_NV), (dg.DG_OP_GEMV_A4W4, 2, N, K, dg.DG_FP4_MX)], path, reps=3)
    x = _x(M, K, 1)
    Wq, sw, _, _ = _weights(N, K, dg.DG_FP4_NV, None, 2)
    ref = dg.dg_gemv_a4w4_blockscale(x, Wq, sw, dg.DG_FP4_NV)
    dg.dg_table_load(path)
    try:
        assert dg.dg_table_entries() == 2
        assert dg.dg_select(dg.DG_OP_GEMV_A4W4, M, N, K).from_table == 1
        y = dg.dg_gemv_a4w4_blockscale(x, Wq, sw, dg.DG_FP4_NV)
    finally:
        dg.dg_table_clear()
    assert torch.equal(y.view(torch.int16), ref.view(torch.int16))


def test_linear_refusals(cuda_device):
    Wq, sw, _, _ = _weights(64, 256, 1, None, 1)
    x = _x(2, 256, 1)
    ws = dg.workspace(dg.DG_OP_GEMV_A4W4, 2, 64, 256)
    for bad in (dg.Choice.make(dg.DG_VAR_CC_WARP, 4, 8), dg.Choice.make(dg.DG_VAR_TC, 1), dg.Choice.make(dg.DG_VAR_TC, 9),
                dg.Choice.make(dg.DG_VAR_TC, 0, 2), dg.Choice.make(dg.DG_VAR_TC, 0, 0, 1)):
        with pytest.raises(dg.DGError) as e:
            dg.dg_gemv_a4w4_blockscale(x, Wq, sw, 1, ws=ws, choice=bad)
        assert e.value.status == dg.DG_ERR_BAD_VARIANT
    with pytest.raises(dg.DGError) as e:
        dg.dg_gemv_a4w4_blockscale(x, Wq, sw, 1, ws=ws[:1024])
    assert e.value.status == dg.DG_ERR_WORKSPACE_TOO_SMALL
    assert torch.isfinite(dg.dg_gemv_a4w4_blockscale(x, Wq, sw, 1, ws=ws)).all()
