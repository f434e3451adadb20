"""The 8-bit integer linear, the sort by expert with its rows, and the edits of logits where calls meet: two at
once, chains over shared buffers, graphs that share a workspace, outputs inside larger buffers, and buffers whose
offsets pass 32 bits."""
import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg
from tests import _ref_more as R
from tests.test_gpu_i8 import _bits, _w, _x
from tests.test_gpu_logits import _edits, _gpu
from tests.test_gpu_moe_sort import _ids

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def _bf(shape, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF)


def test_two_calls_at_once():
    """Two streams, each with its own workspaces and buffers: cluster, persistent and split launches side by side."""
    def work(seed):
        out = []
        for M, N, K in ((1, 1000, 4096), (16, 640, 4096), (64, 20480, 256), (77, 1283, 2064), (300, 4096, 1040)):
            w, sw = _w(N, K, seed + M)
            out.append((_x(M, K, seed).cuda(), w.cuda(), sw.cuda()))
        ids = [torch.from_numpy(_ids(M, 8, 256, seed + M)).cuda() for M in (10, 3000)]
        rows = _bf((3000, 520), seed)
        logits = [(_bf((M, V), seed + M), _gpu(_edits(M, V, 90, 7, True, seed + M))) for M, V in ((2, 5000), (40, 64000))]
        return out, ids, rows, logits

    def run(case, ws):
        linears, ids, rows, logits = case
        got = [dg.dg_gemv_i8_rowscale(*t, ws=w) for t, w in zip(linears, ws)]
        for i in ids:
            offsets, pos, slots = dg.dg_moe_sort(i, 256)
            x = rows[:i.shape[0]]
            xs = dg.dg_moe_gather(x, pos)
            wt = torch.full(i.shape, 0.25, device="cuda")
            got += [offsets, pos, slots, dg.dg_moe_combine(xs, pos, wt), *dg.dg_moe_combine_grad(x, xs, pos, wt)]
        got += [dg.dg_logits_adjust(x, out=torch.empty_like(x), **e) for x, e in logits]
        return got

    cases = [work(1), work(50)]
    ws = [[dg.workspace(dg.DG_OP_GEMV_I8, t[0].shape[0], t[1].shape[0], t[1].shape[1]) for t in c[0]] for c in cases]
    want = []
    for c, w in zip(cases, ws):
        want.append(run(c, w))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(cases[i], ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
        assert all(dg.dg_device_status(w) == 0 for w in ws[i])


def test_chain_over_shared_buffers():
    """Sort, rows, linear, combine, head's edits one behind the other without a wait, over and over in the same
    buffers: no kernel begins on what the one ahead has not finished."""
    M, topk, E, K, N = 40, 4, 16, 512, 640
    w, sw = (t.cuda() for t in _w(N, K, 1))
    P = M * topk
    offsets, pos, slots = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((E + 1,), (M, topk), (P,)))
    xs, z, y = (torch.empty(s, dtype=BF, device="cuda") for s in ((P, K), (P, N), (M, N)))
    ws = dg.workspace(dg.DG_OP_GEMV_I8, P, N, K)
    edits = _gpu(_edits(M, N, 30, 5, True, 3))
    gates = torch.rand((M, topk), device="cuda")
    cases = [(torch.from_numpy(_ids(M, topk, E, s)).cuda(), _bf((M, K), s)) for s in range(6)]

    def step(ids, x, wait):
        for f in (lambda: dg.dg_moe_sort(ids, E, offsets=offsets, pos=pos, slots=slots),
                  lambda: dg.dg_moe_gather(x, pos, xs=xs),
                  lambda: dg.dg_gemv_i8_rowscale(xs, w, sw, y=z, ws=ws),
                  lambda: dg.dg_moe_combine(z, pos, gates, y=y),
                  lambda: dg.dg_logits_adjust(y, **edits)):
            f()
            if wait:
                torch.cuda.synchronize()
        return y.clone()

    want = [step(*c, True) for c in cases]
    for _ in range(5):
        got = [step(*c, False) for c in cases]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    xw, ww = cases[0][1].cpu(), w.cpu()
    alone = R.i8_linear(R.f32(xw), ww.numpy(), sw.cpu().numpy())
    step(*cases[0], True)
    rows = slots[:int(offsets[E])].cpu().numpy() // topk
    np.testing.assert_array_equal(_bits(z)[:len(rows)], alone[rows])


def test_two_graphs_share_a_workspace():
    K = 2064
    w, sw = _w(1283, K, 2)
    wc, sc = w.cuda(), sw.cuda()
    ws = dg.workspace(dg.DG_OP_GEMV_I8, 300, 1283, K)
    graphs = []
    for M in (300, 16, 77):
        x, y = torch.zeros((M, K), dtype=BF, device="cuda"), torch.empty((M, 1283), dtype=BF, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dg.dg_gemv_i8_rowscale(x, wc, sc, y=y, ws=ws)
        graphs.append((M, x, y, g))
    for r in range(3):
        xs = [_x(M, K, 10 * r + M) for M, _, _, _ in graphs]
        for (_, x, _, _), v in zip(graphs, xs):
            x.copy_(v)
        for _, _, _, g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (_, _, y, _), v in zip(graphs, xs):
            np.testing.assert_array_equal(_bits(y), R.i8_linear(R.f32(v), w.numpy(), sw.numpy()))
    assert dg.dg_device_status(ws) == 0


def _framed(shape, dtype, fill):
    """A dense tensor of this shape with 64 bytes of `fill` on either side."""
    n, pad = int(np.prod(shape)), 64 // torch.empty((), dtype=dtype).element_size()
    whole = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    return whole, whole[pad:pad + n].view(shape), pad


@pytest.mark.parametrize("M", [1, 3, 5, 16, 77, 129])
@pytest.mark.parametrize("N,K", [(1, 16), (127, 48), (136, 1040), (1283, 2064)])
def test_nothing_around_the_outputs_is_written(M, N, K):
    frames = []

    def out(shape, dtype, fill):
        whole, inner, pad = _framed(shape, dtype, fill)
        frames.append((whole, pad, fill))
        return inner

    w, sw = (t.cuda() for t in _w(N, K, 1))
    x = _x(M, K, 2).cuda()
    dg.dg_gemv_i8_rowscale(x, w, sw, y=out((M, N), BF, 7.0))
    dg.dg_quant_i8_rowscale(x, q=out((M, K), torch.int8, 7), s=out((M,), torch.float32, 7.0))
    topk, E = min(6, N), max(6, min(N, 1024))
    ids = torch.from_numpy(_ids(M, topk, E, 3, 0.2)).cuda()
    _, pos, _ = dg.dg_moe_sort(ids, E, offsets=out((E + 1,), torch.int32, 7), pos=out((M, topk), torch.int32, 7),
                               slots=out((M * topk,), torch.int32, 7))
    xs = dg.dg_moe_gather(x, pos, xs=out((M * topk, K), BF, 7.0))
    dg.dg_moe_combine(xs, pos, y=out((M, K), BF, 7.0))
    dg.dg_moe_combine_grad(x, xs, pos, torch.ones((M, topk), device="cuda"), dz=out((M * topk, K), BF, 7.0),
                           dw=out((M, topk), torch.float32, 7.0))
    logits = _bf((M, N), 4)
    dg.dg_logits_adjust(logits, out=out((M, N), BF, 7.0), **_gpu(_edits(M, N, 20, 3, True, 5)))
    torch.cuda.synchronize()
    for whole, pad, fill in frames:
        assert (whole[:pad] == fill).all() and (whole[-pad:] == fill).all()


def test_one_row_in_several_slots():
    """Positions may name a row more than once where rows are only read."""
    z = _bf((4, 264), 1)
    pos = torch.tensor([[2, 2, -1], [0, 2, 0], [3, 3, 3]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25, 9.0], [1.0, 2.0, -1.0], [1.0, 1.0, 1.0]], device="cuda")
    y = dg.dg_moe_combine(z, pos, w).cpu()
    zf = z.cpu().double()
    for m, want in enumerate((0.75 * zf[2], 2.0 * zf[2], 3.0 * zf[3])):
        # (three products and sums of at most 4 |z| rounded to binary32 before the last)
        assert ((y[m].double() - want).abs() <= want.abs() * 2.0 ** -8 + 3 * zf[m if m else 2].abs().max() * 2.0 ** -22).all()


# ---------------------------------------------------------------- offsets past 32 bits

def test_weights_past_32_bits():
    N, K = 2 ** 20 + 37, 4112                                  # 4.3e9 bytes of weights
    w = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    sw = torch.rand((N,), device="cuda") * 1e-2 + 1e-4
    rows = torch.tensor(sorted({0, 1, N - 1, N - 38, *(r + d for r in (2 ** 31 // K, 2 ** 32 // K) for d in range(-2, 3))}))
    for M in (3, 20, 130):
        x = _x(M, K, M)
        y = dg.dg_gemv_i8_rowscale(x.cuda(), w, sw)
        want = R.i8_linear(R.f32(x), w[rows.cuda()].cpu().numpy(), sw[rows.cuda()].cpu().numpy())
        np.testing.assert_array_equal(_bits(y[:, rows.cuda()]), want)


def test_outputs_past_32_bits():
    M, N, K = 512, 2 ** 23 + 129, 16                           # 4.3e9 outputs
    w = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    sw = torch.rand((N,), device="cuda") * 1e-2 + 1e-4
    x = _x(M, K, 1)
    y = dg.dg_gemv_i8_rowscale(x.cuda(), w, sw)
    cols = torch.tensor([0, 1, 127, 128, 4097, N // 2, N - 130, N - 129, N - 1]).cuda()
    np.testing.assert_array_equal(_bits(y[:, cols]), R.i8_linear(R.f32(x), w[cols].cpu().numpy(), sw[cols].cpu().numpy()))


def test_codes_past_32_bits():
    M, K = 2 ** 21 + 3, 2064
    x = torch.empty((M, K), dtype=BF, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    q, s = dg.dg_quant_i8_rowscale(x)
    rows = torch.tensor(sorted({0, M - 1, M - 4, *(r + d for r in (2 ** 31 // K, 2 ** 32 // K) for d in (-1, 0, 1))})).cuda()
    wq, wsc = R.i8_codes(R.f32(x[rows]))
    np.testing.assert_array_equal(q[rows].cpu().numpy(), wq)
    np.testing.assert_array_equal(s[rows].cpu().numpy(), wsc)


def test_rows_past_32_bits():
    M, topk, N = 2 ** 14 + 1, 8, 2 ** 15                       # 4.3e9 elements of rows
    P = M * topk
    x = _bf((M, N), 1)
    pos = torch.randperm(P, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(M, topk).cuda()
    pos[5, 3] = -1
    xs = dg.dg_moe_gather(x, pos)
    for m in (0, 5, M // 2, M - 1):
        for k in range(topk):
            if pos[m, k] >= 0:
                assert torch.equal(xs[pos[m, k].long()], x[m])
    y = dg.dg_moe_combine(xs, pos)
    for m in (0, M // 2, M - 1):
        assert torch.equal(y[m], x[m] * 8)                     # (exact: each partial sum has at most 3 bits more)
    w = torch.rand((M, topk), device="cuda")
    dz, dw = dg.dg_moe_combine_grad(x, xs, pos, w)
    for m in (0, 5, M - 1):
        for k in range(topk):
            p = int(pos[m, k])
            if p < 0:
                assert dw[m, k] == 0
                continue
            assert torch.equal(dz[p], (w[m, k] * x[m].float()).to(BF))
            want = (x[m].double() ** 2).sum()
            assert abs(float(dw[m, k] - want)) <= float(want) * N / 8 * 2.0 ** -24


@pytest.mark.parametrize("L", [40, 9000])
def test_logits_past_32_bits(L):
    """Lists that the hash table takes, and longer ones, over 4.3e9 logits in place."""
    M, V, B = 17500, 248320, 3
    x = torch.empty((M, V), dtype=BF, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    g = torch.Generator(device="cuda").manual_seed(2)
    e = {"tokens": torch.randint(0, V, (M, L), dtype=torch.int32, device="cuda", generator=g),
         "prompt_lengths": torch.randint(0, L, (M,), dtype=torch.int32, device="cuda", generator=g),
         "repetition": torch.rand((M,), device="cuda", generator=g) + 0.7,
         "presence": torch.rand((M,), device="cuda", generator=g),
         "bias_ids": torch.randint(0, V, (M, B), dtype=torch.int32, device="cuda", generator=g),
         "bias": torch.rand((M, B), device="cuda", generator=g),
         "mask": torch.randint(-2 ** 31, 2 ** 31 - 1, (M, (V + 31) // 32), dtype=torch.int32, device="cuda", generator=g)}
    rows = torch.tensor(sorted({0, M - 1, *(r + d for r in (2 ** 31 // V, 2 ** 32 // V) for d in (0, 1))})).cuda()
    before = R.f32(x[rows])
    want = R.adjust(before, **{k: t[rows].cpu().numpy() for k, t in e.items()})
    dg.dg_logits_adjust(x, **e)
    np.testing.assert_array_equal(x[rows].cpu().view(torch.int16).numpy(), R.bf16_of(want))
