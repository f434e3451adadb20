"""Pairs sorted by expert, rows there and back, and the gradients, on the GPU."""
import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg
from tests import _ref_more as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _ids(M, topk, E, seed, absent=0.0, repeats=False):
    g = np.random.default_rng(seed)
    if repeats:
        ids = g.integers(-2, E + 2, (M, topk))
    else:
        like = g.normal(size=E)
        ids = np.argsort(-(like + g.gumbel(size=(M, E))), 1)[:, :topk]
    ids = ids.astype(np.int32)
    ids[g.random((M, topk)) < absent] = -1
    return ids


def _sorted(ids, E):
    offsets, pos, slots = dg.dg_moe_sort(torch.from_numpy(ids).cuda(), E)
    for got, want in zip((offsets, pos, slots), R.moe_sort(ids, E)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    return offsets, pos, slots


@pytest.mark.parametrize("M,topk,E", [(1, 1, 1), (1, 8, 256), (2, 32, 40), (31, 3, 7), (64, 6, 128), (300, 8, 256), (129, 32, 1024), (700, 5, 1000),
                                      (1024, 4, 8), (1025, 4, 8), (2049, 8, 256), (5000, 7, 64), (9001, 8, 384)])
@pytest.mark.parametrize("kind", ["all", "some", "repeats"])
def test_sort(M, topk, E, kind):
    _sorted(_ids(M, min(topk, E), E, M + E, 0.3 if kind == "some" else 0.0, kind == "repeats"), E)


def test_sort_of_one_expert_and_of_nothing():
    _sorted(np.full((5000, 1), 3, np.int32), 5)
    _sorted(np.full((5000, 4), 3, np.int32), 5)              # repeats of the first slot
    _sorted(np.full((70, 4), -1, np.int32), 5)
    _sorted(np.array([[2 ** 31 - 1, -2 ** 31, 5, 4]], np.int32), 5)


def test_sort_of_a_long_prompt():
    """262144 pairs, against torch's stable sort."""
    ids = torch.rand((32768, 256), generator=torch.Generator().manual_seed(1)).topk(8, -1).indices.int()
    offsets, pos, slots = dg.dg_moe_sort(ids.cuda(), 256)
    order = ids.reshape(-1).sort(stable=True)
    assert torch.equal(slots.cpu(), order.indices.int())
    assert torch.equal(pos.cpu().reshape(-1)[order.indices], torch.arange(ids.numel(), dtype=torch.int32))
    assert torch.equal(offsets.cpu(), torch.searchsorted(order.values, torch.arange(257, dtype=torch.int32)).int())


@pytest.mark.parametrize("dtype,K", [(BF, 8), (BF, 264), (BF, 4096), (torch.float32, 20), (torch.int8, 48), (torch.uint8, 16), (torch.float16, 2056),
                                     (torch.float64, 6)])
def test_gather(dtype, K):
    M, topk, E = 37, 5, 24
    ids = _ids(M, topk, E, K, 0.2)
    offsets, pos, slots = _sorted(ids, E)
    x = (torch.randn((M, K)) * 50).to(dtype)
    xs = torch.full((M * topk + 3, K), 7, dtype=dtype).cuda()
    dg.dg_moe_gather(x.cuda(), pos, xs=xs)
    n, s = int(offsets[-1]), slots.cpu().long()
    assert torch.equal(xs[:n].cpu(), x[s[:n] // topk])
    assert (xs[n:].cpu() == 7).all()                          # rows behind the last stay


def test_positions_outside_are_skipped():
    M, topk, N, P = 4, 3, 16, 5
    pos = torch.tensor([[0, 9, -1], [5, 1, -7], [2 ** 31 - 1, 2, -2 ** 31], [-1, -1, -1]], dtype=torch.int32).cuda()
    x = torch.randn((M, N)).to(BF).cuda()
    xs = torch.full((P, N), 3.0, dtype=BF, device="cuda")
    dg.dg_moe_gather(x, pos, xs=xs)
    assert torch.equal(xs[:3], x[:3]) and (xs[3:] == 3).all()
    w = torch.rand((M, topk)).cuda()
    y = dg.dg_moe_combine(xs, pos, w)
    want = torch.stack([w[0, 0] * x[0].float(), w[1, 1] * x[1].float(), w[2, 1] * x[2].float(), torch.zeros(N).cuda()]).to(BF)
    assert torch.equal(y, want)
    dz, dw = dg.dg_moe_combine_grad(x, xs, pos, w)
    assert (dz[3:] == 0).all() and (dw[3] == 0).all() and (dw[0, 1:] == 0).all() and (dw[:3].abs().sum(1) > 0).all()


def _problem(M, topk, E, N, absent, seed):
    ids = _ids(M, topk, E, seed, absent)
    _, pos, slots = R.moe_sort(ids, E)
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((M * topk, N), generator=g).to(BF)
    dy = torch.randn((M, N), generator=g).to(BF)
    w = torch.softmax(torch.randn((M, topk), generator=g), -1)
    return pos, z, dy, w


@pytest.mark.parametrize("M,topk,E,N,absent", [(1, 1, 2, 8, 0.0), (1, 8, 64, 4096, 0.0), (5, 2, 4, 24, 0.4), (33, 6, 128, 2056, 0.1), (9, 32, 40, 264, 0.2),
                                               (7, 9, 16, 4104, 0.9), (300, 8, 256, 520, 0.0), (3, 17, 20, 16392, 0.1)])
@pytest.mark.parametrize("weights", [True, False])
def test_combine(M, topk, E, N, absent, weights):
    pos, z, _, w = _problem(M, topk, E, N, absent, M + N)
    z[M * topk - 1] = float("nan") if (pos < M * topk - 1).all() else z[M * topk - 1]     # a row that no slot names
    y = dg.dg_moe_combine(z.cuda(), torch.from_numpy(pos).cuda(), w.cuda() if weights else None).cpu().double().numpy()
    live = pos >= 0
    ww = np.where(live, w.numpy().astype(np.float64) if weights else 1.0, 0.0)[..., None]
    zz = np.where(live[..., None], z.double().numpy()[np.maximum(pos, 0)], 0.0)
    ref, size = (ww * zz).sum(1), np.abs(ww * zz).sum(1)
    # one rounding of at most 2^-24 for each slot's step, then the output's (bf16: 2^-8)
    bound = topk * 2.0 ** -24 * size * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) + 1e-38
    assert (np.abs(y - ref) <= bound).all()


@pytest.mark.parametrize("M,topk,E,N,absent", [(1, 1, 2, 8, 0.0), (5, 2, 4, 24, 0.4), (33, 6, 128, 2056, 0.1), (9, 32, 40, 264, 0.2), (300, 8, 256, 520, 0.0),
                                               (3, 17, 20, 16392, 0.1), (2, 8, 16, 4096, 0.0)])
def test_combine_gradient(M, topk, E, N, absent):
    pos, z, dy, w = _problem(M, topk, E, N, absent, M + N)
    keep = torch.full((M * topk, N), 9.0, dtype=BF).cuda()
    dz, dw = dg.dg_moe_combine_grad(dy.cuda(), z.cuda(), torch.from_numpy(pos).cuda(), w.cuda(), dz=keep)
    used = np.zeros(M * topk, bool)
    used[pos[pos >= 0]] = True
    want = torch.full((M * topk, N), 9.0, dtype=BF)
    for m in range(M):
        for k in range(topk):
            if pos[m, k] >= 0:
                want[pos[m, k]] = (w[m, k] * dy[m].float()).to(BF)
    assert torch.equal(dz.cpu(), want)
    zz = np.where((pos >= 0)[..., None], z.double().numpy()[np.maximum(pos, 0)], 0.0)
    prod = dy.double().numpy()[:, None] * zz
    # fused multiply-adds and additions in a tree: at most N roundings of 2^-24 of the terms' sizes
    assert (np.abs(dw.cpu().double().numpy() - prod.sum(-1)) <= N * 2.0 ** -24 * np.abs(prod).sum(-1)).all()
    again = dg.dg_moe_combine_grad(dy.cuda(), z.cuda(), torch.from_numpy(pos).cuda(), w.cuda())
    assert torch.equal(again[1], dw) and (again[0].cpu()[~used] == 0).all()


def test_gradients_against_differences():
    """loss = sum(g * combine(experts(gather(x)))) with experts z = 2 xs - 0.5, in 64 bits by central differences (it is
    bilinear in x and w, so they are exact), against the library's own chain."""
    M, topk, E, N = 6, 3, 5, 16
    ids = _ids(M, topk, E, 3, 0.2)
    _, pos, slots = R.moe_sort(ids, E)
    pc = torch.from_numpy(pos).cuda()
    g = torch.Generator().manual_seed(4)
    x, dy, w = torch.randn((M, N), generator=g).to(BF), torch.randn((M, N), generator=g).to(BF), torch.rand((M, topk), generator=g)
    xs = dg.dg_moe_gather(x.cuda(), pc, xs=torch.zeros((M * topk, N), dtype=BF, device="cuda"))
    z = (2 * xs.float() - 0.5).to(BF)
    dz, dw = dg.dg_moe_combine_grad(dy.cuda(), z, pc, w.cuda())
    dx = dg.dg_moe_combine((2 * dz.float()).to(BF), pc).cpu().double()

    def loss(xv, wv):
        zv = 2 * xv[:, None].expand(M, topk, N) - 0.5
        y = (torch.where(torch.from_numpy(pos)[..., None] >= 0, zv, torch.zeros_like(zv)) * wv[..., None]).sum(1)
        return float((dy.double() * y).sum())

    xd, wd, h = x.double(), w.double(), 2.0 ** -6
    for m in range(M):
        for n in (0, 5, N - 1):
            e = torch.zeros_like(xd)
            e[m, n] = h
            diff = (loss(xd + e, wd) - loss(xd - e, wd)) / (2 * h)
            size = 2 * float(w[m].sum()) * abs(float(dy[m, n]))
            assert abs(float(dx[m, n]) - diff) <= size * 3 * 2.0 ** -8 + 1e-9      # z, dz and dx rounded to bf16
        for k in range(topk):
            e = torch.zeros_like(wd)
            e[m, k] = h
            diff = (loss(xd, wd + e) - loss(xd, wd - e)) / (2 * h)
            size = float((dy[m].double().abs() * (2 * xd[m].abs() + 0.5)).sum())
            assert abs(float(dw[m, k]) - diff) <= size * 2.0 ** -8 * 1.01 + 1e-9    # z rounded to bf16
    assert sum(p >= 0 for p in pos.reshape(-1)) < M * topk


def test_streams_and_graph():
    M, topk, E, N = 50, 4, 32, 128
    cases = [torch.from_numpy(_ids(M, topk, E, s, 0.1)).cuda() for s in range(3)]
    x = torch.randn((M, N)).to(BF).cuda()
    w = torch.rand((M, topk)).cuda()

    def step(ids, stream=None):
        offsets, pos, slots = dg.dg_moe_sort(ids, E, stream=stream)
        xs = dg.dg_moe_gather(x, pos, stream=stream)
        return offsets, pos, slots, dg.dg_moe_combine(xs, pos, w, stream=stream), dg.dg_moe_combine_grad(x, xs, pos, w, stream=stream)[1]

    want = [[t.clone() for t in step(c)] for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for c, v in zip(cases, want):
        got = step(c, side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, v))
    ids = cases[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(ids)
    for c, v in zip(cases, want):
        ids.copy_(c)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, v))


def test_routed_layer_through_sorted_rows():
    """Router -> sort -> gather -> one 8-bit linear for each expert's rows -> combine, against the definition: every
    (token, expert) product alone, weighted and added in slot order."""
    M, topk, E, K, N = 40, 3, 8, 256, 192
    g = torch.Generator().manual_seed(0)
    x = torch.randn((M, K), generator=g).to(BF).cuda()
    logits = torch.randn((M, E), generator=g).cuda()
    logits[:, 5] = float("-inf")                              # an expert without rows
    packed = [dg.dg_quant_i8_rowscale((torch.randn((N, K), generator=g) * K ** -0.5).to(BF).cuda()) for _ in range(E)]
    ids, w = dg.dg_moe_route(logits, topk)
    offsets, pos, slots = dg.dg_moe_sort(ids, E)
    xs = dg.dg_moe_gather(x, pos)
    z = torch.empty((M * topk, N), dtype=BF, device="cuda")
    at = offsets.tolist()
    assert at[6] == at[5] and at[-1] == M * topk
    for e in range(E):
        if at[e + 1] > at[e]:
            dg.dg_gemv_i8_rowscale(xs[at[e]:at[e + 1]], *packed[e], y=z[at[e]:at[e + 1]])
    y = dg.dg_moe_combine(z, pos, w)
    ids, w, idl = ids.cpu(), w.cpu(), ids.tolist()
    for m in range(M):
        acc = torch.zeros(N, dtype=torch.float64)
        size = torch.zeros(N, dtype=torch.float64)
        for k in range(topk):
            one = dg.dg_gemv_i8_rowscale(x[m:m + 1], *packed[idl[m][k]])[0].cpu().double()
            acc += float(w[m, k]) * one
            size += abs(float(w[m, k])) * one.abs()
        assert ((y[m].cpu().double() - acc).abs() <= 2.0 ** -8 * acc.abs() + topk * 2.0 ** -23 * size + 1e-38).all()
