"""Penalties, biases and masks on logits on the GPU: every entry to the last bit."""
import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg
from tests import _ref_more as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _edits(M, V, L, B, mask, seed):
    g = np.random.default_rng(seed)
    e = {}
    if L:
        e["tokens"] = (g.random((M, L)) ** 3 * (V + 2)).astype(np.int32) - 1          # (-1 and V among them)
        e["lengths"] = g.integers(0, L + 1, M).astype(np.int32)
        e["lengths"][0] = L
        e["prompt_lengths"] = (g.random(M) * (e["lengths"] + 1)).astype(np.int32)
        e["repetition"] = (0.7 + g.random(M)).astype(np.float32)
        e["frequency"] = (g.random(M) - 0.3).astype(np.float32)
        e["presence"] = (g.random(M) - 0.3).astype(np.float32)
    if B:
        e["bias_ids"] = g.integers(-1, V + 1, (M, B)).astype(np.int32)
        e["bias_ids"][:, B // 2:] = np.where(g.random((M, B - B // 2)) < 0.5, e["bias_ids"][:, :B - B // 2], e["bias_ids"][:, B // 2:])
        e["bias"] = (8 * g.random((M, B)) - 4).astype(np.float32)
        if L:
            e["bias_ids"][:, 0] = e["tokens"][:, 0]
    if mask:
        keep = np.array([0.5, 0.0, 1.0, 0.02])[np.arange(M) % 4]
        words = (V + 31) // 32
        bits = (g.random((M, words, 32)) < keep[:, None, None]).astype(np.uint64)
        e["mask"] = (bits << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)
    return e


def _x(M, V, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((M, V), generator=g) * 4).to(dtype)


def _same(got, want, dtype):
    if dtype == BF:
        got, want = got.cpu().contiguous().view(torch.int16).numpy(), R.bf16_of(want)
    else:
        got, want = got.cpu().contiguous().view(torch.int32).numpy(), want.view(np.int32)
    np.testing.assert_array_equal(got, want)


def _gpu(e):
    return {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in e.items()}


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("M,V,L,B,mask", [(1, 1, 3, 1, True), (1, 31, 9, 2, True), (3, 33, 0, 0, True), (2, 500, 40, 0, False), (5, 517, 0, 9, False),
                                          (4, 2048, 100, 30, True), (7, 4099, 300, 17, True), (1, 40003, 2000, 50, True), (40, 20000, 64, 5, True),
                                          (330, 1003, 20, 3, True), (2, 100003, 900, 300, False), (1400, 1003, 20, 3, True), (1300, 2000, 5, 70, False),
                                          (90, 24000, 300, 1024, True), (700, 3001, 500, 0, True), (40, 40001, 0, 9, True), (3, 2001, 9000, 5, True)])
def test_every_entry(dtype, M, V, L, B, mask):
    x, e = _x(M, V, dtype, M + V), _edits(M, V, L, B, mask, M + V)
    want = R.adjust(R.f32(x), **e)
    xc = x.cuda()
    out = torch.full_like(xc, 5.0)
    _same(dg.dg_logits_adjust(xc, out=out, **_gpu(e)), want, dtype)
    assert torch.equal(xc.cpu(), x)                            # the input stays
    assert dg.dg_logits_adjust(xc, **_gpu(e)) is xc            # in place
    _same(xc, want, dtype)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("off,pad,opad", [(0, 5, 5), (1, 7, 8), (3, 2, 1), (8, 8, 16), (4, 13, 0)])
def test_strides_and_alignment(dtype, off, pad, opad):
    M, V, L, B = 5, 3001, 50, 6
    base = torch.full((M, off + V + pad), 2.0, dtype=dtype)
    x = base[:, off:off + V]
    x.copy_(_x(M, V, dtype, 1))
    e = _edits(M, V, L, B, True, 2)
    want = R.adjust(R.f32(x), **e)
    tok = torch.zeros((M, L + 9), dtype=torch.int32)
    tok[:, 4:4 + L] = torch.from_numpy(e["tokens"])
    words = e["mask"].shape[1]
    mk = torch.full((M, words + 3), -1, dtype=torch.int32)
    mk[:, 1:1 + words] = torch.from_numpy(e["mask"])
    dev = {**_gpu(e), "tokens": tok.cuda()[:, 4:4 + L], "mask": mk.cuda()[:, 1:1 + words]}
    bc = base.cuda()
    ob = torch.full((M, V + opad), 3.0, dtype=dtype).cuda()
    _same(dg.dg_logits_adjust(bc[:, off:off + V], out=ob[:, :V], **dev), want, dtype)
    assert (ob[:, V:] == 3).all()
    dg.dg_logits_adjust(bc[:, off:off + V], **dev)
    _same(bc[:, off:off + V], want, dtype)
    assert (bc[:, :off] == 2).all() and (bc[:, off + V:] == 2).all()


def test_each_edit_alone_and_none():
    M, V, L, B = 3, 700, 60, 8
    x, e = _x(M, V, torch.float32, 5), _edits(M, V, L, B, True, 6)
    lists = ("tokens", "lengths", "prompt_lengths")
    for names in (lists + ("repetition",), lists + ("frequency",), lists + ("presence",), ("tokens", "repetition", "presence"), ("tokens", "lengths", "frequency"),
                  ("tokens", "prompt_lengths", "repetition"), lists, ("bias_ids", "bias"), ("mask",), ()):
        part = {k: e[k] for k in names}
        xc = x.cuda()
        _same(dg.dg_logits_adjust(xc, out=torch.empty_like(xc), **_gpu(part)), R.adjust(x.numpy(), **part), torch.float32)
        _same(dg.dg_logits_adjust(xc, **_gpu(part)), R.adjust(x.numpy(), **part), torch.float32)
    xc = x.cuda()
    empty = torch.empty((M, 0), dtype=torch.int32).cuda()
    _same(dg.dg_logits_adjust(xc, tokens=empty, lengths=torch.zeros(M, dtype=torch.int32).cuda(), repetition=torch.ones(M).cuda()), x.numpy(), torch.float32)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_extreme_logits(dtype):
    """Infinities, NaN and the type's largest and lowest values, named by the lists or not, masked or not."""
    V, big = 64, torch.finfo(dtype).max
    x = torch.zeros((2, V), dtype=dtype)
    x[:, :8] = torch.tensor([float("inf"), -float("inf"), float("nan"), big, -big, 0.0, -0.0, 1.0])
    x[:, 8:16] = x[:, :8]
    e = {"tokens": np.tile(np.arange(8, dtype=np.int32), (2, 1)), "prompt_lengths": np.array([4, 0], np.int32), "repetition": np.array([1.5, 0.5], np.float32),
         "frequency": np.array([0.5, -0.5], np.float32), "presence": np.array([0.25, 0.0], np.float32), "bias_ids": np.tile(np.array([[0, 1, 2, 3, 30]], np.int32), (2, 1)),
         "bias": np.array([[1, 2, 3, -4, 5]] * 2, np.float32)}
    m = np.full((2, 2), -1, np.int32)
    m[1, 0] = 0x0000FF00
    for mask in (None, m):
        ed = dict(e, mask=mask) if mask is not None else e
        want = R.adjust(R.f32(x), **ed)
        out = dg.dg_logits_adjust(x.cuda(), **_gpu(ed)).cpu().float().numpy()
        np.testing.assert_array_equal(np.isnan(out), np.isnan(want))
        want = torch.from_numpy(want).to(dtype).float().numpy()
        np.testing.assert_array_equal(out[~np.isnan(out)], want[~np.isnan(want)])


def test_lengths_past_their_range_and_many_repeats():
    M, V, L = 4, 300, 5000
    x = _x(M, V, torch.float32, 1)
    e = {"tokens": np.zeros((M, L), np.int32), "lengths": np.array([L + 50, -3, 2 ** 31 - 1, L], np.int32), "prompt_lengths": np.array([-5, 9, L - 1, 2 ** 31 - 1], np.int32),
         "frequency": np.full(M, 0.01, np.float32), "repetition": np.full(M, 1.3, np.float32)}
    e["tokens"][:, ::2] = 7
    _same(dg.dg_logits_adjust(x.cuda(), **_gpu(e)), R.adjust(x.numpy(), **e), torch.float32)


def test_streams_and_graph():
    M, V, L, B = 6, 5000, 80, 7
    xs = [_x(M, V, BF, s) for s in range(3)]
    es = [_edits(M, V, L, B, True, s) for s in range(3)]
    want = [R.adjust(R.f32(x), **e) for x, e in zip(xs, es)]
    side = torch.cuda.Stream()
    for x, e, v in zip(xs, es, want):
        xc, dev = x.cuda(), _gpu(e)
        side.wait_stream(torch.cuda.current_stream())
        dg.dg_logits_adjust(xc, stream=side, **dev)
        side.synchronize()
        _same(xc, v, BF)
    x, dev = xs[0].cuda(), _gpu(es[0])
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.dg_logits_adjust(x, out=out, **dev)
    for i in range(3):
        x.copy_(xs[i])
        for k, t in _gpu(es[i]).items():
            dev[k].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        _same(out, want[i], BF)


def test_head_edits_and_log_probabilities():
    """Head -> edits -> log-probabilities, as a sampler runs them: the probabilities of the edited logits."""
    M, V, K = 3, 1000, 128
    g = torch.Generator().manual_seed(0)
    x = torch.randn((M, K), generator=g).to(BF).cuda()
    W = (torch.randn((V, K), generator=g) * 40).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    logits, _ = dg.dg_head_fp8_argmax(x, W, torch.tensor([2e-3]).cuda())
    e = _edits(M, V, 30, 4, True, 3)
    want = torch.from_numpy(R.adjust(R.f32(logits), **e)).to(BF).double()
    dg.dg_logits_adjust(logits, **_gpu(e))
    tok = torch.where(want.amax(-1) > -float("inf"), want.argmax(-1), torch.zeros((), dtype=torch.int64))
    r = dg.dg_logprobs(logits, tok.cuda(), n_top=3)
    lp = (want - torch.logsumexp(want, -1, keepdim=True)).gather(1, tok[:, None])[:, 0]
    live = torch.isfinite(want.amax(-1))
    assert live.tolist() == [True, False, True]               # one row's grammar allows nothing
    assert ((r["logprob"].cpu().double() - lp)[live].abs() < 1e-4).all()
    assert r["logprob"][1] == -float("inf") and (r["top_ids"][1] == -1).all()
    assert (r["rank"].cpu()[live] == 0).all()
