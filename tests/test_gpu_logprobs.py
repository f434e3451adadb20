"""Log-probabilities, rank, entropy and alternatives against a plain 64-bit reference.

Bounds: a thread adds up to about 500 terms in binary32 before the sums are joined, so the
sums are within 500 * 2^-24 = 3e-5 relative (plus 2^-22 for each power of two): 4e-5 on a
logprob, plus 2^-21 of it for its own roundings; the entropy has two such sums, 1e-4 (1 + H).
Ranks and alternatives compare logits as they are and must agree exactly.
"""
import math

import numpy as np
import pytest
import torch

import gemv_dg_bf16_gb300 as dg
from tests import _ref64 as R

pytestmark = pytest.mark.gpu

INF = math.inf


def _near(got, want, rel, absolute):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)), (got, want)
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
    err = np.abs(got[fin] - want[fin])
    assert (err <= rel * np.abs(want[fin]) + absolute).all(), err.max()


def _check(x, tokens, n_top=5, scale=1.0):
    r = dg.dg_logprobs(x, tokens, n_top=n_top, scale=scale)
    ref = R.logprobs(x.float().cpu().numpy(), None if tokens is None else tokens.cpu().numpy(), n_top, scale)
    if tokens is not None:
        _near(r["logprob"].cpu(), ref["logprob"], 2.0 ** -21, 4e-5)
        assert np.array_equal(r["rank"].cpu().numpy(), ref["rank"])
    _near(r["entropy"].cpu(), ref["entropy"], 1e-4, 1e-4)
    if n_top:
        assert np.array_equal(r["top_ids"].cpu().numpy(), ref["top_ids"])
        _near(r["top_logprobs"].cpu(), ref["top_logprobs"], 2.0 ** -21, 4e-5)
    return r


def _logits(M, V, seed, dtype=torch.bfloat16, std=2.5):
    return (std * torch.randn((M, V), generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


def _tokens(M, V, seed):
    return torch.randint(0, V, (M,), generator=torch.Generator().manual_seed(seed)).cuda()


SHAPES = [(1, 1), (2, 3), (3, 7), (4, 8), (2, 9), (5, 31), (3, 511), (2, 4096), (3, 4099), (4, 20001), (2, 32769),
          (1, 65541), (1, 248320), (9, 50000), (160, 9001)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V", SHAPES)
def test_logprobs_shapes(cuda_device, M, V, dtype):
    _check(_logits(M, V, M + V, dtype), _tokens(M, V, V), n_top=min(20, 1 + V // 2), scale=1.0 if M % 2 else 1.3)


@pytest.mark.parametrize("n_top", [0, 1, 2, 7, 31, 32])
def test_logprobs_counts_of_alternatives(cuda_device, n_top):
    for V in (5, 1000, 40001):
        _check(_logits(3, V, n_top, torch.float32), _tokens(3, V, 1), n_top=n_top)


def test_logprobs_many_rows_and_the_same_bits_again(cuda_device):
    x = _logits(700, 3001, 4)
    tok = _tokens(700, 3001, 5)
    a = _check(x, tok, n_top=4)
    for _ in range(3):
        b = dg.dg_logprobs(x, tok, n_top=4)
        assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [5, 130, 4099, 30011])
def test_logprobs_many_short_rows(cuda_device, dtype, V):
    """Rows that take small thread blocks, equal values and masked rows among them."""
    M = 310
    x = _logits(M, V, V, dtype)
    x[3] = 1.5
    x[4, ::2] = -INF
    x[5] = -INF
    x[6] = torch.finfo(dtype).min
    x[7, V // 2] = float("nan")
    _check(x, _tokens(M, V, 3), n_top=min(V, 12))
    one = dg.dg_logprobs(x[:9].contiguous(), n_top=min(V, 12))     # (a few rows take large ones)
    many = dg.dg_logprobs(x, n_top=min(V, 12))
    assert torch.equal(one["top_ids"], many["top_ids"][:9])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprobs_ties_and_orders(cuda_device, dtype):
    """Equal logits, sorted rows, the largest ones all in one thread's share, signed zeros."""
    V = 70000
    x = torch.zeros((9, V))
    x[1] = -1.0e9                                              # a finite mask for most
    x[1, [5, 69999, 333]] = torch.tensor([1.0, 2.0, 1.0])
    x[2] = torch.arange(V) / V * 8
    x[3] = -torch.arange(V) / V * 8
    x[4] = torch.randint(-3, 4, (V,), generator=torch.Generator().manual_seed(1)).float()
    x[5] = -5.0
    x[5, 7::4096] = torch.arange(len(range(7, V, 4096))).float()
    x[5, 8::4096] = 3.0
    x[6, ::2] = -0.0
    x[7] = -1.0
    x[7, 64000:] = 1.0
    x[8] = torch.where(torch.arange(V) % 512 < 9, 4.0, -4.0)
    for cols in (V, 4097, 33):
        y = x[:, :cols].to(dtype).cuda()
        _check(y, _tokens(9, cols, 2), n_top=20)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprobs_masks_infinities_and_nan(cuda_device, dtype):
    low = torch.finfo(dtype).min
    V = 5003
    x = _logits(14, V, 3, dtype)
    tok = _tokens(14, V, 4)
    x[0] = -INF                                                # nothing left
    x[1, 1:] = -INF                                            # one left
    tok[1] = 0
    x[2, 100:] = -INF
    tok[2] = 4000                                              # a masked token
    x[3] = low                                                 # all at the type's lowest: uniform
    x[4, 3:] = low
    x[5, 17] = float("nan")
    x[6] = float("nan")
    x[7, 9] = INF
    tok[8], tok[9] = -1, V                                     # not tokens
    x[10, ::2] = -INF
    x[11, :2500] = low
    x[11, 2500:] = -INF                                        # lowest beside masked: only the former count
    x[12, 40:] = -1.0e30
    x[13] = -5.0e29
    for scale in (1.0, 0.7):
        _check(x, tok, n_top=6, scale=scale)


def test_logprobs_large_offsets_keep_differences(cuda_device):
    """Logits far from zero: only differences count."""
    x = _logits(4, 3000, 8, torch.float32)
    for off in (1.0e3, -1.0e4):
        y = x + off
        _check(y, _tokens(4, 3000, 1))


def test_logprobs_extreme_scales(cuda_device):
    x = _logits(4, 3000, 8, torch.float32)
    _check(x, _tokens(4, 3000, 1), scale=1e-6)
    y = (x * 4).round() / 4                                    # exact products, a sharp distribution
    _check(y, _tokens(4, 3000, 1), scale=64.0)


def test_logprobs_strided_misaligned_and_optional(cuda_device):
    for dtype in (torch.bfloat16, torch.float32):
        base = _logits(6, 9000, 6, dtype)
        tok = _tokens(6, 8001, 2)
        for o in (0, 1, 3, 5, 8):
            ref = dg.dg_logprobs(base[:, o:o + 8001].contiguous(), tok, n_top=3)
            got = _check(base[:, o:o + 8001], tok, n_top=3)
            assert torch.equal(ref["top_ids"], got["top_ids"]) and torch.equal(ref["rank"], got["rank"])
        r = dg.dg_logprobs(base, n_top=2)
        assert r["logprob"] is None and r["rank"] is None
        full = dg.dg_logprobs(base, tok, n_top=2)
        assert torch.equal(r["entropy"], full["entropy"]) and torch.equal(r["top_ids"], full["top_ids"])
        assert dg.dg_logprobs(base, tok)["top_ids"] is None


def test_logprobs_offsets_past_32_bits(cuda_device):
    M, V = 9000, 248320                                        # 2.2e9 logits
    x = torch.empty((M, V), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(5))
    tok = torch.randint(0, V, (M,), device="cuda")
    r = dg.dg_logprobs(x, tok, n_top=2)
    one = dg.dg_logprobs(x[-200:].contiguous(), tok[-200:].contiguous(), n_top=2)
    assert all(torch.equal(r[k][-200:], one[k]) for k in r)


def test_logprobs_over_the_head_in_a_graph(cuda_device):
    """Head, then log-probabilities of its pick, on a captured stream."""
    from synth import decode_inputs as S
    x, Wq, scale = S.head_inputs(3, 4099, 512, device=cuda_device)
    ws = dg.workspace(dg.DG_OP_HEAD_FP8_ARGMAX, 3, 4099, 512)
    logits, pick = dg.dg_head_fp8_argmax(x, Wq, scale, ws=ws)
    want = dg.dg_logprobs(logits, pick.long(), n_top=4)
    torch.cuda.synchronize()
    bufs = {k: torch.empty_like(v) for k, v in want.items()}
    tok = pick.long()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.dg_head_fp8_argmax(x, Wq, scale, logits=logits, argmax=pick, ws=ws)
        dg.dg_logprobs(logits, tok, n_top=4, **bufs)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(bufs[k], want[k]) for k in want)
    # (the head picks on fp32 logits: its pick is among the largest bf16 ones)
    top = logits.float().amax(-1)
    assert torch.equal(logits.float().gather(1, tok[:, None])[:, 0], top) and (want["rank"] == 0).all()


def test_logprobs_refusals(cuda_device):
    x = _logits(2, 64, 1)
    tok = _tokens(2, 64, 1)
    for kw, status in ((dict(n_top=33), 3), (dict(n_top=-1), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
                       (dict(scale=1e7), 1)):
        with pytest.raises(dg.DGError) as e:
            dg.dg_logprobs(x, tok, **kw)
        assert e.value.status == status, kw
    with pytest.raises(ValueError):
        dg.dg_logprobs(x, tok.int())
    with pytest.raises(ValueError):
        dg.dg_logprobs(x.t(), tok)
