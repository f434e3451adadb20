"""Plain references of the 4-bit formats, the routing and the log-probabilities (numpy).

What an operator decides (codes, scales) is decided in binary32 and restated in numpy's
binary32, one correctly rounded operation at a time; sums are taken in 64 bits.
"""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {0: 32, 1: 16}                       # DG_FP4_MX, DG_FP4_NV


def e4m3_table():
    """The 127 non-negative finite e4m3 values, by code."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e > 0, 2.0 ** (e - 7.0) * (1 + m / 8.0), m * 2.0 ** -9)


def nearest_even(v, grid):
    """Index of the grid value nearest to each v >= 0, ties to the even index, saturating."""
    v = np.minimum(v.astype(np.float64), grid[-1])
    hi = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = v - grid[lo], grid[hi] - v
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def fp4_quant(x, fmt, g=1.0):
    """(codes [M, K] 0..15, scale bytes [M, K / block]) of bf16 values x given as float32."""
    b = BLOCK[fmt]
    M, K = x.shape
    xb = x.astype(np.float32).reshape(M, K // b, b)
    g = np.float32(g)
    bad = ~np.isfinite(xb).all(-1)
    xs = np.where(bad[..., None], np.float32(0), xb)
    amax = np.abs(xs).max(-1)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        if fmt == 0:
            e = np.where(amax > 0, np.frexp(amax)[1] - 3, -127)
            e = np.maximum(e, -127)
            byte = (e + 127).astype(np.uint8)
            v = xs.astype(np.float64) * np.exp2(-e.astype(np.float64))[..., None]      # exact
        else:
            q = (amax / (np.float32(6) * g)).astype(np.float32)
            byte = nearest_even(q, e4m3_table()).astype(np.uint8)
            s = e4m3_table()[byte].astype(np.float32)
            sg = (s * g).astype(np.float32)[..., None]
            v = np.where(byte[..., None] > 0, (xs / sg).astype(np.float32), np.float32(0))
    code = nearest_even(np.abs(v), E2M1).astype(np.uint8)
    dead = bad | (byte == 0) if fmt == 1 else bad | (amax == 0)
    code = np.where(dead[..., None], 0, code | (np.signbit(v).astype(np.uint8) << 3))
    byte = np.where(bad, 0xFF if fmt == 0 else 0x7F, byte).astype(np.uint8)
    return code.reshape(M, K).astype(np.uint8), byte


def fp4_scale_value(byte, fmt):
    if fmt == 0:
        return np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    return np.where(byte == 127, np.nan, e4m3_table()[np.minimum(byte, 126)])


def fp4_value(code):
    return np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]


def fp4_values(code, byte, fmt):
    """Codes times block scales (no tensor scale), 64 bits, exact."""
    b = BLOCK[fmt]
    M, K = code.shape
    return (fp4_value(code).reshape(M, K // b, b) * fp4_scale_value(byte, fmt)[..., None]).reshape(M, K)


def pack(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    out = np.empty((q.shape[0], 2 * q.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def tile(byte):
    """Scale bytes [R, nb] to their tiles, element by element as the layout is stated."""
    R, nb = byte.shape
    out = np.zeros(((R + 127) // 128, (nb + 3) // 4, 512), np.uint8)
    r, b = np.meshgrid(np.arange(R), np.arange(nb), indexing="ij")
    out[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = byte
    return out


def route(x, topk, sigmoid, bias=None, n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0):
    """(ids, w, margin): margin is the smallest distance between a key (or a run's score) that
    was taken and one that was not or came after it, 0 distances (true ties) aside."""
    x = x.astype(np.float64)
    M, E = x.shape
    ids = np.full((M, topk), -1, np.int32)
    w = np.zeros((M, topk))
    margin = np.full(M, np.inf)
    for t in range(M):
        can = x[t] > -np.inf                                   # (NaN: not available)
        if not can.any():
            continue
        with np.errstate(over="ignore", invalid="ignore"):
            if sigmoid:
                p = 1.0 / (1.0 + np.exp(-x[t]))
            else:
                m = x[t][can].max()
                e = np.where(can, np.where(x[t] == m, 1.0, np.exp(x[t] - m)), 0.0)
                p = e / e.sum()
        p = p.astype(np.float32).astype(np.float64)            # (scores that underflow are 0)
        key = np.where(can, p + (bias.astype(np.float64) if bias is not None else 0.0), -np.inf)

        def order(v, n):
            o = sorted(range(len(v)), key=lambda i: (-v[i], i))
            for a in range(min(n, len(v) - 1)):
                hi, lo = v[o[a]], v[o[a + 1]]
                if lo > -np.inf and hi != lo:
                    margin[t] = min(margin[t], hi - lo)
            return o[:n]

        if n_group > 1:
            runs = key.reshape(n_group, -1)
            gs = []
            for r in runs:
                best = sorted(r, reverse=True)[:group_top]
                gs.append(-np.inf if best[0] == -np.inf else sum(b for b in best if b > -np.inf))
            keep = set(order(np.array(gs), topk_group))
            size = E // n_group
            key = np.array([k if i // size in keep else -np.inf for i, k in enumerate(key)])
        for s, i in enumerate(order(key, topk)):
            if key[i] > -np.inf:
                ids[t, s], w[t, s] = i, p[i]
        if renorm:
            tot = w[t].sum()
            w[t] = w[t] / tot if tot > 0 else 0.0
    return ids, w * scale, margin


def logprobs(x, tokens, n_top, scale=1.0):
    """dict of logprob, rank, entropy, top_ids, top_logprobs in 64 bits."""
    x = x.astype(np.float64)
    M, V = x.shape
    out = {"logprob": np.full(M, np.nan), "rank": np.full(M, -1, np.int64), "entropy": np.zeros(M),
           "top_ids": np.full((M, n_top), -1, np.int64), "top_logprobs": np.full((M, n_top), -np.inf)}
    for m in range(M):
        z = x[m] * scale
        poison = np.isnan(z).any() or (z == np.inf).any()
        live = z > -np.inf
        lse = np.nan
        if poison:
            out["entropy"][m] = np.nan
        elif live.any():
            top = z[live].max()
            s = np.exp(z[live] - top).sum()                    # (differences: lse - sum p z would cancel)
            lse = top + np.log(s)
            out["entropy"][m] = np.log(s) - (np.exp(z[live] - top) * (z[live] - top)).sum() / s
        else:
            lse = np.inf                                       # everything masked

        def lp(v):
            if poison:
                return np.nan
            if lse == np.inf or v == -np.inf:
                return -np.inf
            top = z[live].max()
            return (v - top) - np.log(np.exp(z[live] - top).sum())

        if tokens is not None and 0 <= tokens[m] < V:
            out["logprob"][m] = lp(z[tokens[m]])
            out["rank"][m] = (x[m] > x[m][tokens[m]]).sum()
        order = [i for i in np.lexsort((np.arange(V), -np.where(np.isnan(x[m]), -np.inf, x[m]))) if live[i]][:n_top]
        for k, i in enumerate(order):
            out["top_ids"][m, k], out["top_logprobs"][m, k] = i, lp(z[i])
    return out
