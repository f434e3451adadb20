"""Operators around a decode step, as they are measured: the microscaled 4-bit quantisation and
linear, the routing of tokens to experts, and the log-probabilities of given tokens.

listed() names the cases, draw() gives more of the same ranges, prepare() makes what a serving
program has in hand, run() makes one pass -- with elementary torch operations where `own` is
false, through this library's entry points where it is true -- work() counts what a pass cannot do
without, and exact() restates each operator in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
# Block length and scale bytes of the two 4-bit formats: "mx" has 32-element blocks with a
# power-of-two scale (e8m0), "nv" has 16-element blocks with an e4m3 scale under one fp32 scale
# for the whole tensor.
BLOCK = {"mx": 32, "nv": 16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # 16 token rows entering a 4-bit linear: one small launch, latency counts.
        {"name": "quantise 16 rows", "op": "quant", "fmt": "nv", "M": 16, "K": 4096, "g": True},
        # A gate/up weight matrix converted when a model is loaded: pure bandwidth.
        {"name": "quantise weights", "op": "quant", "fmt": "mx", "M": 24576, "K": 4096, "g": False},
        # One decoding sequence through a square projection: the smallest weight stream.
        {"name": "linear 1 row", "op": "linear", "fmt": "nv", "M": 1, "N": 4096, "K": 4096, "g": True},
        # A small decode batch through a wide projection.
        {"name": "linear 16 rows", "op": "linear", "fmt": "mx", "M": 16, "N": 12288, "K": 4096, "g": False},
        # A ragged batch and ragged weight rows with a long reduction (a down projection).
        {"name": "linear 77 rows ragged", "op": "linear", "fmt": "nv", "M": 77, "N": 4099, "K": 12288, "g": True},
        # The largest batch of the linear (a chunk of a prompt) through gate/up rows.
        {"name": "linear 512 rows", "op": "linear", "fmt": "nv", "M": 512, "N": 24576, "K": 4096, "g": True},
        # One token routed: sigmoid scores, a balance bias, 4 of 8 groups, 8 of 256 experts.
        {"name": "route 1 token", "op": "route", "M": 1, "E": 256, "topk": 8, "score": "sigmoid", "bias": True,
         "n_group": 8, "topk_group": 4, "group_top": 2, "renorm": True, "scale": 2.5, "bits": 32, "masked": False},
        # A decode batch over 128 experts by softmax, logits straight from a bf16 linear.
        {"name": "route 16 tokens", "op": "route", "M": 16, "E": 128, "topk": 6, "score": "softmax", "bias": False,
         "n_group": 1, "topk_group": 1, "group_top": 1, "renorm": True, "scale": 1.0, "bits": 16, "masked": True},
        # A long prompt's tokens routed at once.
        {"name": "route 32768 tokens", "op": "route", "M": 32768, "E": 256, "topk": 8, "score": "sigmoid",
         "bias": True, "n_group": 8, "topk_group": 4, "group_top": 2, "renorm": True, "scale": 2.5, "bits": 32,
         "masked": False},
        # One sampled token's log-probability with its alternatives, over the fp8 head's vocabulary.
        {"name": "logprobs 1 row", "op": "logprobs", "M": 1, "V": 248320, "top": 20, "bits": 16, "scale": 1.0,
         "masked": False},
        # A decode batch with a temperature and a grammar's mask, a vocabulary that no vector divides.
        {"name": "logprobs 8 rows odd", "op": "logprobs", "M": 8, "V": 100003, "top": 5, "bits": 32, "scale": 1.25,
         "masked": True},
        # A prompt scored token by token.
        {"name": "logprobs 2048 rows", "op": "logprobs", "M": 2048, "V": 248320, "top": 5, "bits": 16, "scale": 1.0,
         "masked": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "route", "logprobs"])
    fmt = rng.choice(["mx", "nv"])
    if op == "quant":
        K = 32 * _log_int(rng, 1, 384)
        M = _log_int(rng, 1, min(24576, 24576 * 4096 // K))
        return {"op": op, "fmt": fmt, "M": M, "K": K, "g": fmt == "nv" and rng.random() < 0.7}
    if op == "linear":
        K = 32 * _log_int(rng, 2, 384)
        N = _log_int(rng, 16, 24576)
        M = _log_int(rng, 1, max(1, min(512, 512 * 24576 * 4096 // (N * K))))
        return {"op": op, "fmt": fmt, "M": M, "N": N, "K": K, "g": fmt == "nv" and rng.random() < 0.7}
    if op == "route":
        E = rng.choice([_log_int(rng, 2, 1024), 32 * rng.randint(1, 32)])
        M = _log_int(rng, 1, min(32768, 32768 * 256 // E))
        n_group = rng.choice([1] + [g for g in (2, 3, 4, 5, 8, 16) if E % g == 0 and E // g >= 2])
        topk_group = rng.randint(1, n_group)
        topk = rng.randint(1, min(16, topk_group * (E // n_group)))
        return {"op": op, "M": M, "E": E, "topk": topk, "score": rng.choice(["sigmoid", "softmax"]),
                "bias": rng.random() < 0.5, "n_group": n_group, "topk_group": topk_group,
                "group_top": rng.choice([1, 2]), "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, round(rng.uniform(1.0, 3.0), 3)]), "bits": rng.choice([16, 32]),
                "masked": rng.random() < 0.3}
    V = _log_int(rng, 500, 248320)
    bits = rng.choice([16, 32])
    M = _log_int(rng, 1, min(4096, 2048 * 248320 * 16 // (V * bits)))
    return {"op": op, "M": M, "V": V, "top": rng.choice([0, rng.randint(1, 20)]), "bits": bits,
            "scale": rng.choice([1.0, round(rng.uniform(0.5, 2.0), 3)]), "masked": rng.random() < 0.3}


def work(c):
    if c["op"] == "quant":          # bf16 in, codes and scales made, their values back as bf16
        M, K = c["M"], c["K"]
        held = M * K // 2 + M * K // BLOCK[c["fmt"]]
        return {"bytes": 2 * M * K + 2 * held + 2 * M * K, "flops": 3 * M * K}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": N * K // 2 + N * K // BLOCK[c["fmt"]] + 2 * M * K + 2 * M * N, "flops": 2 * M * N * K}
    if c["op"] == "route":
        M, E, k = c["M"], c["E"], c["topk"]
        return {"bytes": M * E * c["bits"] // 8 + (4 * E if c["bias"] else 0) + 8 * M * k, "flops": 4 * M * E}
    M, V = c["M"], c["V"]
    return {"bytes": M * V * c["bits"] // 8 + M * (8 + 12 + 8 * c["top"]), "flops": 6 * M * V}


# ------------------------------------------------------------------------------- inputs

def _pow2(e):
    """2^e in fp32 of whole numbers -127 <= e <= 127, by its bits (a pow() may round)."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 0x00400000)).int().view(torch.float32)


def _quant_plain(x, fmt, g):
    """(signed values on the e2m1 grid [M, K], scales [M, K / block]) of fp32 x, as the format defines them."""
    b = BLOCK[fmt]
    xb = x.view(x.shape[0], -1, b)
    amax = xb.abs().amax(-1)
    if fmt == "mx":
        _, e = torch.frexp(amax)                                   # amax = m * 2^e, 0.5 <= m < 1
        e = torch.where(amax > 0, e - 3, torch.full_like(e, -127)).clamp(-127, 127)
        s = _pow2(e)
        v = xb * _pow2(-e).unsqueeze(-1)
    else:
        s = (amax / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
        sg = (s * g).unsqueeze(-1)
        v = torch.where(sg > 0, xb / sg, torch.zeros_like(xb))
    a = v.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
            + (a >= 3.5).byte() + (a > 5.0).byte())                # ties to the even code
    q = torch.tensor(E2M1, device=x.device)[code.int()]
    return torch.copysign(q, v).view(x.shape), s


def _tile(s8):
    """Scale bytes [R, nb] -> [ceil(R/128), ceil(nb/4), 512]: in a tile of 128 rows x 4 blocks, row r and block b
    are at byte (r % 32) * 16 + (r // 32) * 4 + b."""
    R, nb = s8.shape
    rt, kt = -(-R // 128), -(-nb // 4)
    pad = torch.zeros((rt * 128, kt * 4), dtype=torch.uint8, device=s8.device)
    pad[:R, :nb] = s8
    return pad.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(rt, kt, 512).contiguous()


def _untile(t, R, nb):
    rt, kt, _ = t.shape
    return t.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:R, :nb]


def _weights(N, K, fmt, g, gen):
    """A weight matrix as a checkpoint holds it: two codes a byte (the lower nibble first), tiled scales."""
    w = torch.randn((N, K), generator=gen, device=DEV) * K ** -0.5
    gw = (w.abs().amax() / 2688.0).reshape(1) if g else None
    q, s = _quant_plain(w, fmt, gw if g else 1.0)
    a = q.abs()
    code = ((a >= 0.5).byte() + (a >= 1).byte() + (a >= 1.5).byte() + (a >= 2).byte() + (a >= 3).byte()
            + (a >= 4).byte() + (a >= 6).byte()) | (torch.signbit(q).byte() << 3)
    s8 = s.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "nv" else (torch.frexp(s)[1] + 126).byte()
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), _tile(s8), gw


def _activations(M, K, gen):
    """N(0, 1) rows with a few channels that are twenty times larger, as hidden states have them."""
    x = torch.randn((M, K), generator=gen, device=DEV)
    x[:, torch.randint(0, K, (max(1, K // 512),), generator=gen, device=DEV)] *= 20.0
    return x.to(torch.bfloat16)


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    st = {"c": c}
    if c["op"] in ("quant", "linear"):
        M, K, fmt = c["M"], c["K"], c["fmt"]
        st["x"] = _activations(M, K, gen)
        st["gx"] = torch.full((1,), 117.5 / 2688.0, device=DEV) if c["g"] else None   # calibrated ahead
        if c["op"] == "quant":
            nb = K // BLOCK[fmt]
            st["q"] = torch.empty((M, K // 2), dtype=torch.uint8, device=DEV)
            st["s"] = torch.empty((-(-M // 128), -(-nb // 4), 512), dtype=torch.uint8, device=DEV)
            st["y"] = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
        else:
            N = c["N"]
            st["Wq"], st["sw"], st["gw"] = _weights(N, K, fmt, c["g"], gen)
            st["y"] = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
            if own:                                                # a serving loop keeps its workspace
                import gemv_dg_bf16_gb300 as dg
                st["ws"] = dg.workspace(dg.DG_OP_GEMV_A4W4, M, N, K)
    elif c["op"] == "route":
        M, E = c["M"], c["E"]
        x = 1.5 * torch.randn((M, E), generator=gen, device=DEV)
        if c["masked"]:                                            # experts that are not available now
            x[:, torch.rand((E,), generator=gen, device=DEV) < 0.1] = -math.inf
        st["logits"] = x.to(torch.bfloat16) if c["bits"] == 16 else x
        std = 0.1 if c["score"] == "sigmoid" else 0.2 / E
        st["bias"] = std * torch.randn((E,), generator=gen, device=DEV) if c["bias"] else None
        st["ids"] = torch.empty((M, c["topk"]), dtype=torch.int32, device=DEV)
        st["w"] = torch.empty((M, c["topk"]), dtype=torch.float32, device=DEV)
    else:
        M, V, n = c["M"], c["V"], c["top"]
        x = torch.randn((M, V), generator=gen, device=DEV, dtype=torch.bfloat16 if c["bits"] == 16 else torch.float32)
        x.mul_(2.5)
        if c["masked"]:                                            # a grammar that allows half of the vocabulary
            x.masked_fill_(torch.rand((V,), generator=gen, device=DEV) < 0.5, -math.inf)
        st["logits"] = x
        st["tokens"] = torch.randint(0, V, (M,), generator=gen, device=DEV, dtype=torch.int64)
        near = x.argmax(-1)                                        # every other row's token is its likeliest
        st["tokens"][::2] = near[::2]
        st["out"] = {"logprob": torch.empty((M,), device=DEV), "rank": torch.empty((M,), dtype=torch.int32, device=DEV),
                     "entropy": torch.empty((M,), device=DEV),
                     "top_ids": torch.empty((M, n), dtype=torch.int32, device=DEV) if n else None,
                     "top_logprobs": torch.empty((M, n), device=DEV) if n else None}
    return st


# ------------------------------------------------------------------------------- one pass

def run(st):
    c = st["c"]
    if own:
        return _run_own(st, c)
    return {"quant": _plain_quant, "linear": _plain_linear, "route": _plain_route, "logprobs": _plain_logprobs}[
        c["op"]](st, c)


def _run_own(st, c):
    import gemv_dg_bf16_gb300 as dg
    if c["op"] in ("quant", "linear"):
        fmt = dg.DG_FP4_MX if c["fmt"] == "mx" else dg.DG_FP4_NV
        if c["op"] == "quant":
            q, s = dg.dg_quant_fp4_blockscale(st["x"], fmt, g=st["gx"], q=st["q"], s=st["s"])
            return {"values": dg.dg_dequant_fp4_blockscale(q, s, fmt, g=st["gx"], y=st["y"])}
        return {"y": dg.dg_gemv_a4w4_blockscale(st["x"], st["Wq"], st["sw"], fmt, gx=st["gx"], gw=st["gw"], y=st["y"],
                                                ws=st["ws"])}
    if c["op"] == "route":
        ids, w = dg.dg_moe_route(st["logits"], c["topk"],
                                 score=dg.DG_SCORE_SIGMOID if c["score"] == "sigmoid" else dg.DG_SCORE_SOFTMAX,
                                 bias=st["bias"], n_group=c["n_group"], topk_group=c["topk_group"],
                                 group_top=c["group_top"], renorm=c["renorm"], scale=c["scale"], ids=st["ids"],
                                 w=st["w"])
        return {"ids": ids, "w": w}
    r = dg.dg_logprobs(st["logits"], st["tokens"], n_top=c["top"], scale=c["scale"], **st["out"])
    return {k: v for k, v in r.items() if v is not None}


def _plain_quant(st, c):
    g = st["gx"] if c["g"] else 1.0
    q, s = _quant_plain(st["x"].float(), c["fmt"], g)
    return {"values": (q.view(*s.shape, -1) * (s * g).unsqueeze(-1)).view(q.shape).to(torch.bfloat16)}


def _plain_linear(st, c):
    N, K, b = c["N"], c["K"], BLOCK[c["fmt"]]
    q, s = _quant_plain(st["x"].float(), c["fmt"], st["gx"] if c["g"] else 1.0)
    x = (q.view(*s.shape, b) * s.unsqueeze(-1)).view(q.shape)
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    codes = torch.stack((st["Wq"] & 15, st["Wq"] >> 4), -1).view(N, K)
    s8 = _untile(st["sw"], N, K // b).contiguous()
    sw = s8.view(torch.float8_e4m3fn).float() if c["fmt"] == "nv" else _pow2(s8.int() - 127)
    w = (grid[codes.int()].view(N, -1, b) * sw.unsqueeze(-1)).view(N, K)
    y = x @ w.t()
    if c["g"]:
        y = y * (st["gx"] * st["gw"])
    return {"y": y.to(torch.bfloat16)}


def _plain_route(st, c):
    x = st["logits"].float()
    M, E = x.shape
    can = x > -math.inf
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-x))
    else:
        m = x.amax(-1, keepdim=True)
        e = torch.where(x == m, torch.ones_like(x), torch.exp(x - m))
        # The pick compares sums of p and the bias, so the normaliser is the rounded sum of all terms, whatever
        # their order: a sum that depends on the order would pick by it.
        p = e / torch.where(can, e, torch.zeros_like(e)).sum(-1, keepdim=True, dtype=torch.float64).float()
    none = torch.full_like(p, -math.inf)
    key = torch.where(can, p + st["bias"] if c["bias"] else p, none)
    G = c["n_group"]
    if G > 1:
        kg = key.view(M, G, E // G)
        best = kg.sort(-1, descending=True).values[..., :2]
        gs = best[..., 0]
        if c["group_top"] == 2:
            gs = gs + torch.where(best[..., 1] > -math.inf, best[..., 1], torch.zeros_like(gs))
        order = gs.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros((M, G), dtype=torch.bool, device=x.device).scatter_(1, order, True)
        key = torch.where(keep.unsqueeze(-1), kg, none.view(M, G, E // G)).reshape(M, E)
    k, ids = key.sort(dim=-1, descending=True, stable=True)
    k, ids = k[:, :c["topk"]], ids[:, :c["topk"]]
    found = k > -math.inf
    w = torch.where(found, p.gather(1, ids), torch.zeros_like(k))
    if c["renorm"]:
        t = w.sum(-1, keepdim=True)
        w = torch.where(t > 0, w / t, torch.zeros_like(w))
    return {"ids": torch.where(found, ids, torch.full_like(ids, -1)).int(), "w": w * c["scale"]}


def _plain_logprobs(st, c):
    x, tok = st["logits"].float(), st["tokens"]
    z = x * c["scale"]
    m = z.amax(-1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    s = e.sum(-1)
    ls = torch.log(s)
    xt = x.gather(1, tok.unsqueeze(1))
    out = {"logprob": d.gather(1, tok.unsqueeze(1)).squeeze(1) - ls,
           "rank": (x > xt).sum(-1).int(),
           "entropy": ls - torch.where(e > 0, e * d, torch.zeros_like(e)).sum(-1) / s}
    if c["top"]:
        # Equal logits go by the lower index: one whole number orders both.
        bits = x.view(torch.int32)
        up = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        key = (up << 32) - torch.arange(x.shape[1], device=x.device)
        ids = key.topk(c["top"], -1).indices
        out["top_ids"] = ids.int()
        out["top_logprobs"] = d.gather(1, ids) - ls.unsqueeze(1)
    return out


# ------------------------------------------------------------------------------- in 64 bits

def _exp2(e):
    """2^e in 64 bits of whole numbers -1022 <= e <= 1023."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _floor_log2(v):
    """floor(log2(v)) of v > 0 (0 gives -1)."""
    return torch.frexp(v)[1] - 1


def _round_float(v, mantissa, least, most):
    """v to the nearest number of `mantissa` fraction bits and exponents from `least` up, ties to even, at most `most`."""
    step = _exp2(_floor_log2(v.abs()).clamp(min=least) - mantissa)
    return (torch.round(v / step) * step).clamp(-most, most)


def _exact_quant(x, fmt, g):
    """The quantised values without the tensor scale, and the block scales, from the formats' definitions."""
    b = BLOCK[fmt]
    x = x.double().reshape(x.shape[0], -1, b)
    top = x.abs().max(-1, keepdim=True).values
    if fmt == "mx":
        s = _exp2(torch.where(top > 0, _floor_log2(top) - 2, -127).clamp(-127, 127))
        return _round_float(x / s, 1, 0, 6.0), s
    s = _round_float(top / 6.0 / g, 3, -6, 448.0)
    return torch.where(s > 0, _round_float(x / (s * g).clamp(min=1e-300), 1, 0, 6.0), torch.zeros_like(x)), s


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] in ("quant", "linear"):
        g = st["gx"].double() if c["g"] else 1.0
        q, s = _exact_quant(st["x"], c["fmt"], g)
        if c["op"] == "quant":
            return {"values": (q * s * g).reshape(st["x"].shape)}
        N, K, b = c["N"], c["K"], BLOCK[c["fmt"]]
        nib = torch.empty((N, K), dtype=torch.uint8, device=DEV)
        nib[:, ::2], nib[:, 1::2] = st["Wq"] % 16, st["Wq"] // 16
        mag, sign = nib % 8, 1.0 - 2.0 * (nib // 8).double()
        ex, fr = (mag // 2).int(), (mag % 2).double()
        val = sign * torch.where(ex > 0, _exp2(ex - 1) * (1 + fr / 2), fr / 2)
        n, k = torch.arange(N, device=DEV).unsqueeze(1), torch.arange(K // b, device=DEV).unsqueeze(0)
        raw = st["sw"][n // 128, k // 4, (n % 32) * 16 + (n % 128) // 32 * 4 + k % 4].int()
        if c["fmt"] == "nv":
            f, m = raw // 8, (raw % 8).double()
            sw = torch.where(f > 0, _exp2(f - 7) * (1 + m / 8), m * 2.0 ** -9)
        else:
            sw = _exp2(raw - 127)
        y = (q * s).reshape(st["x"].shape) @ (val.view(N, -1, b) * sw.unsqueeze(-1)).view(N, K).t()
        return {"y": y * (g * st["gw"].double() if c["g"] else 1.0)}
    if c["op"] == "route":
        x = st["logits"].double()
        M, E = x.shape
        p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1)
        key = p + st["bias"].double() if c["bias"] else p.clone()
        key[x == -math.inf] = -math.inf
        G = c["n_group"]
        if G > 1:
            per = key.reshape(M, G, -1)
            best = per.topk(c["group_top"], -1).values
            best[..., 1:] = best[..., 1:].masked_fill(best[..., 1:] == -math.inf, 0.0)
            cut = best.sum(-1).argsort(dim=-1, descending=True, stable=True).argsort(dim=-1) >= c["topk_group"]
            key = per.masked_fill(cut.unsqueeze(-1), -math.inf).reshape(M, E)
        k, ids = torch.sort(key, dim=-1, descending=True, stable=True)
        w = p.gather(1, ids)[:, :c["topk"]].masked_fill(k[:, :c["topk"]] == -math.inf, 0.0)
        if c["renorm"]:
            w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
        return {"ids": None, "w": w * c["scale"]}
    z = st["logits"].double() * c["scale"]
    lp = z - torch.logsumexp(z, -1, keepdim=True)
    del z
    out = {"logprob": lp.gather(1, st["tokens"].unsqueeze(1)).squeeze(1), "rank": None,
           "entropy": -(torch.exp(lp) * lp.clamp(min=-1e300)).sum(-1)}
    if c["top"]:
        out["top_ids"] = None
        out["top_logprobs"] = lp.topk(c["top"], -1).values
    return out
