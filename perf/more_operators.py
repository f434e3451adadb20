"""More operators around a decode step, as they are measured: the 8-bit integer quantisation and
linear with a scale for each token and each channel, tokens sorted by expert and back (with the
gradients), and the penalties, biases and masks on logits before a token is drawn.

listed() names the cases, draw() gives more of the same ranges, prepare() makes what a program has
in hand, run() makes one pass -- with elementary torch operations where `own` is false, through
this library's entry points where it is true -- work() counts what a pass cannot do without, and
exact() restates each operator in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # 16 token rows entering an integer linear: one small launch, latency counts.
        {"name": "quantise 16 rows", "op": "quant", "M": 16, "K": 4096},
        # A gate/up weight matrix converted, row by row, when a model is loaded: pure bandwidth.
        {"name": "quantise weights", "op": "quant", "M": 24576, "K": 4096},
        # One decoding sequence through a square projection: the smallest weight stream.
        {"name": "linear 1 row", "op": "linear", "M": 1, "N": 4096, "K": 4096},
        # A small decode batch through a wide projection.
        {"name": "linear 16 rows", "op": "linear", "M": 16, "N": 12288, "K": 4096},
        # A ragged batch and ragged weight rows with a long reduction (a down projection).
        {"name": "linear 77 rows ragged", "op": "linear", "M": 77, "N": 4099, "K": 12288},
        # The largest batch of the linear (a chunk of a prompt) through gate/up rows.
        {"name": "linear 512 rows", "op": "linear", "M": 512, "N": 24576, "K": 4096},
        # A decode batch past the small-batch expert kernels, sorted and gathered: latency counts.
        {"name": "dispatch 64 tokens", "op": "dispatch", "M": 64, "E": 128, "topk": 6, "K": 4096, "absent": 0.1, "grad": False},
        # A long prompt's tokens sorted by expert, with the gradient that comes back to them.
        {"name": "dispatch 32768 tokens", "op": "dispatch", "M": 32768, "E": 256, "topk": 8, "K": 4096, "absent": 0.0, "grad": True},
        # The same small batch on its way back from the experts.
        {"name": "combine 64 tokens", "op": "combine", "M": 64, "E": 128, "topk": 6, "K": 4096, "absent": 0.1, "grad": False},
        # A training step's tokens weighted and added, and the gradients of the rows and of the weights.
        {"name": "combine 8192 tokens", "op": "combine", "M": 8192, "E": 256, "topk": 8, "K": 4096, "absent": 0.0, "grad": True},
        # One sequence before it draws a token: a long history, a few biases and a grammar's mask.
        {"name": "logits 1 row", "op": "logits", "M": 1, "V": 248320, "L": 2000, "B": 16, "bits": 16, "mask": True},
        # A large decode batch, histories of all lengths, rows whose grammar allows nothing among them.
        {"name": "logits 256 rows", "op": "logits", "M": 256, "V": 248320, "L": 4096, "B": 64, "bits": 16, "mask": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "dispatch", "combine", "logits"])
    if op == "quant":
        K = 16 * _log_int(rng, 1, 1024)
        return {"op": op, "M": _log_int(rng, 1, min(24576, 24576 * 4096 // K)), "K": K}
    if op == "linear":
        K = 16 * _log_int(rng, 4, 1024)
        N = _log_int(rng, 16, 24576)
        return {"op": op, "M": _log_int(rng, 1, max(1, min(512, 512 * 24576 * 4096 // (N * K)))), "N": N, "K": K}
    if op in ("dispatch", "combine"):
        E = _log_int(rng, 2, 1024)
        topk = rng.randint(1, min(16, E))
        K = 8 * _log_int(rng, 4, 1024)
        most = (32768 if op == "dispatch" else 8192) * 8 * 4096 // (topk * K)
        return {"op": op, "M": _log_int(rng, 1, min(32768, most)), "E": E, "topk": topk, "K": K,
                "absent": rng.choice([0.0, 0.0, 0.1, 0.9]), "grad": rng.random() < 0.5}
    V = _log_int(rng, 500, 248320)
    bits = rng.choice([16, 32])
    M = _log_int(rng, 1, min(1024, 256 * 248320 * 16 // (V * bits)))
    return {"op": op, "M": M, "V": V, "L": rng.choice([0, _log_int(rng, 1, max(2, min(32768, 256 * 4096 // M)))]),
            "B": rng.choice([0, _log_int(rng, 1, 256)]), "bits": bits, "mask": rng.random() < 0.6}


def work(c):
    M = c["M"]
    if c["op"] == "quant":
        return {"bytes": 3 * M * c["K"] + 4 * M, "flops": 3 * M * c["K"]}
    if c["op"] == "linear":
        N, K = c["N"], c["K"]
        return {"bytes": N * K + 4 * N + 2 * M * K + 2 * M * N, "flops": 2 * M * N * K}
    if c["op"] in ("dispatch", "combine"):
        row, rows = 2 * c["K"], int(M * c["topk"] * (1 - c["absent"]))
        if c["op"] == "dispatch":                                      # ids in; positions and slots out; rows
            moved = (M + rows) * row * (2 if c["grad"] else 1)
            return {"bytes": moved + 12 * M * c["topk"] + 4 * c["E"], "flops": rows * c["K"] if c["grad"] else 0}
        moved = (rows + M) * row + (rows + M) * row * c["grad"]        # rows read once for both directions
        return {"bytes": moved + M * c["topk"] * (12 if c["grad"] else 8),
                "flops": rows * c["K"] * (5 if c["grad"] else 2)}
    V = c["V"]
    return {"bytes": 2 * M * V * c["bits"] // 8 + (M * V // 8 if c["mask"] else 0) + M * (2 * c["L"] + 8 * c["B"] + 20),
            "flops": M * V}


# ------------------------------------------------------------------------------- inputs

def _activations(M, K, gen):
    """N(0, 1) rows with a few channels that are twenty times larger, as hidden states have them."""
    x = torch.randn((M, K), generator=gen, device=DEV)
    x[:, torch.randint(0, K, (max(1, K // 512),), generator=gen, device=DEV)] *= 20.0
    return x.to(torch.bfloat16)


def _experts(c, gen):
    """Distinct experts for each token, some much more popular than others; ids of -1 where a slot is absent."""
    M, E, topk = c["M"], c["E"], c["topk"]
    liking = torch.randn((E,), generator=gen, device=DEV)
    u = torch.rand((M, E), generator=gen, device=DEV).clamp_(1e-6, 1 - 1e-6)
    ids = (liking - torch.log(-torch.log(u))).topk(topk, -1).indices.int()
    if c["absent"]:
        ids[torch.rand((M, topk), generator=gen, device=DEV) < c["absent"]] = -1
    return ids


def _positions(ids, E):
    """(rows before each expert [E + 1], row of each slot [M, topk] or -1, slot of each row, -1 past the last)."""
    flat = torch.where(ids >= 0, ids, torch.full_like(ids, E)).reshape(-1).long()
    order = flat.sort(stable=True).indices
    counts = torch.zeros((E + 1,), dtype=torch.int64, device=DEV).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat((counts.new_zeros(1), counts[:E].cumsum(0)))
    rows = torch.arange(flat.numel(), device=DEV)
    live = rows < offsets[E]
    pos = torch.empty_like(flat).scatter_(0, order, torch.where(live, rows, torch.full_like(rows, -1)))
    return offsets.int(), pos.int().view(ids.shape), torch.where(live, order, torch.full_like(order, -1)).int()


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    st = {"c": c}
    M = c["M"]
    bf = {"dtype": torch.bfloat16, "device": DEV}
    if c["op"] == "quant":
        st["x"] = _activations(M, c["K"], gen)
        st["q"] = torch.empty((M, c["K"]), dtype=torch.int8, device=DEV)
        st["s"] = torch.empty((M,), device=DEV)
    elif c["op"] == "linear":
        N, K = c["N"], c["K"]
        st["x"] = _activations(M, K, gen)
        w = torch.randn((N, K), generator=gen, device=DEV) * K ** -0.5
        st["sw"] = w.abs().amax(-1) / 127.0                            # as a checkpoint holds them
        st["Wq"] = torch.round(w / st["sw"].unsqueeze(1)).to(torch.int8)
        st["y"] = torch.empty((M, N), **bf)
        if own:                                                        # a serving loop keeps its workspace
            import gemv_dg_bf16_gb300 as dg
            st["ws"] = dg.workspace(dg.DG_OP_GEMV_I8, M, N, K)
    elif c["op"] in ("dispatch", "combine"):
        E, topk, K = c["E"], c["topk"], c["K"]
        P = M * topk
        st["ids"] = _experts(c, gen)
        if c["op"] == "dispatch":
            st["x"] = _activations(M, K, gen)
            st["offsets"] = torch.empty((E + 1,), dtype=torch.int32, device=DEV)
            st["pos"] = torch.empty((M, topk), dtype=torch.int32, device=DEV)
            st["slots"] = torch.empty((P,), dtype=torch.int32, device=DEV)
            st["xs"] = torch.zeros((P, K), **bf)                       # rows behind the last stay as they are
            if c["grad"]:
                st["dxs"] = torch.randn((P, K), generator=gen, **bf)
                st["dx"] = torch.empty((M, K), **bf)
        else:
            st["offsets"], st["pos"], st["slots"] = _positions(st["ids"], E)
            st["z"] = torch.randn((P, K), generator=gen, **bf)
            st["w"] = torch.softmax(torch.randn((M, topk), generator=gen, device=DEV), -1)
            st["y"] = torch.empty((M, K), **bf)
            if c["grad"]:
                st["dy"] = torch.randn((M, K), generator=gen, **bf)
                st["dz"] = torch.zeros((P, K), **bf)
                st["dw"] = torch.empty((M, topk), device=DEV)
    else:
        V, L, B = c["V"], c["L"], c["B"]
        x = torch.randn((M, V), generator=gen, device=DEV, dtype=torch.bfloat16 if c["bits"] == 16 else torch.float32)
        st["logits"] = x.mul_(2.5)
        st["out"] = torch.empty_like(x)
        u = lambda *s: torch.rand(s, generator=gen, device=DEV)
        if L:                                                          # a few tokens make up much of a text
            st["tokens"] = (u(M, L) ** 6 * V).int().clamp_(max=V - 1)
            st["lengths"] = (u(M) * (L + 1)).int().clamp_(max=L)
            st["lengths"][0] = L
            st["prompt_lengths"] = (u(M) * st["lengths"]).int()
            off = u(M) < 0.2                                           # requests that ask for no penalty
            st["repetition"] = torch.where(off, torch.ones_like(u(M)), 0.8 + 0.7 * u(M))
            st["frequency"] = torch.where(off, torch.zeros_like(u(M)), u(M) - 0.2)
            st["presence"] = torch.where(off, torch.zeros_like(u(M)), u(M) - 0.2)
        if B:
            ids = (u(M, B) * V).int().clamp_(max=V - 1)
            st["bias_ids"] = torch.where(u(M, B) < 0.3, torch.full_like(ids, -1), ids)
            st["bias"] = 8.0 * u(M, B) - 4.0
        if c["mask"]:                                                  # a grammar: nothing, little, half or all allowed
            words = (V + 31) // 32
            keep = torch.tensor([0.5, 0.001, 1.0, 0.5, 0.0], device=DEV)[torch.arange(M, device=DEV) % 5]
            st["mask"] = torch.empty((M, words), dtype=torch.int32, device=DEV)
            step = max(1, (1 << 24) // (32 * words))
            bit = 1 << torch.arange(32, dtype=torch.int64, device=DEV)
            for m in range(0, M, step):
                k = keep[m:m + step, None, None]
                bits = (u(k.shape[0], words, 32) < k).long()
                v = (bits * bit).sum(-1)
                st["mask"][m:m + step] = torch.where(v >= 1 << 31, v - (1 << 32), v).int()
    return st


# ------------------------------------------------------------------------------- one pass

def run(st):
    c = st["c"]
    if own:
        return _run_own(st, c)
    return {"quant": _plain_quant, "linear": _plain_linear, "dispatch": _plain_dispatch, "combine": _plain_combine,
            "logits": _plain_logits}[c["op"]](st, c)


def _run_own(st, c):
    import gemv_dg_bf16_gb300 as dg
    if c["op"] == "quant":
        q, s = dg.dg_quant_i8_rowscale(st["x"], q=st["q"], s=st["s"])
        return {"q": q, "s": s}
    if c["op"] == "linear":
        return {"y": dg.dg_gemv_i8_rowscale(st["x"], st["Wq"], st["sw"], y=st["y"], ws=st["ws"])}
    if c["op"] == "dispatch":
        offsets, pos, slots = dg.dg_moe_sort(st["ids"], c["E"], offsets=st["offsets"], pos=st["pos"], slots=st["slots"])
        out = {"offsets": offsets, "pos": pos, "slots": slots, "xs": dg.dg_moe_gather(st["x"], pos, xs=st["xs"])}
        if c["grad"]:
            out["dx"] = dg.dg_moe_combine(st["dxs"], pos, y=st["dx"])
        return out
    if c["op"] == "combine":
        out = {"y": dg.dg_moe_combine(st["z"], st["pos"], st["w"], y=st["y"])}
        if c["grad"]:
            out["dz"], out["dw"] = dg.dg_moe_combine_grad(st["dy"], st["z"], st["pos"], st["w"], dz=st["dz"], dw=st["dw"])
        return out
    names = ("tokens", "lengths", "prompt_lengths", "repetition", "frequency", "presence", "bias_ids", "bias", "mask", "out")
    return {"logits": dg.dg_logits_adjust(st["logits"], **{k: st[k] for k in names if k in st})}


def _codes(x):
    """(whole numbers -127..127 as fp32, scales) of fp32 rows."""
    amax = x.abs().amax(-1).clamp(min=2.0 ** -100)
    return torch.round(x * (127.0 / amax).unsqueeze(1)).clamp(-127, 127), amax / 127.0


def _plain_quant(st, c):
    q, s = _codes(st["x"].float())
    return {"q": q.to(torch.int8), "s": s}


def _plain_linear(st, c):
    q, s = _codes(st["x"].float())
    return {"y": ((q @ st["Wq"].float().t()) * (s.unsqueeze(1) * st["sw"])).to(torch.bfloat16)}


def _take(rows, pos):
    """rows[pos], zeros where pos is -1."""
    got = rows[pos.clamp(min=0).long()]
    return torch.where((pos >= 0).unsqueeze(-1), got, torch.zeros_like(got))


def _plain_dispatch(st, c):
    offsets, pos, slots = _positions(st["ids"], c["E"])
    token = torch.where(slots >= 0, slots // c["topk"], slots)
    out = {"offsets": offsets, "pos": pos, "slots": slots, "xs": _take(st["x"], token)}
    if c["grad"]:
        out["dx"] = _take(st["dxs"], pos).float().sum(1).to(torch.bfloat16)
    return out


def _plain_combine(st, c):
    pos, w = st["pos"], st["w"]
    z = _take(st["z"], pos).float()
    out = {"y": (w.unsqueeze(-1) * z).sum(1).to(torch.bfloat16)}
    if c["grad"]:
        dy, slots = st["dy"].float(), st["slots"]
        at = slots.clamp(min=0).long()
        dz = w.reshape(-1)[at].unsqueeze(1) * dy[at // c["topk"]]
        out["dz"] = torch.where((slots >= 0).unsqueeze(1), dz, torch.zeros_like(dz)).to(torch.bfloat16)
        out["dw"] = (dy.unsqueeze(1) * z).sum(-1)
    return out


def _plain_logits(st, c):
    x = st["logits"].float()
    M, V = x.shape
    if c["L"]:
        tok = st["tokens"].long()
        at = torch.arange(c["L"], device=DEV).unsqueeze(0)
        here = at < st["lengths"].unsqueeze(1)
        made = here & (at >= st["prompt_lengths"].unsqueeze(1))
        count = torch.zeros_like(x).scatter_add_(1, tok, made.float())
        seen = torch.zeros_like(x).scatter_add_(1, tok, here.float()) > 0
        r = st["repetition"].unsqueeze(1)
        x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
        x = x - st["frequency"].unsqueeze(1) * count
        x = x - torch.where(count > 0, st["presence"].unsqueeze(1), torch.zeros_like(x))
    if c["B"]:
        use = st["bias_ids"] >= 0
        add = torch.zeros((M, V), dtype=torch.float64, device=DEV)
        add.scatter_add_(1, st["bias_ids"].clamp(min=0).long(), torch.where(use, st["bias"], torch.zeros_like(st["bias"])).double())
        x = x + add.float()
    if c["mask"]:
        v = torch.arange(V, device=DEV)
        allowed = (st["mask"][:, v // 32] >> (v % 32).int()) & 1
        x = torch.where(allowed == 1, x, torch.full_like(x, -math.inf))
    return {"logits": x.to(st["logits"].dtype)}


# ------------------------------------------------------------------------------- in 64 bits

def _exact_codes(x):
    x = x.double()
    s = x.abs().max(1, keepdim=True).values.clamp(min=2.0 ** -100) / 127.0
    return torch.round(x / s), s


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "quant":
        return {"q": None, "s": _exact_codes(st["x"])[1].squeeze(1)}
    if c["op"] == "linear":
        q, s = _exact_codes(st["x"])
        return {"y": (q * s) @ (st["Wq"].double() * st["sw"].double().unsqueeze(1)).t()}
    if c["op"] in ("dispatch", "combine"):
        M, topk, K = c["M"], c["topk"], c["K"]
        flat = st["ids"].reshape(-1).cpu()
        live = torch.nonzero(flat >= 0).squeeze(1)
        order = live[flat[live].argsort(stable=True)].to(DEV)          # slot of each row
        n = order.numel()
        step = max(1, (1 << 28) // K)
        if c["op"] == "dispatch":
            xs = torch.zeros((M * topk, K), dtype=torch.bfloat16, device=DEV)      # (a copy has its own type's values)
            xs[:n] = st["x"][order // topk]
            out = {"offsets": None, "pos": None, "slots": None, "xs": xs.double() if xs.numel() < 1 << 28 else None}
            if c["grad"]:
                dx = torch.zeros((M, K), dtype=torch.float64, device=DEV)
                for i in range(0, n, step):
                    dx.index_add_(0, order[i:i + step] // topk, st["dxs"][:n][i:i + step].double())
                out["dx"] = dx
            return out
        y = torch.zeros((M, K), dtype=torch.float64, device=DEV)
        dz = torch.zeros((M * topk, K), dtype=torch.float64, device=DEV) if c["grad"] else None
        dw = torch.zeros((M * topk,), dtype=torch.float64, device=DEV) if c["grad"] else None
        for i in range(0, n, step):
            o = order[i:i + step]
            z, w = st["z"][:n][i:i + step].double(), st["w"].double().reshape(-1)[o].unsqueeze(1)
            y.index_add_(0, o // topk, w * z)
            if c["grad"]:
                dy = st["dy"].double()[o // topk]
                dz[i:i + o.numel()] = w * dy
                dw[o] = (dy * z).sum(1)
        return {"y": y, "dz": dz, "dw": dw.view(M, topk)} if c["grad"] else {"y": y}
    x = st["logits"].double()
    M, V = x.shape
    for m in range(M):
        row = x[m]
        if c["L"]:
            n, p = int(st["lengths"][m]), int(st["prompt_lengths"][m])
            r, f, q = (float(st[k][m]) for k in ("repetition", "frequency", "presence"))
            ids = st["tokens"][m, :n].long()
            seen = torch.unique(ids)
            row[seen] = torch.where(row[seen] > 0, row[seen] / r, row[seen] * r)
            made, times = torch.unique(ids[p:], return_counts=True)
            row[made] -= f * times.double() + q
        if c["B"]:
            use = st["bias_ids"][m] >= 0
            row.index_add_(0, st["bias_ids"][m][use].long(), st["bias"][m][use].double())
        if c["mask"]:
            words = st["mask"][m].long() & 0xFFFFFFFF
            bits = (words.unsqueeze(1) >> torch.arange(32, device=DEV)) & 1
            row[bits.reshape(-1)[:V] == 0] = -math.inf
    return {"logits": x}
