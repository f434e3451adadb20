"""Plain references of the 8-bit integer linear, the sort by expert and the edits of logits: whole
numbers exactly, sums in 64 bits, and each binary32 step that a definition names as one numpy operation."""
import numpy as np
import torch

F32 = np.float32


def f32(t):
    return t.detach().float().cpu().numpy()


def bf16_of(a):
    """fp32 array -> bf16 patterns (torch's cast, round to nearest even)."""
    return torch.from_numpy(np.ascontiguousarray(a, F32)).to(torch.bfloat16).view(torch.int16).numpy()


def i8_codes(x):
    """(codes int8, scales fp32) of fp32 rows; a row with a NaN or an infinity: codes 0, scale NaN."""
    with np.errstate(invalid="ignore", over="ignore"):
        amax = np.abs(x).max(1)
        bad = ~np.isfinite(amax)
        A = np.maximum(np.where(bad, F32(1), amax), F32(2.0 ** -100)).astype(F32)
        r = F32(127.0) * (F32(1.0) / A)
        q = np.rint(np.where(bad[:, None], F32(0), x).astype(F32) * r[:, None])
    return q.astype(np.int8), np.where(bad, F32(np.nan), A * (F32(1.0) / F32(127.0))).astype(F32)


def i8_linear(x, Wq, sw):
    """bf16 patterns of y, from fp32 x, int8 weights and fp32 scales."""
    q, sx = i8_codes(x)
    # (products below 2^53 in all: a float64 matrix product is exact)
    acc = (q.astype(np.float64) @ Wq.astype(np.float64).T).astype(np.int64)
    assert np.abs(acc).max(initial=0) < 2 ** 31
    with np.errstate(over="ignore", under="ignore"):
        return bf16_of(acc.astype(np.int32).astype(F32) * (sx[:, None] * sw[None, :]))


def moe_sort(ids, E):
    M, topk = ids.shape
    rows = []
    for m in range(M):
        for k in range(topk):
            e = int(ids[m, k])
            if 0 <= e < E and e not in ids[m, :k]:
                rows.append((e, m * topk + k))
    rows.sort()
    offsets = np.zeros(E + 1, np.int32)
    pos = np.full(M * topk, -1, np.int32)
    slots = np.full(M * topk, -1, np.int32)
    for p, (e, i) in enumerate(rows):
        offsets[e + 1:] += 1
        pos[i] = p
        slots[p] = i
    return offsets, pos.reshape(M, topk), slots


def adjust(x, tokens=None, lengths=None, prompt_lengths=None, repetition=None, frequency=None, presence=None,
           bias_ids=None, bias=None, mask=None):
    """fp32 logits after every edit, one rounded step at a time."""
    x = x.astype(F32).copy()
    M, V = x.shape
    touched = np.zeros((M, V), bool)
    with np.errstate(all="ignore"):
        for m in range(M):
            if tokens is not None:
                L = tokens.shape[1]
                n = L if lengths is None else min(max(int(lengths[m]), 0), L)
                p = 0 if prompt_lengths is None else min(max(int(prompt_lengths[m]), 0), n)
                count, prompt = {}, set()
                for i in range(n):
                    v = int(tokens[m, i])
                    if 0 <= v < V:
                        if i < p:
                            prompt.add(v)
                        else:
                            count[v] = count.get(v, 0) + 1
                for v in prompt | set(count):
                    if repetition is not None:
                        r = F32(repetition[m])
                        x[m, v] = x[m, v] / r if x[m, v] > 0 else x[m, v] * r
                    if v in count:
                        if frequency is not None:
                            x[m, v] = x[m, v] - F32(frequency[m]) * F32(count[v])
                        if presence is not None:
                            x[m, v] = x[m, v] - F32(presence[m])
            if bias_ids is not None:
                add = {}
                for v, b in zip(bias_ids[m].tolist(), bias[m]):
                    if 0 <= v < V:
                        add[v] = add[v] + F32(b) if v in add else F32(b)
                for v, b in add.items():
                    x[m, v] = x[m, v] + b
            if mask is not None:
                bits = (mask[m].view(np.uint32)[np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1
                x[m, bits == 0] = -np.inf
    return x
