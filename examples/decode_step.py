"""One decode step of a routed-expert model on this library's entry points: a 4-bit projection,
the router, the experts, the fp8 head, and the picked token with its log-probability.

  python examples/decode_step.py [--rows 4] [--hidden 4096] [--vocab 248320]

Weights are random and the step has one layer; what it shows is how the calls fit together:
every buffer is made once, the step is captured in a CUDA graph and replayed.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemv_dg_bf16_gb300 as dg  # noqa: E402


def fp8_rows(w):
    """fp32 [..., n, k] -> (e4m3 codes, one fp32 scale per row)."""
    s = w.abs().amax(-1) / 448.0
    return (w / s.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8), s


class Step:
    def __init__(self, rows, hidden, vocab, experts=32, inter=512, topk=6, n_top=5, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5
        M, H = rows, hidden
        self.M, self.topk, self.n_top = M, topk, n_top
        # 4-bit projection: NV blocks under one tensor scale per side (the activations' calibrated ahead)
        w = rand(H, H).to(torch.bfloat16)
        self.gw = (w.float().abs().amax() / 2688.0).reshape(1)
        self.gx = torch.full((1,), 5.0 / 2688.0, device="cuda")
        self.Wq, self.sw = dg.dg_quant_fp4_blockscale(w, dg.DG_FP4_NV, g=self.gw)
        self.Wr = rand(experts, H).to(torch.bfloat16)
        self.bias = 0.01 * torch.randn((experts,), generator=g, device="cuda")
        self.W1, self.s1 = fp8_rows(rand(experts, 2 * inter, H))
        self.W2, self.s2 = fp8_rows(rand(experts, H, inter))
        head = rand(vocab, H)
        self.head_scale = (head.abs().amax() / 448.0).reshape(1)
        self.head = (head / self.head_scale).to(torch.float8_e4m3fn).view(torch.uint8)
        del head
        self.ws = {name: dg.workspace(op, M, n, k, t) for name, op, n, k, t in (
            ("proj", dg.DG_OP_GEMV_A4W4, H, H, 0), ("router", dg.DG_OP_GEMV_BF16, experts, H, 0),
            ("w1", dg.DG_OP_MOE_W1, inter, H, topk), ("w2", dg.DG_OP_MOE_W2, H, inter, topk),
            ("head", dg.DG_OP_HEAD_FP8_ARGMAX, vocab, H, 0))}
        self.x = torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16)
        self.token = torch.zeros((M,), dtype=torch.int64, device="cuda")

    def __call__(self):
        ws = self.ws
        h = dg.dg_gemv_a4w4_blockscale(self.x, self.Wq, self.sw, dg.DG_FP4_NV, gx=self.gx, gw=self.gw, ws=ws["proj"])
        scores = dg.dg_gemv_bf16(h, self.Wr, ws=ws["router"])
        ids, gate = dg.dg_moe_route(scores, self.topk, score=dg.DG_SCORE_SIGMOID, bias=self.bias, n_group=4, topk_group=2,
                                    group_top=2, scale=2.5)
        a = dg.dg_moe_w1_silu(h, ids, self.W1, self.s1, ws=ws["w1"])
        y = dg.dg_moe_w2(a, ids, gate, self.W2, self.s2, ws=ws["w2"])
        logits, pick = dg.dg_head_fp8_argmax(y, self.head, self.head_scale, ws=ws["head"])
        self.token.copy_(pick)
        return {"ids": ids, "gate": gate, "logits": logits, "token": self.token,
                **dg.dg_logprobs(logits, self.token, n_top=self.n_top)}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=248320)
    a = ap.parse_args()
    step = Step(a.rows, a.hidden, a.vocab)
    step()                                    # first calls load kernels; not inside a capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        graph.replay()
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{a.rows} rows: {start.elapsed_time(end) / 20 * 1000:.1f} us a step")
    for m in range(a.rows):
        print(f"row {m}: experts {out['ids'][m].tolist()}, token {int(out['token'][m])} at "
              f"{float(out['logprob'][m]):.3f} (rank {int(out['rank'][m])}, entropy {float(out['entropy'][m]):.3f}), "
              f"next {out['top_ids'][m].tolist()}")


if __name__ == "__main__":
    main()
