"""Calls given a stream make their buffers on it: a workspace zeroed on another stream, or a block
that is still in use there, would be written by both."""
import pytest
import torch

import gemv_dg_bf16_gb300 as dg

pytestmark = pytest.mark.gpu


def test_buffers_are_made_on_the_stream_given(cuda_device, monkeypatch):
    x = torch.randn((20, 256), device="cuda").to(torch.bfloat16)
    w = torch.randn((96, 256), device="cuda").to(torch.bfloat16)
    logits = torch.randn((5, 64), device="cuda")
    tok = torch.arange(5, device="cuda")
    q, s = dg.dg_quant_fp4_blockscale(w, dg.DG_FP4_NV)
    calls = [(lambda **kw: dg.dg_quant_fp4_blockscale(x, dg.DG_FP4_NV, **kw), 2),
             (lambda **kw: dg.dg_dequant_fp4_blockscale(q, s, dg.DG_FP4_NV, **kw), 1),
             (lambda **kw: dg.dg_gemv_a4w4_blockscale(x, q, s, dg.DG_FP4_NV, **kw), 2),
             (lambda **kw: dg.dg_moe_route(logits, 4, **kw), 2),
             (lambda **kw: dg.dg_logprobs(logits, tok, n_top=3, **kw), 5)]
    want = [c() for c, _ in calls]
    torch.cuda.synchronize()
    made = []
    for name in ("empty", "zeros"):
        real = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, real=real, **kw: (made.append(torch.cuda.current_stream()), real(*a, **kw))[1])
    st, before = torch.cuda.Stream(), torch.cuda.current_stream()
    for (call, n), ref in zip(calls, want):
        made.clear()
        got = call(stream=st)
        assert made == [st] * n and torch.cuda.current_stream() == before
        st.synchronize()
        for a, b in zip(*(v.values() if isinstance(v, dict) else v if isinstance(v, tuple) else (v,) for v in (got, ref))):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
