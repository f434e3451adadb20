"""The example's decode step: eager and replayed from a graph, checked call by call."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import _ref64 as R
from tests._helpers import ROOT

pytestmark = pytest.mark.gpu


def test_decode_step_example(cuda_device):
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    step = mod.Step(rows=4, hidden=512, vocab=4099, experts=32, inter=128)
    out = step()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in out.items()}
    # the step's last call against the reference, on the step's own logits
    ref = R.logprobs(want["logits"].float().cpu().numpy(), want["token"].cpu().numpy(), step.n_top)
    assert np.allclose(want["logprob"].cpu().numpy(), ref["logprob"], rtol=0, atol=4e-5 + 2 ** -21 * 20)
    assert np.array_equal(want["top_ids"].cpu().numpy(), ref["top_ids"])
    assert np.array_equal(want["rank"].cpu().numpy(), ref["rank"])
    assert (want["ids"] >= 0).all() and torch.allclose(want["gate"].sum(-1), torch.full((4,), 2.5, device="cuda"), rtol=1e-5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want)
