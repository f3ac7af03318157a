"""The plain form and the 64-bit form of the selection's cases against the oracle, where fewer pairs exist than are asked for (CPU)."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from conftest import ROOT
from oracle import beam


@pytest.fixture(scope="module")
def cases():
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("alpha", [0.0, 0.7])
@pytest.mark.parametrize("W,K,ended", [(1, 4, [[1], [0]]), (2, 5, [[1, 1], [0, 1], [0, 0]]), (3, 6, [[1, 1, 1], [1, 0, 1]]), (2, 2, [[1, 1]])])
def test_selections_that_run_out_of_pairs(cases, W, K, ended, alpha):
    """An ended beam offers itself alone; what is missing from K is token -1, parent -1, score -inf, ended, of length 0."""
    B, V, eos = len(ended), 40, 2
    g = torch.Generator().manual_seed(W)
    ended = torch.tensor(ended, dtype=torch.int32)
    s = {"case": {"K": K, "alpha": alpha}, "logits": 2.5 * torch.randn(B, W, V, generator=g), "scores": -torch.rand(B, W, generator=g) - 8.0,
         "eos": eos, "ended": ended, "length": torch.where(ended > 0, torch.randint(1, 12, (B, W), generator=g).int(), 12).int()}
    want = beam.beam_select(s["logits"].double().numpy(), s["scores"].numpy(), K, eos=eos, ended=ended.numpy(), length=s["length"].numpy(), alpha=alpha)
    for form in (cases._run_select, cases._exact_select):
        got = form(s)
        for name in ("token", "parent", "ended", "length"):
            np.testing.assert_array_equal(got[name].numpy(), want[name], err_msg=f"{form.__name__} {name}")
        # 40 exponentials and their sum's logarithm in 32 bits, and the score's own rounding, half a step of at most 16
        np.testing.assert_allclose(got["score"].numpy(), want["score"], rtol=0, atol=48 * 2.0 ** -24 + 16 * 2.0 ** -24)
