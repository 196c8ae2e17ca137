"""Calls at the edges of the gated delta rule's and the head norms' entry points: no tokens, streams,
frozen weights, gradients as autograd hands them, rows far apart."""
import numpy as np
import pytest
import torch

import linear_attention_diffusion_litela_b200 as ll
from linear_attention_diffusion_litela_b200 import seq
from tests.test_gpu_delta import autograd, fwd, make, ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_diffusion_litela_b200.build import build
    build()


@pytest.mark.parametrize("lens,packed", [([0, 0, 0], True), ([0], True), ([0, 0], False)])
@pytest.mark.parametrize("d,carry", [(32, True), (128, True), (64, False)])
def test_a_training_step_without_tokens(lens, packed, d, carry):
    """The states pass through, and so do their gradients"""
    t = make(lens, packed, 1, 2, d, carry, seed=d)
    for n in ("q", "k", "v", "g", "beta"):
        t[n].requires_grad_()
    out, state, grads = autograd(t)
    assert out.shape == t["v"].shape and all(grads[n].shape == t[n].shape for n in grads)
    assert torch.equal(state, t["state_in"] if carry else torch.zeros_like(t["dstate"]))
    if carry:
        assert torch.equal(grads["state_in"], t["dstate"])
