"""The quantisation-aware distillation example: its operators together, as a training step uses them."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import fp4_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qad(nv):
    path = os.path.join(os.path.dirname(os.path.dirname(__file__)), "examples", "qad_step.py")
    spec = importlib.util.spec_from_file_location("qad_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_lowers_the_loss(qad):
    """From the loss of plain rounding to the grid, 30 steps of gradient descent take off a good part."""
    losses = qad.train(30)
    assert np.isfinite(losses).all() and losses[0] > 0
    assert min(losses[-5:]) < 0.8 * losses[0]


def test_training_is_reproducible(qad):
    assert qad.train(4) == qad.train(4)


def test_one_step_against_64_bits(qad):
    """Logits, loss and both weight gradients of a step against the same step in 64 bits, where each stage takes the
    values that the stage before it handed on (so that a code at a rounding edge cannot come out differently)."""
    nv = qad.nv
    tokens, features, hidden, vocab, k = 70, 64, 96, 320, 9
    g = torch.Generator("cuda").manual_seed(3)
    w1 = (torch.randn(hidden, features, device="cuda", generator=g) / 8).bfloat16()
    w2 = (torch.randn(vocab, hidden, device="cuda", generator=g) / 3).bfloat16()
    x = torch.randn(tokens, features, device="cuda", generator=g).bfloat16()
    index, logp = qad.teacher_entries(x, w1, w2, k)
    s = qad.Student(w1, w2, tokens)
    z, saved = s.forward(x)
    h = ref.to64(saved[2])
    cols = lambda v: ref.mx_round(np.ascontiguousarray(ref.pad_rows(v).T))  # noqa: E731
    z64 = ref.mx_round(h) @ ref.mx_round(ref.to64(s.w2)).T
    assert (np.abs(ref.to64(z) - z64) <= 2.0 ** -8 * np.abs(z64) + 1e-4).all()
    loss, dz = nv.distill_topk_loss_grad(z, index, logp, tail=True)
    rl, rd = ref.distill(ref.to64(z), index.cpu().numpy(), ref.to64(logp), tail=True)
    assert np.allclose(ref.to64(loss), rl, rtol=1e-4, atol=1e-5)
    assert (np.abs(ref.to64(dz) - rd) <= 2.0 ** -8 * np.abs(rd) + 1e-5).all()
    dw1, dw2 = s.backward(dz, saved)
    d64 = ref.to64(dz)
    want2 = cols(d64) @ cols(h).T
    assert (np.abs(ref.to64(dw2) - want2) <= 1e-5 * (np.abs(cols(d64)) @ np.abs(cols(h)).T) + 1e-9).all()
    assert dw1.shape == w1.shape and torch.isfinite(dw1).all()
