"""The distillation operators together, as examples/distill_step.py runs them: the first step's gradients against
torch's autograd in fp64, and a loss that falls."""
import importlib.util
import os

import pytest
import torch

from gpu_common import load_library, sync

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    load_library()
    spec = importlib.util.spec_from_file_location("distill_step", os.path.join(ROOT, "examples", "distill_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_gradients_of_a_step(ex):
    tokens, width, vocab, top, tau = 96, 72, 515, 12, 2.0
    st = ex.Student(tokens, width, vocab, 2, torch.float32)
    te = ex.Teacher(torch.ones(width, device="cuda"), torch.randn(vocab, width, device="cuda") * 0.1, tokens)
    for r, (x, residual) in enumerate(ex.batches(2, tokens, width, torch.float32)):
        t = te.top(x, residual, top)
        # the 8-bit teacher's logits: a row of either operand is off by half a step (1/254 of its largest value), so a
        # logit, a sum of width products, by at most that share of |h|max·Σ|w| + |w|max·Σ|h|
        h = x.double() + residual.double()
        n = h / ((h * h).mean(1, keepdim=True) + ex.EPS).sqrt()
        w = te.w.double() * te.w_scale.double()[:, None]
        exact = n @ w.t()
        bound = (n.abs().amax(1)[:, None] * w.abs().sum(1)) / 254
        assert torch.all((te.logits.double() - exact).abs() <= bound * 1.001 + 1e-5)
        loss = st.backward(r, x, residual, t.indices, t.values, tau).clone()
        sync()
        gamma = st.param(st.theta, 0).double().requires_grad_()
        head = st.param(st.theta, 1).double().requires_grad_()
        log_q = torch.log_softmax((n * gamma) @ head.t() / tau, 1).gather(1, t.indices)
        log_p = torch.log_softmax(t.values.double() / tau, 1)
        want = tau * tau * (log_p.exp() * (log_p - log_q)).sum(1)
        want.mean().backward()
        # fp32 throughout: sums of at most 515 products, each off by a few 2^-24 of its terms' size
        assert torch.all((loss.double() - want).abs() <= 1e-4 * (1 + want.abs()))
        for i, p in enumerate((gamma, head)):
            got = st.param(st.grads[r], i).double()
            assert (got - p.grad).norm() <= 1e-4 * p.grad.norm(), i


def test_loss_falls(ex):
    losses = ex.train(steps=12, tokens=128, width=64, vocab=1001, top=16)
    assert losses[-1] < 0.7 * losses[0] and all(v == v for v in losses)
