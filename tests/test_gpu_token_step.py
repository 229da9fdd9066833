"""The training step's operators together, as examples/token_step.py runs them: a step's loss and gradients against
torch's autograd in fp64, and its update against the definitions."""
import importlib.util
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from gpu_common import load_library, sync
from oracle import train_oracle as O

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    load_library()
    spec = importlib.util.spec_from_file_location("token_step", os.path.join(ROOT, "examples", "token_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_gradients_and_update_of_a_step(ex):
    tokens, width, vocab, replicas = 96, 72, 515, 2
    b = ex.Block(tokens, width, vocab, replicas, torch.float32)
    top_i = torch.empty(tokens, 3, dtype=torch.int64, device="cuda")
    top_l = torch.empty(tokens, 3, device="cuda")
    for r, (x, target) in enumerate(ex.batches(replicas, tokens, width, vocab, torch.float32)):
        logp, entropy = (t.clone() for t in b.forward(x, target, top_i, top_l))
        b.backward(r, x, target)
        sync()
        p = {n: b.param(b.theta, n).double().requires_grad_() for n in b.NAMES}
        ln = torch.nn.functional.layer_norm
        y1 = ln(x.double(), (width,), p["gamma1"], p["beta1"], ex.EPS)
        h = x.double() + torch.relu(y1 @ p["w1"]) @ p["w2"]
        z = torch.log_softmax(ln(h, (width,), p["gamma2"], p["beta2"], ex.EPS) @ p["head"].t(), 1)
        inside = target >= 0
        want = torch.where(inside, z.gather(1, target.clamp(min=0)[:, None])[:, 0], 0.0)
        ent = -(z.exp() * z).sum(1)
        (-want.mean() - ex.BETA * ent.mean()).backward()
        # fp32 throughout: sums of at most 515 products, each off by a few 2^-24 of its terms' size
        assert torch.all((logp.double() - want).abs() <= 1e-4 * (1 + want.abs()))
        assert torch.all((entropy.double() - ent).abs() <= 1e-4 * (1 + ent))
        best = torch.topk(z, 3, dim=1)
        assert torch.all((top_l.double() - best.values).abs() <= 1e-4 * (1 + best.values.abs()))
        assert torch.all((z.gather(1, top_i) - best.values).abs() <= 2e-4)
        for n in b.NAMES:
            got = b.param(b.grads[r], n).double()
            assert float((got - p[n].grad).norm()) <= 1e-4 * float(p[n].grad.norm()), n
    before = {n: b.param(b.theta, n).double().cpu().numpy() for n in b.NAMES}
    b.step(0.02)
    sync()
    for n in b.NAMES:
        gr = [b.param(x, n).double().cpu().numpy() for x in b.grads]
        got = b.param(b.theta, n).double().cpu().numpy()
        if n in ("w1", "w2"):
            want, buf = O.muon_step(gr, before[n], np.zeros_like(before[n]), 0.02, 0.95, 0.01, 0.2 * max(gr[0].shape) ** 0.5)
            tol = 6e-3                       # of the orthogonalised update: test_gpu_muon derives it
        else:
            buf = np.mean(gr, axis=0)
            want, tol = before[n] - 0.02 * buf, 1e-6
        moved = np.linalg.norm(want - before[n])
        assert np.linalg.norm(got - want) <= tol * moved + 2.0 ** -22 * np.linalg.norm(want), n
        assert np.allclose(b.param(b.momentum, n).double().cpu().numpy(), buf, rtol=1e-6, atol=1e-12), n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_runs(ex, dtype):
    losses, index, logprob = ex.train(steps=4, tokens=128, width=64, vocab=1001, top=4, dtype=dtype)
    assert len(losses) == 4 and all(math.isfinite(v) for v in losses)
    assert torch.all((index >= 0) & (index < 1001)) and torch.all(logprob[:, :-1] >= logprob[:, 1:])


def test_example_as_a_program():
    load_library()
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "token_step.py"), "--steps", "2", "--tokens", "64",
                        "--width", "64", "--vocab", "515"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.count("loss") == 2, r.stderr[-2000:]
