"""Distilling a student from an 8-bit teacher, data-parallel: every operator of a step together.

Per step and replica: the teacher's residual stream is normalised into 8-bit rows (rmsnorm_forward_q8) and multiplied
with its 8-bit head (q8_matmul); its k largest logits are the targets.  The student normalises its own stream
(rmsnorm_forward), computes its logits, takes loss and gradient of the logits in one call
(distill_topk_forward_backward) and goes back through its norm (rmsnorm_backward).  The replicas' gradients lie in flat
buckets (ddp_plan_buckets) that are averaged with the SGD step fused (ddp_bucket_allreduce_sgd).

    python examples/distill_step.py [--steps 20] [--tokens 512] [--width 256] [--vocab 4099] [--top 32]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gradient_sync_ddp_gb300 as g  # noqa: E402

EPS = 1e-6


def quantise_rows(w):
    """Weights laid out once: 8-bit rows with one scale each."""
    scale = w.abs().amax(1) / 127
    return torch.round(w / scale[:, None]).to(torch.int8), scale


class Teacher:
    """The last norm and the head of a teacher that runs in 8 bits."""

    def __init__(self, gamma, head, tokens):
        self.gamma, (self.w, self.w_scale) = gamma, quantise_rows(head)
        V, D = head.shape
        self.q = torch.empty(tokens, D, dtype=torch.int8, device="cuda")
        self.scale = torch.empty(tokens, device="cuda")
        self.logits = torch.empty(tokens, V, device="cuda")
        self.ws = torch.empty(g.q8_matmul_workspace_bytes(tokens, V, D), dtype=torch.uint8, device="cuda")

    def top(self, x, residual, k):
        g.rmsnorm_forward_q8(x, self.gamma, self.q, self.scale, EPS, residual=residual)
        g.q8_matmul(self.q, self.scale, self.w, self.w_scale, self.logits, self.ws)
        return torch.topk(self.logits, k, dim=1)


class Student:
    """Norm and head; parameters gamma [D] and head [V, D] in one flat fp32 buffer, laid out by the bucket plan."""

    def __init__(self, tokens, width, vocab, replicas, dtype, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.shapes = [(width,), (vocab, width)]
        self.plan = g.ddp_plan_buckets([width, vocab * width], 4, 25 << 20)
        n = self.plan["total_elems"]
        self.theta, self.momentum = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        self.grads = [torch.zeros(n, device="cuda") for _ in range(replicas)]
        self.param(self.theta, 0).fill_(1.0)
        self.param(self.theta, 1).copy_(torch.randn(vocab, width, generator=gen, device="cuda") * 0.02)
        self.dtype, make = dtype, lambda *s, t=dtype: torch.empty(*s, dtype=t, device="cuda")
        self.h, self.y, self.dy, self.dx = (make(tokens, width) for _ in range(4))
        self.rstd, self.loss = make(tokens, t=torch.float32), make(tokens, t=torch.float32)
        self.logits = make(tokens, vocab)
        self.up = torch.full((tokens,), 1.0 / tokens, device="cuda")
        self.ws = make(g.rmsnorm_backward_workspace_bytes(tokens, width), t=torch.uint8)

    def param(self, flat, i):
        off = self.plan["tensor_offset"][i]
        n = 1
        for s in self.shapes[i]:
            n *= s
        return flat[off:off + n].view(self.shapes[i])

    def backward(self, replica, x, residual, index, teacher, temperature):
        """Loss per token of one replica's batch; its gradients go to its flat buffer."""
        gamma, head = self.param(self.theta, 0), self.param(self.theta, 1).to(self.dtype)
        dgamma, dhead = self.param(self.grads[replica], 0), self.param(self.grads[replica], 1)
        g.rmsnorm_forward(x, gamma, self.y, EPS, residual=residual, h_out=self.h, rstd_out=self.rstd)
        torch.matmul(self.y, head.t(), out=self.logits)
        g.distill_topk_forward_backward(self.logits, index, teacher, self.up, self.loss, None, self.logits,
                                        temperature=temperature)              # the gradient in the logits' place
        dhead.copy_(self.logits.t() @ self.y)
        torch.matmul(self.logits, head, out=self.dy)
        g.rmsnorm_backward(self.dy, self.h, self.rstd, gamma, self.dx, dgamma, self.ws)
        return self.loss

    def step(self, lr, momentum):
        for off, n, _, _ in self.plan["buckets"]:
            g.ddp_bucket_allreduce_sgd([b[off:off + n] for b in self.grads], self.theta[off:off + n],
                                       self.momentum[off:off + n], lr, momentum, 0.0)


def batches(replicas, tokens, width, dtype, seed=1):
    """One fixed batch per replica: a residual stream and what the last block adds to it."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [tuple((torch.randn(tokens, width, generator=gen, device="cuda")).to(dtype) for _ in range(2))
            for _ in range(replicas)]


def train(steps=20, tokens=512, width=256, vocab=4099, top=32, replicas=2, dtype=torch.bfloat16, temperature=2.0,
          lr=3.0, momentum=0.9):
    """Mean loss of every step."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    teacher = Teacher(1 + 0.1 * torch.randn(width, generator=gen, device="cuda"),
                      torch.randn(vocab, width, generator=gen, device="cuda") * 0.1, tokens)
    student, data, losses = Student(tokens, width, vocab, replicas, dtype), batches(replicas, tokens, width, dtype), []
    for _ in range(steps):
        total = torch.zeros((), device="cuda")
        for r, (x, residual) in enumerate(data):
            targets = teacher.top(x, residual, top)
            total += student.backward(r, x, residual, targets.indices, targets.values, temperature).mean()
        student.step(lr, momentum)
        losses.append(total / replicas)
    return [float(v) for v in torch.stack(losses)]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 20), ("tokens", 512), ("width", 256), ("vocab", 4099), ("top", 32)):
        ap.add_argument("--" + name, type=int, default=value)
    for i, loss in enumerate(train(**vars(ap.parse_args()))):
        print(f"step {i}: loss {loss:.4f}")
