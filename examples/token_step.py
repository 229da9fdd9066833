"""Training a small transformer block data-parallel: every operator of a step together.

A block of pre-norm residual form over given token vectors x, and a head over the vocabulary:

    y1 = layernorm(x);  a = y1 W1;  h = x + relu(a) W2;  y2 = layernorm(h);  logits = y2 head^T

Per step and replica: layernorm_forward (the second one adds the block's output to the stream), the log probability of
every token's target with the entropy (token_logprobs_forward), the loss -mean(log p) - beta * mean(entropy), and back:
token_logprobs_backward in the logits' place, layernorm_backward (the stream's gradient added to the norm's).  The
gradients lie in a flat buffer laid out by ddp_plan_buckets.  The matrices W1 and W2 take the orthogonalised step on the
replicas' average (ddp_bucket_allreduce_muon), the rest the SGD step (ddp_bucket_allreduce_sgd).

    python examples/token_step.py [--steps 20] [--tokens 512] [--width 256] [--vocab 4099] [--top 5]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gradient_sync_ddp_gb300 as g  # noqa: E402

EPS, BETA = 1e-5, 0.01


class Block:
    """Parameters in one flat fp32 buffer, laid out by the bucket plan; activations and gradients of one replica's batch."""

    NAMES = ("gamma1", "beta1", "w1", "w2", "gamma2", "beta2", "head")

    def __init__(self, tokens, width, vocab, replicas, dtype, seed=0):
        D, F, V = width, 4 * width, vocab
        self.shapes = dict(zip(self.NAMES, ((D,), (D,), (D, F), (F, D), (D,), (D,), (V, D))))
        sizes = [math.prod(s) for s in self.shapes.values()]
        self.plan = g.ddp_plan_buckets(sizes, 4, 25 << 20)
        n = self.plan["total_elems"]
        self.theta, self.momentum = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        self.grads = [torch.zeros(n, device="cuda") for _ in range(replicas)]
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for name, std in (("w1", D ** -0.5), ("w2", F ** -0.5), ("head", 0.02)):
            p = self.param(self.theta, name)
            p.copy_(torch.randn(p.shape, generator=gen, device="cuda") * std)
        for name in ("gamma1", "gamma2"):
            self.param(self.theta, name).fill_(1.0)
        self.dtype, make = dtype, lambda *s, t=dtype: torch.empty(*s, dtype=t, device="cuda")
        self.y1, self.y2, self.h, self.dy, self.dh, self.dx = (make(tokens, D) for _ in range(6))
        self.stats = [make(tokens, t=torch.float32) for _ in range(4)]               # mean and rstd of either norm
        self.logprob, self.entropy, self.lse = (make(tokens, t=torch.float32) for _ in range(3))
        self.logits = make(tokens, V)
        self.up = torch.full((tokens,), -1.0 / tokens, device="cuda")                # of the loss by each log probability
        self.ue = torch.full((tokens,), -BETA / tokens, device="cuda")
        self.ws = make(g.layernorm_backward_workspace_bytes(tokens, D), t=torch.uint8)
        self.ns_ws = make(max(g.newton_schulz_workspace_bytes(1, D, F), g.newton_schulz_workspace_bytes(1, F, D)), t=torch.uint8)

    def offset(self, name):
        return self.plan["tensor_offset"][self.NAMES.index(name)]

    def param(self, flat, name):
        o = self.offset(name)
        return flat[o:o + math.prod(self.shapes[name])].view(self.shapes[name])

    def forward(self, x, target, top_index=None, top_logprob=None):
        """Log probability of every token's target, entropies, and, where asked for, the most probable tokens."""
        p = {n: self.param(self.theta, n) for n in self.NAMES}
        m1, r1, m2, r2 = self.stats
        g.layernorm_forward(x, p["gamma1"], p["beta1"], self.y1, EPS, mean_out=m1, rstd_out=r1)
        self.a = torch.relu(self.y1 @ p["w1"].to(self.dtype))
        g.layernorm_forward(self.a @ p["w2"].to(self.dtype), p["gamma2"], p["beta2"], self.y2, EPS, residual=x, h_out=self.h,
                            mean_out=m2, rstd_out=r2)
        torch.matmul(self.y2, p["head"].to(self.dtype).t(), out=self.logits)
        g.token_logprobs_forward(self.logits, target, self.logprob, self.entropy, self.lse, top_index, top_logprob)
        return self.logprob, self.entropy

    def backward(self, replica, x, target):
        """After forward: the replica's gradients, into its flat buffer."""
        p = {n: self.param(self.theta, n) for n in self.NAMES}
        d = {n: self.param(self.grads[replica], n) for n in self.NAMES}
        m1, r1, m2, r2 = self.stats
        g.token_logprobs_backward(self.logits, target, self.lse, self.up, self.logits, self.entropy, self.ue)
        d["head"].copy_(self.logits.t() @ self.y2)
        torch.matmul(self.logits, p["head"].to(self.dtype), out=self.dy)
        g.layernorm_backward(self.dy, self.h, m2, r2, p["gamma2"], self.dh, d["gamma2"], d["beta2"], self.ws)
        d["w2"].copy_(self.a.t() @ self.dh)
        da = (self.dh @ p["w2"].to(self.dtype).t()) * (self.a > 0)
        d["w1"].copy_(self.y1.t() @ da)
        torch.matmul(da, p["w1"].to(self.dtype).t(), out=self.dy)
        g.layernorm_backward(self.dy, x, m1, r1, p["gamma1"], self.dx, d["gamma1"], d["beta1"], self.ws, dh=self.dh)

    def step(self, lr, momentum=0.95, weight_decay=0.01):
        for name in ("w1", "w2"):
            rows, cols = self.shapes[name]
            g.ddp_bucket_allreduce_muon(self.grads, [self.offset(name)], rows, cols, self.theta, self.momentum, self.ns_ws,
                                        lr, momentum, weight_decay, update_scale=0.2 * max(rows, cols) ** 0.5)
        for name in ("gamma1", "beta1", "gamma2", "beta2", "head"):
            o, n = self.offset(name), math.prod(self.shapes[name])
            g.ddp_bucket_allreduce_sgd([b[o:o + n] for b in self.grads], self.theta[o:o + n], self.momentum[o:o + n], lr,
                                       momentum, 0.0)


def batches(replicas, tokens, width, vocab, dtype, seed=1):
    """One fixed batch per replica: token vectors, and targets of which a few are padding."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(replicas):
        x = torch.randn(tokens, width, generator=gen, device="cuda").to(dtype)
        target = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
        target[::17] = -100
        out.append((x, target))
    return out


def train(steps=20, tokens=512, width=256, vocab=4099, top=5, replicas=2, dtype=torch.bfloat16, lr=0.02):
    """Mean negative log probability of every step, and the last step's most probable tokens with their log probabilities."""
    block, data, losses = Block(tokens, width, vocab, replicas, dtype), batches(replicas, tokens, width, vocab, dtype), []
    index = torch.empty(tokens, top, dtype=torch.int64, device="cuda")
    logprob = torch.empty(tokens, top, device="cuda")
    for _ in range(steps):
        total = torch.zeros((), device="cuda")
        for r, (x, target) in enumerate(data):
            total -= block.forward(x, target, index, logprob)[0].mean()
            block.backward(r, x, target)
        block.step(lr)
        losses.append(total / replicas)
    return [float(v) for v in torch.stack(losses)], index, logprob


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 20), ("tokens", 512), ("width", 256), ("vocab", 4099), ("top", 5)):
        ap.add_argument("--" + name, type=int, default=value)
    for i, loss in enumerate(train(**vars(ap.parse_args()))[0]):
        print(f"step {i}: loss {loss:.4f}")
