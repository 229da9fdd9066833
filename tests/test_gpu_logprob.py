"""Token log probabilities, entropy, top entries and their gradient on the GPU against the fp64 oracle.

Tolerances, with u = 2^-24 and x = (z − reference)·log2(e)/τ:
  2^x: the exponent is one multiply-add with a rounded log2(e)/τ, off by 2u·|x|; ex2.approx adds 2^-22 relative.  Terms
  with |x| above 30 are under 2^-30 of the sum.  The sum is a chain of at most V/512 pairs and a tree.  So a sum's
  relative error is at most S = (V/512 + 64)·u + 2^-22 + 60·u, and that of the sum of x·2^x the same of its absolute
  terms, whose share of Σ2^x is at most log2(V) + 8 (entropy's largest value, and what a reference may lie too low).
  lse = M/τ + ln Σ: S, and 4 roundings of |M/τ| and ln Σ.  log p: S, and 4 roundings of itself and of ln Σ.
  entropy: S·(log2(V) + 10).
  gradient: p is off by |lse|·u·2 (an fp32 lse), 4u·|log p| and 2^-22; its factor by a few roundings of its terms.
"""
import numpy as np
import pytest
import torch

from gpu_common import load_library, sync
from oracle import train_oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def g():
    return load_library()


def rand(shape, seed, std=1.0, dtype=torch.float32):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def targets(T, V, seed, dtype=torch.int64):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = torch.randint(0, V, (T,), generator=gen, device="cuda")
    if T > 2:
        t[1], t[2] = -100, V
    return t.to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def run(g, z, target, k, tau, index=torch.int64):
    T = z.shape[0]
    out = [torch.full((T,), 7.0, device="cuda") for _ in range(3)]
    ti = torch.full((T, k), -7, dtype=index, device="cuda") if k else None
    tl = torch.full((T, k), 7.0, device="cuda") if k else None
    g.token_logprobs_forward(z, target, *out, ti, tl, temperature=tau)
    sync()
    return (*out, ti, tl)


def near(got, want, tol):
    same = got == want                                   # infinities
    return np.all(same | (np.abs(got - np.where(same, got, want)) <= tol))


def check(z, target, tau, out, k):
    V = z.shape[1]
    logp, entropy, lse, ti, tl = out
    lw, ew, sw, iw, tw = O.token_logprobs(f64(z), target.cpu().numpy(), tau, k)
    S = (V / 512 + 64) * U + 2.0 ** -22 + 60 * U
    fin = np.isfinite(sw)
    top = np.abs(f64(z) / tau)
    top = np.where(np.isfinite(top), np.max(f64(z), axis=1, keepdims=True) / tau, 0)[:, 0]
    ln = np.log(V) + 8
    assert near(f64(lse)[fin], sw[fin], (S + 4 * U * (np.abs(top) + ln))[fin]) and np.array_equal(f64(lse)[~fin], sw[~fin])
    assert near(f64(logp), lw, S + 4 * U * (np.where(np.isfinite(lw), np.abs(lw), 0) + ln))
    assert near(f64(entropy), ew, S * (np.log2(V) + 10))
    if k:
        assert np.array_equal(ti.cpu().numpy(), iw)
        assert near(f64(tl), tw, S + 4 * U * (np.where(np.isfinite(tw), np.abs(tw), 0) + ln))


SHAPES = [(1, 1, 1), (3, 5, 8), (5, 17, 3), (2, 1000, 20), (1, 50257, 20), (4, 50257, 128), (1, 16385, 64),
          (2, 160000, 128), (700, 515, 5), (330, 9000, 128), (400, 32003, 64), (9, 2049, 1), (310, 2300, 77), (1, 4095, 2)]


@pytest.mark.parametrize("T,V,k", SHAPES)
@pytest.mark.parametrize("dt,tau", [("bf16", 1.0), ("f32", 0.7), ("f32", 2.0)])
def test_forward(g, T, V, k, dt, tau):
    z, target = rand((T, V), 1, 2.5, DT[dt]), targets(T, V, 2)
    out = run(g, z, target, k, tau)
    check(z, target, tau, out, k)
    again = run(g, z, target.int(), k, tau, torch.int32)
    for a, b in zip(out, again):
        assert torch.equal(a, b.to(a.dtype))
    plain = run(g, z, target, 0, tau)                    # without the entries: another kernel
    check(z, target, tau, plain, 0)


@pytest.mark.parametrize("T", [2, 320, 700])
@pytest.mark.parametrize("V", [700, 8003, 9001, 40000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_masks_and_shapes_of_rows(g, T, V, dt):
    """Every row of another kind; what no list holds goes by digits."""
    z = rand((T, V), 3, 2.0, DT[dt])
    low = torch.finfo(DT[dt]).min
    v = torch.arange(V, device="cuda")
    kinds = [lambda r: r.masked_fill_(v % 3 != 0, float("-inf")),       # part of the vocabulary
             lambda r: r.fill_(float("-inf")),                          # nothing left
             lambda r: r.fill_(float("-inf"))[V // 2:V // 2 + 1].fill_(3.0),   # one entry left
             lambda r: r.fill_(-1e9),                                   # a finite mask over all: uniform
             lambda r: r.masked_fill_(v != V - 1, low),                 # the type's lowest value
             lambda r: r.fill_(low),
             lambda r: r.fill_(1.5),                                    # all equal
             lambda r: r.fill_(0.0)[::2].fill_(-0.0),                   # 0 and −0 are equal
             lambda r: r.copy_(v.float() / V * 4),                      # ascending, with ties in bf16
             lambda r: r.copy_(-v.float() / V * 40),
             lambda r: r[v % 2048 < 8].add_(20.0),                      # the large ones with one thread
             lambda r: r[V - 150:].add_(30.0),
             lambda r: r[:150].add_(30.0),
             lambda r: r.add_(1e4),                                     # far from 0
             lambda r: r.add_(-3e5),
             lambda r: r.mul_(0.01)[V // 3].add_(60.0),                 # sure of one entry
             lambda r: r.clamp_(max=0.0)]                               # half of it tied at the top
    for k in (1, 20, 128):
        for i in range(0, len(kinds), T):
            x = z.clone()
            for t, kind in enumerate(kinds[i:i + T]):
                kind(x[t])
            target = targets(T, V, 4)
            out = run(g, x, target, k, 1.0)
            check(x[:len(kinds)], target[:len(kinds)], 1.0, tuple(o[:len(kinds)] for o in out), k)


@pytest.mark.parametrize("T,V", [(3, 9001), (320, 9001), (700, 9001), (700, 8003)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nan_and_infinity(g, T, V, dt):
    k = 6
    z = rand((T, V), 5, 2.0, DT[dt])
    z[0, [17, 8000]] = float("nan")
    z[0, 4] = float("inf")
    z[1, 5000] = float("inf")
    target = torch.zeros(T, dtype=torch.int64, device="cuda")
    logp, entropy, lse, ti, tl = run(g, z, target, k, 1.0)
    for t in (0, 1):
        assert torch.isnan(torch.stack([logp[t], entropy[t], lse[t]])).all() and torch.isnan(tl[t]).all()
    assert ti[0, :3].tolist() == [17, 8000, 4] and int(ti[1, 0]) == 5000
    check(z[2:], target[2:], 1.0, (logp[2:], entropy[2:], lse[2:], ti[2:], tl[2:]), k)
    z[2] = float("nan")                                  # nothing but NaN: in index order
    logp, entropy, lse, ti, tl = run(g, z, target, k, 1.0)
    assert torch.isnan(lse[2]) and ti[2].tolist() == list(range(k))


def grad_tol(z, lse, A, B, tau):
    lp = z / tau - lse[:, None]
    p = np.exp(np.where(np.isfinite(lp), lp, -1e4))
    lp = np.where(np.isfinite(lp), np.maximum(lp, -140), -140)
    rel = 2 * U * np.abs(lse)[:, None] + 6 * U * np.abs(lp) + 2.0 ** -22 + 8 * U
    return p * (np.abs(A)[:, None] + np.abs(B)[:, None] * (np.abs(lp) + 1)) / tau * rel


@pytest.mark.parametrize("T,V,_", SHAPES)
@pytest.mark.parametrize("dt,tau", [("bf16", 1.0), ("f32", 0.7), ("f32", 2.0)])
def test_backward(g, T, V, _, dt, tau):
    z, target = rand((T, V), 6, 2.0, DT[dt]), targets(T, V, 7)
    if V > 16:
        z[:, 3::7] = float("-inf")
    _, entropy, lse, _, _ = run(g, z, target, 0, tau)
    up, ue = rand((T,), 8), rand((T,), 9, 0.3)
    if T > 4:
        up[3] = ue[3] = 0
        z[3, 0] = float("nan")                           # of a token that takes nothing
    half = U if dt == "f32" else 2.0 ** -8
    for u, e in ((up, ue), (up, None), (None, ue)):
        dz = torch.full_like(z, float("nan"))
        g.token_logprobs_backward(z, target if u is not None else None, lse, u, dz, entropy if e is not None else None, e,
                                  temperature=tau)
        sync()
        zz, uu, ee = z.clone(), None if u is None else f64(u), None if e is None else f64(e)
        if T > 4:
            zz[3] = 0
        want = O.token_logprobs_grad(f64(zz), target.cpu().numpy(), tau, uu, ee)
        H = f64(entropy)
        A = (0 if u is None else np.abs(uu)) + (0 if e is None else np.abs(ee) * (H + 1))
        B = np.zeros(T) if e is None else np.abs(ee)
        tol = grad_tol(f64(zz), f64(lse), A * np.ones(T), B, tau)
        # the entropy it reads is off by its own tolerance
        tol += 0 if e is None else tol * 0 + np.abs(ee)[:, None] / tau * ((V / 512 + 64) * U + 2.0 ** -20) * (np.log2(V) + 10) * \
            np.exp(np.where(np.isfinite(f64(zz)), f64(zz) / tau - f64(lse)[:, None], -1e4))
        rows = np.arange(T)[(target.cpu().numpy() >= 0) & (target.cpu().numpy() < V)]
        if u is not None:
            tol[rows, target.cpu().numpy()[rows]] += 4 * U * np.abs(uu)[rows] / tau
        if T > 4:
            assert torch.all(dz[3] == 0)
            want[3] = 0
        assert np.all(np.abs(f64(dz) - want) <= tol + half * np.abs(want) + 1e-38)
        same = z.clone()                                 # in the logits' place
        g.token_logprobs_backward(same, target if u is not None else None, lse, u, same, entropy if e is not None else None,
                                  e, temperature=tau)
        sync()
        assert torch.equal(same, dz)


def test_backward_of_rows_without_a_distribution(g):
    T, V = 3, 5000
    z = rand((T, V), 10)
    z[0] = float("-inf")
    target = torch.zeros(T, dtype=torch.int64, device="cuda")
    z[1, 7] = float("nan")
    _, entropy, lse, _, _ = run(g, z, target, 0, 1.0)
    dz, up = torch.empty_like(z), torch.ones(T, device="cuda")
    g.token_logprobs_backward(z, target, lse, up, dz, entropy, up)
    sync()
    assert torch.all(dz[0] == 0) and torch.isnan(dz[1]).all() and torch.isfinite(dz[2]).all()


@pytest.mark.parametrize("V", [96, 5001])
def test_backward_against_differences(g, V):
    """Central differences of the forward kernel's own outputs along random directions."""
    T, e = 4, 2.0 ** -7
    z, target = rand((T, V), 11, 1.0), targets(T, V, 12)
    up, ue = rand((T,), 13), rand((T,), 14)

    def f(z):
        logp, entropy, lse, _, _ = run(g, z, target, 0, 1.0)
        return logp, entropy, lse
    _, entropy, lse = f(z)
    dz = torch.empty_like(z)
    g.token_logprobs_backward(z, target, lse, up, dz, entropy, ue)
    S = ((V / 512 + 64) * U + 2.0 ** -22 + 60 * U) * (np.log2(V) + 10)
    for seed in range(4):
        d = rand((T, V), 20 + seed)
        (lp, ep, _), (lm, em, _) = f(z + e * d), f(z - e * d)
        num = ((lp - lm).double() * up + (ep - em).double() * ue) / (2 * e)
        got = (dz.double() * d.double()).sum(1)
        # rounding of both ends over 2e; truncation e²/6 of third derivatives: moments of d under p, times ln V for H
        tol = 2 * S * (up.abs() + ue.abs()) / (2 * e) + e * e * 30 * np.log(V) * (up.abs() + ue.abs())
        assert torch.all((num - got).abs() <= tol)


@pytest.mark.parametrize("T", [5, 310, 700])
@pytest.mark.parametrize("V", [515, 8003, 8195])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strides_and_offsets(g, T, V, dt):
    """Column slices at odd offsets of wider buffers; what lies beside them stays."""
    k = 9
    buf = rand((T, V + 13), 30, 2.0, DT[dt])
    z, target = buf[:, 5:5 + V], targets(T, V, 31)
    ti = torch.full((T, k + 4), -7, dtype=torch.int64, device="cuda")
    tl = torch.full((T, k + 3), 7.0, device="cuda")
    out = [torch.empty(T, device="cuda") for _ in range(3)]
    g.token_logprobs_forward(z, target, *out, ti[:, 2:2 + k], tl[:, 1:1 + k])
    sync()
    check(z, target, 1.0, (*out, ti[:, 2:2 + k], tl[:, 1:1 + k]), k)
    assert torch.all(ti[:, :2] == -7) and torch.all(ti[:, 2 + k:] == -7)
    assert torch.all(tl[:, :1] == 7) and torch.all(tl[:, 1 + k:] == 7)
    up = rand((T,), 32)
    dense = torch.empty(T, V, device="cuda", dtype=DT[dt])
    g.token_logprobs_backward(z.contiguous(), target, out[2], up, dense)
    for off in (0, 3):                                   # rows of dz that do not lie as those of z
        db = torch.full((T, V + 10), 7.0, device="cuda", dtype=DT[dt])
        g.token_logprobs_backward(z, target, out[2], up, db[:, off:off + V])
        sync()
        assert torch.equal(db[:, off:off + V], dense)
        assert torch.all(db[:, :off] == 7) and torch.all(db[:, off + V:] == 7)


def test_outputs_alone_and_empty(g):
    z, target = rand((6, 3000), 40), targets(6, 3000, 41)
    want = run(g, z, target, 4, 1.0)
    for i in range(5):
        one = torch.full_like(want[i], 5)
        args = [one if j == i else None for j in range(5)]
        g.token_logprobs_forward(z, target, *args)
        sync()
        assert torch.equal(one, want[i])
    g.token_logprobs_forward(z, None, None, *[None] * 4)
    e = torch.empty(0, 64, device="cuda")
    none = torch.empty(0, device="cuda")
    g.token_logprobs_forward(e, torch.empty(0, dtype=torch.int64, device="cuda"), none)
    g.token_logprobs_backward(e, None, none, None, e, none, none)
    sync()


@pytest.mark.parametrize("T,V", [(3, 50257), (400, 8003)])
def test_other_stream_repeat_and_graph(g, T, V):
    """The same bits on a side stream, on every repeat and in a graph's replay."""
    z, target, k = rand((T, V), 50, 2.0, torch.bfloat16), targets(T, V, 51), 33
    bufs = [torch.empty(T, device="cuda") for _ in range(3)] + [
        torch.empty(T, k, dtype=torch.int64, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty_like(z)]

    def step(stream=None):
        g.token_logprobs_forward(z, target, *bufs[:5], stream=stream)
        g.token_logprobs_backward(z, target, bufs[2], bufs[0], bufs[5], bufs[1], bufs[1], stream=stream)
    step()
    sync()
    first = [b.clone() for b in bufs]
    side = torch.cuda.Stream()
    for how in ("side", "graph"):
        for b in bufs:
            b.zero_()
        sync()
        if how == "side":
            step(side)
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            graph.replay()
        sync()
        for b, f in zip(bufs, first):
            assert torch.equal(b, f), how


def test_entries_feed_the_distillation_loss(g):
    """The teacher's entries as log probabilities instead of logits: a softmax does not see the difference."""
    T, V, k = 20, 3001, 40
    z, teacher = rand((T, V), 60), rand((T, V), 61, 2.0)
    index, logp = torch.empty(T, k, dtype=torch.int64, device="cuda"), torch.empty(T, k, device="cuda")
    g.token_logprobs_forward(teacher, None, None, None, None, index, logp)
    a, b = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    g.distill_topk_forward(z, index, logp, a)
    g.distill_topk_forward(z, index, teacher.gather(1, index), b)
    sync()
    assert torch.all((a - b).abs() <= 64 * U * 20)


def test_offsets_past_32_bits(g):
    T, V, k = (1 << 31) // 131072 + 3, 131072, 5
    z = torch.zeros(T, V, device="cuda", dtype=torch.bfloat16)
    z[-2:] = rand((2, V), 70, 2.0, torch.bfloat16)
    target = targets(T, V, 71)
    out = run(g, z, target, k, 1.0)
    check(z[-2:], target[-2:], 1.0, tuple(o[-2:] for o in out), k)
    dz, up = torch.empty_like(z), torch.ones(T, device="cuda")
    g.token_logprobs_backward(z, target, out[2], up, dz)
    sync()
    want = O.token_logprobs_grad(f64(z[-2:]), target[-2:].cpu().numpy(), 1.0, np.ones(2), None)
    tol = grad_tol(f64(z[-2:]), f64(out[2][-2:]), np.ones(2), np.zeros(2), 1.0)
    assert np.all(np.abs(f64(dz[-2:]) - want) <= tol + 8 * U * (want > 0.5) + 2.0 ** -8 * np.abs(want) + 1e-38)
