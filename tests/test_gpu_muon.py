"""Newton-Schulz orthogonalisation and the optimizer step that takes it, on the GPU against the fp64 oracle.

Tolerances.  The kernels round operands to fp16 at known places; `emulate` does the same roundings with 64-bit sums, so
what is left between the two are fp32 sums (relative 2^-24·sqrt(K) of a 2-norm, at most 2^-18 here) and the entries that
these move across a rounding boundary: a share of 2^-18 / 2^-11 of them by 2^-11, 2^-14.5 in the 2-norm.  A step
carries a difference on at most by a factor a = 3.4445 in absolute terms, where it grows X itself as much as long as
singular values are small, and by about 1 from then on: six roundings of five steps, one after another, 30·2^-14.5.
Steps past the fifth act on singular values of about 1, where the polynomial's slope a + 3bs² + 5cs⁴ is steepest at
s² = −3b/10c = 0.705, −1.605: each carries a difference on by up to that factor.
The emulation itself is within 4e-3 of the exact steps for the matrices used here, 8e-3 with fewer than 16 rows, whose
roundings do not average out: computed below as well.
"""
import math

import numpy as np
import pytest
import torch

from gpu_common import load_library, sync
from oracle import train_oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NEAR = 30 * 2.0 ** -14.5


def exact_tol(rows, cols):
    return 4e-3 if min(rows, cols) >= 16 else 8e-3


@pytest.fixture(scope="module")
def g():
    return load_library()


def rand(shape, seed, std=1.0, dtype=torch.float32):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def emulate(x, steps=5, eps=1e-7):
    a, b, c = O.NS
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    norm = float(x.norm())
    if norm == 0:
        return torch.zeros_like(x).t() if tall else torch.zeros_like(x)
    k = 2.0 ** math.floor(math.log2(min(math.sqrt(x.numel()), 32768.0) / norm))
    alpha, full = 1 / ((norm + eps) * k), x * k

    def r(v):
        return v.half().double()
    for i in range(steps):
        hi = r(full)
        lo = r(full - hi) if i < steps - 2 else 0
        s = 1.0 if i >= max(steps - 2, 2) else 0.0       # of A − I
        gram = r(alpha * alpha * (hi @ hi.t()) - s * torch.eye(len(hi), dtype=torch.float64, device=hi.device))
        poly = r((b + 2 * c * s) * gram + c * (gram @ gram) + s * (a + b + c) * torch.eye(len(hi), dtype=torch.float64, device=hi.device))
        full = alpha * ((1 - s) * a * (hi + lo) + poly @ hi)
        alpha = 1.0
    return full.t() if tall else full


def ws_for(g, count, rows, cols):
    ws = torch.empty(g.newton_schulz_workspace_bytes(count, rows, cols), dtype=torch.uint8, device="cuda")
    return ws.fill_(255)


def check(got, x, steps=5, eps=1e-7):
    em = emulate(x, steps, eps)
    ex = torch.from_numpy(np.ascontiguousarray(O.newton_schulz(x.double().cpu().numpy(), steps, eps))).cuda()
    size = float(ex.norm())
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else U
    EXACT = exact_tol(*x.shape)
    assert float((em - ex).norm()) <= EXACT * size
    assert float((got.double() - em).norm()) <= (NEAR * 1.605 ** max(0, steps - 5) + half) * size, float((got.double() - em).norm()) / size
    # no entry far off: the 2-norm would not see one of them in a large matrix
    assert float((got.double() - ex).abs().max()) <= EXACT * size + half * float(ex.abs().max())


# a vector, widths around the padding and the tiles, both sides of the diagonal's tiles, tall and wide
SHAPES = [(1, 1), (1, 7), (9, 1), (3, 5), (64, 64), (65, 130), (130, 65), (200, 1000), (1000, 200), (256, 256), (300, 300),
          (513, 770), (768, 768), (1000, 2048)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_orthogonalise(g, rows, cols, dt, out):
    x = rand((rows, cols), 1, 1e-3, DT[dt])
    y = torch.full((rows, cols), float("nan"), device="cuda", dtype=DT[out])
    g.newton_schulz([x], [y], ws_for(g, 1, rows, cols))
    sync()
    check(y, x)


@pytest.mark.parametrize("count,rows,cols", [(2, 70, 33), (12, 768, 768), (70, 40, 50), (5, 300, 700), (3, 1100, 600), (9, 256, 512)])
def test_many(g, count, rows, cols):
    """Every matrix as if alone, whatever its size beside the others'."""
    xs = [rand((rows, cols), 10 + i, 10.0 ** (i % 7 - 3)) for i in range(count)]
    ys = [torch.full_like(x, float("nan")) for x in xs]
    g.newton_schulz(xs, ys, ws_for(g, count, rows, cols))
    sync()
    for x, y in zip(xs, ys):
        check(y, x)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 9])
def test_steps(g, steps):
    x = rand((150, 200), 30)
    y = torch.empty_like(x)
    g.newton_schulz([x], [y], ws_for(g, 1, 150, 200), steps=steps)
    sync()
    check(y, x, steps)


@pytest.mark.parametrize("rows,cols", [(200, 300), (640, 640)])
@pytest.mark.parametrize("power", [0, 1])
def test_spectra(g, rows, cols, power):
    """Singular values all equal, and falling as 1/i: the small ones are grown with what they were rounded by."""
    m = min(rows, cols)
    u, v = torch.linalg.qr(rand((rows, m), 31).double())[0], torch.linalg.qr(rand((cols, m), 32).double())[0]
    x = (u * torch.arange(1, m + 1, device="cuda").double() ** -power @ v.t()).float()
    y = torch.empty_like(x)
    g.newton_schulz([x], [y], ws_for(g, 1, rows, cols))
    sync()
    check(y, x)
    if power == 0:                       # equal singular values stay equal: X·Xᵀ is a multiple of the identity
        s = O.newton_schulz(np.diag(np.ones(m)) / 1.0)[0, 0]
        gram = y.double() @ y.double().t() if rows <= cols else y.double().t() @ y.double()
        assert float((gram - s * s * torch.eye(m, device="cuda")).norm()) <= 2 * (exact_tol(rows, cols) + NEAR) * s * s * m ** 0.5


def test_zeros_nan_and_scale(g):
    """Zeros give zeros; a matrix that is not finite gives NaN and leaves the others alone; any magnitude."""
    xs = [rand((100, 140), 40 + i) for i in range(8)]
    xs[1].zero_()
    xs[2][50, 60] = float("nan")
    xs[3][0, 0] = float("inf")
    xs[4] *= 1e-12
    xs[5] *= 1e15
    xs[6].zero_()[7, 9] = -4.0           # a single entry
    ys = [torch.full_like(x, 5.0) for x in xs]
    g.newton_schulz(xs, ys, ws_for(g, 8, 100, 140), eps=0.0)
    sync()
    assert torch.all(ys[1] == 0) and torch.isnan(ys[2]).all() and torch.isnan(ys[3]).all()
    for i in (0, 4, 5, 6, 7):
        check(ys[i], xs[i], eps=0.0)
    small = rand((100, 140), 50, 1e-10)  # beside the eps
    g.newton_schulz([small], [ys[0]], ws_for(g, 1, 100, 140), eps=1e-7)
    sync()
    check(ys[0], small, eps=1e-7)


@pytest.mark.parametrize("rows,cols", [(70, 90), (90, 70), (256, 300)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strides_and_in_place(g, rows, cols, dt):
    buf = rand((rows, cols + 13), 60, 1.0, DT[dt])
    x, x0 = buf[:, 5:5 + cols], buf[:, 5:5 + cols].clone()
    out = torch.full((rows, cols + 6), 7.0, device="cuda", dtype=DT[dt])
    y, ws = out[:, 3:3 + cols], ws_for(g, 1, rows, cols)
    g.newton_schulz([x], [y], ws)
    sync()
    check(y, x0)
    assert torch.all(out[:, :3] == 7) and torch.all(out[:, 3 + cols:] == 7) and torch.equal(x, x0)
    g.newton_schulz([x], [x], ws)
    sync()
    assert torch.equal(x, y)
    assert torch.equal(buf[:, :5], rand((rows, cols + 13), 60, 1.0, DT[dt])[:, :5])


def flat_case(count, rows, cols, n, dt, gap, seed):
    size = rows * cols
    offsets = [3 * gap + i * (size + gap) for i in range(count)][::-1]
    total = max(offsets) + size + 5
    grads = [rand((total,), seed + r, 1e-3, DT[dt]) for r in range(n)]
    return offsets, grads, rand((total,), seed + 50, 0.04), rand((total,), seed + 51, 5e-3)


@pytest.mark.parametrize("count,rows,cols,gap", [(1, 33, 65, 0), (3, 65, 30, 0), (3, 64, 128, 4), (2, 300, 200, 1), (66, 16, 24, 8),
                                                 (12, 768, 256, 0)])
@pytest.mark.parametrize("n,dt", [(1, "f32"), (8, "bf16"), (3, "f32"), (16, "bf16")])
@pytest.mark.parametrize("nesterov", [True, False])
def test_optimizer_step(g, count, rows, cols, gap, n, dt, nesterov):
    offsets, grads, param, buf = flat_case(count, rows, cols, n, dt, gap, 70)
    p0, b0 = param.clone(), buf.clone()
    lr, mu, wd, scale, EXACT = 0.02, 0.95, 0.1, 0.2 * max(rows, cols) ** 0.5, exact_tol(rows, cols)
    half = torch.full_like(param, 9.0, dtype=torch.bfloat16)
    ws = ws_for(g, count, rows, cols)
    g.ddp_bucket_allreduce_muon(grads, offsets, rows, cols, param, buf, ws, lr, mu, wd, update_scale=scale,
                                nesterov=nesterov, param_bf16=half)
    sync()
    rest = torch.ones_like(param, dtype=torch.bool)
    size = rows * cols
    for o in offsets:
        part = slice(o, o + size)
        rest[part] = False
        gw = [x[part].double().view(rows, cols).cpu().numpy() for x in grads]
        tw, bw = O.muon_step(gw, p0[part].double().view(rows, cols).cpu().numpy(),
                             b0[part].double().view(rows, cols).cpu().numpy(), lr, mu, wd, scale, nesterov)
        gm = np.mean(np.abs(gw), axis=0)
        # g: N sums and a product; buf: a product and a sum
        bt = (n + 2) * U * gm + 2 * U * (np.abs(bw) + gm)
        assert np.all(np.abs(buf[part].double().view(rows, cols).cpu().numpy() - bw) <= bt + 1e-40)
        got = param[part].double().view(rows, cols).cpu().numpy()
        step = p0[part].double().view(rows, cols).cpu().numpy() * (1 - lr * wd) - tw
        err = got - tw
        assert np.linalg.norm(err) <= (EXACT + NEAR) * np.linalg.norm(step) + 4 * U * np.linalg.norm(tw)
        assert np.max(np.abs(err)) <= EXACT * np.linalg.norm(step) + 4 * U * np.max(np.abs(tw))
    assert torch.equal(param[rest], p0[rest]) and torch.equal(buf[rest], b0[rest]) and torch.all(half[rest] == 9)
    assert torch.equal(half[~rest], param[~rest].bfloat16())
    # the average's bits are those of the bucket average: with momentum 0 the buffer holds them
    if not nesterov:
        mean, zero = torch.empty_like(param), torch.zeros_like(buf)
        g.ddp_bucket_allreduce_mean(grads, mean)
        g.ddp_bucket_allreduce_muon(grads, offsets, rows, cols, param, zero, ws, lr, 0.0, wd, nesterov=False)
        sync()
        assert torch.equal(zero[~rest], mean[~rest])


def test_steps_of_an_optimizer(g):
    """Three steps follow the oracle's three; the update of each is orthogonal in size."""
    rows, cols, n = 96, 160, 2
    param, buf = rand((rows * cols,), 90, 0.04), torch.zeros(rows * cols, device="cuda")
    ws = ws_for(g, 1, rows, cols)
    tw, bw = param.double().view(rows, cols).cpu().numpy(), np.zeros((rows, cols))
    moved = 0.0
    for k in range(3):
        grads = [rand((rows * cols,), 91 + 10 * k + r, 1e-2) for r in range(n)]
        g.ddp_bucket_allreduce_muon(grads, [0], rows, cols, param, buf, ws, 0.05, 0.9, 0.0)
        t1, bw = O.muon_step([x.double().view(rows, cols).cpu().numpy() for x in grads], tw, bw, 0.05, 0.9, 0.0, 1.0)
        moved, tw = moved + np.linalg.norm(t1 - tw), t1
    sync()
    assert np.linalg.norm(param.double().view(rows, cols).cpu().numpy() - tw) <= (exact_tol(rows, cols) + NEAR) * moved + 8 * U * np.linalg.norm(tw)


@pytest.mark.parametrize("count,rows,cols", [(3, 200, 130), (12, 512, 768)])
def test_other_stream_repeat_and_graph(g, count, rows, cols):
    """The same bits on a side stream, on every repeat and in a graph's replay."""
    xs = [rand((rows, cols), 100 + i, 1.0, torch.bfloat16) for i in range(count)]
    ys = [torch.empty_like(x, dtype=torch.float32) for x in xs]
    offsets, grads, param, buf = flat_case(count, rows, cols, 2, "bf16", 0, 120)
    p0, b0 = param.clone(), buf.clone()
    ws, ws2 = ws_for(g, count, rows, cols), ws_for(g, count, rows, cols)

    def step(stream=None):
        g.newton_schulz(xs, ys, ws, stream=stream)
        g.ddp_bucket_allreduce_muon(grads, offsets, rows, cols, param, buf, ws2, 0.02, 0.95, 0.1, stream=stream)
    step()
    sync()
    first = [t.clone() for t in ys + [param, buf]]
    side = torch.cuda.Stream()
    for how in ("side", "graph"):
        for y in ys:
            y.zero_()
        graph = torch.cuda.CUDAGraph()
        if how == "graph":
            with torch.cuda.graph(graph):
                step()
        param.copy_(p0)
        buf.copy_(b0)
        sync()
        if how == "side":
            step(side)
        else:
            graph.replay()
        sync()
        for t, f in zip(ys + [param, buf], first):
            assert torch.equal(t, f), how


def test_two_calls_at_once(g):
    """Two streams, each with its own workspace: tiles of both want all of an SM's tensor memory."""
    a, b = [rand((700, 900), 130 + i) for i in range(6)], [rand((300, 300), 140 + i) for i in range(8)]
    wa, wb = ws_for(g, 6, 700, 900), ws_for(g, 8, 300, 300)
    ya, yb = [torch.empty_like(x) for x in a], [torch.empty_like(x) for x in b]
    g.newton_schulz(a, ya, wa)
    g.newton_schulz(b, yb, wb)
    sync()
    first = [y.clone() for y in ya + yb]
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        g.newton_schulz(a, ya, wa, stream=s)
        g.newton_schulz(b, yb, wb, stream=t)
    sync()
    for y, f in zip(ya + yb, first):
        assert torch.equal(y, f)


def test_nothing_to_do(g):
    g.newton_schulz([], [], None)
    e = torch.empty(0, 5, device="cuda")
    g.newton_schulz([e], [e.clone()], torch.empty(16, dtype=torch.uint8, device="cuda"))
    p = torch.ones(4, device="cuda")
    g.ddp_bucket_allreduce_muon([p], [], 2, 2, p.clone(), p.clone(), p, 0.1, 0.9, 0.0)
    sync()


def test_large_offsets(g):
    """A matrix that begins past 2^31 elements of the flat buffers."""
    rows, cols, off = 40, 72, (1 << 31) + 8
    total = off + rows * cols
    grads = torch.zeros(total, device="cuda", dtype=torch.bfloat16)
    grads[off:] = rand((rows * cols,), 150, 1e-2, torch.bfloat16)
    param, buf = torch.zeros(total, device="cuda"), torch.zeros(total, device="cuda")
    g.ddp_bucket_allreduce_muon([grads], [off], rows, cols, param, buf, ws_for(g, 1, rows, cols), 1.0, 0.9, 0.0)
    sync()
    check(-param[off:].view(rows, cols), grads[off:].view(rows, cols).float() * 1.9)
    assert torch.all(param[:off] == 0)
