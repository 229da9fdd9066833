"""RMS norm with the residual's addition on the GPU against the fp64 oracle.

Tolerances, with u = 2^-24 (fp32) and b = 2^-8 (one bf16 rounding, with room
for the fp32 value lying on the other side of a rounding boundary):
  a sum over D elements is a chain of at most D/32 per thread and a tree, so
  its terms' absolute sum bounds its error by S = (D/32 + 64)·u of itself;
  rstd carries half of it and a few roundings: S/2 + 4u; an output a few more.
"""
import numpy as np
import pytest
import torch

from gpu_common import load_library, sync
from oracle import distill_oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ROUND = {"f32": U, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def g():
    return load_library()


def rand(shape, seed, std=1.0, dtype=torch.float32):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def stat(D):
    return (D / 32 + 64) * U


def check_forward(x, r, gamma, eps, h, y, rstd):
    D = x.shape[1]
    hw, rw, yw = O.rmsnorm(f64(x), f64(r), f64(gamma), eps)
    tol = stat(D) / 2 + 4 * U
    if rstd is not None:
        assert np.all(np.abs(f64(rstd) - rw) <= tol * rw)
    if h is not None:
        rnd = ROUND["bf16" if h.dtype == torch.bfloat16 else "f32"]
        assert np.all(np.abs(f64(h) - hw) <= rnd * np.abs(hw) + 1e-40)
    # x + residual is rounded once in fp32: an absolute error of u·|h|; the rest is relative
    rnd = ROUND["bf16" if y.dtype == torch.bfloat16 else "f32"]
    assert np.all(np.abs(f64(y) - yw) <= (tol + 8 * U + rnd) * np.abs(yw) + 1e-40)


# one row and many; widths around warps, vectors, CTAs; odd ones; wide ones
SHAPES = [(1, 1), (3, 7), (1, 768), (5, 64), (33, 255), (2, 1000), (7, 1024), (301, 768), (64, 2051), (9, 4096),
          (3, 8200), (2, 16384), (2, 33001), (1, 70000)]


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
def test_forward(g, rows, D, dt, out):
    x, r = rand((rows, D), 1, 1.0, DT[dt]), rand((rows, D), 2, 2.0, DT[dt])
    gamma = 1 + rand((D,), 3, 0.1)
    y, h = torch.full((rows, D), float("nan"), device="cuda", dtype=DT[out]), torch.empty_like(x)
    rstd = torch.empty(rows, device="cuda")
    g.rmsnorm_forward(x, gamma, y, 1e-5, residual=r, h_out=h, rstd_out=rstd)
    sync()
    check_forward(x, r, gamma, 1e-5, h, y, rstd)
    g.rmsnorm_forward(x, None, y, 1e-5)           # no residual, no gamma, nothing kept
    sync()
    check_forward(x, None, None, 1e-5, None, y, None)


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_forward_q8(g, rows, D, dt):
    x, r = rand((rows, D), 4, 1.0, DT[dt]), rand((rows, D), 5, 2.0, DT[dt])
    gamma = 1 + rand((D,), 6, 0.1)
    q, scale = torch.full((rows, D), 99, device="cuda", dtype=torch.int8), torch.empty(rows, device="cuda")
    h, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    g.rmsnorm_forward_q8(x, gamma, q, scale, 1e-5, residual=r, h_out=h, rstd_out=rstd)
    sync()
    check_q8(x, r, gamma, 1e-5, q, scale)
    hw, rw, _ = O.rmsnorm(f64(x), f64(r), f64(gamma), 1e-5)
    assert np.all(np.abs(f64(h) - hw) <= ROUND[dt] * np.abs(hw) + 1e-40)
    assert np.all(np.abs(f64(rstd) - rw) <= (stat(D) / 2 + 4 * U) * rw)


def check_q8(x, r, gamma, eps, q, scale):
    D = x.shape[1]
    _, _, yw = O.rmsnorm(f64(x), f64(r), f64(gamma), eps)
    sw = O.rmsnorm_q8_scale(yw)
    tol = stat(D) / 2 + 10 * U
    assert np.all(np.abs(f64(scale) - sw) <= tol * sw)
    # q is the nearest integer of a quotient of at most 127 that is off by tol (and 4 roundings) of itself
    off = np.abs(f64(q) - yw / np.where(sw > 0, sw, 1.0)[:, None])
    assert np.all(off <= 0.5 + 127 * (2 * tol + 4 * U))
    assert np.all(np.abs(f64(q)).max(1)[sw > 0] == 127)


@pytest.mark.parametrize("rows,D", SHAPES + [(1300, 96), (2500, 16), (700, 1280)])
@pytest.mark.parametrize("dt,dyt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
def test_backward(g, rows, D, dt, dyt):
    h, dy, dh = rand((rows, D), 7, 2.0, DT[dt]), rand((rows, D), 8, 0.5, DT[dyt]), rand((rows, D), 9, 0.5, DT[dt])
    gamma = 1 + rand((D,), 10, 0.1)
    rstd = torch.rsqrt((h.double() ** 2).mean(1) + 1e-5).float()
    for use_dh, gm in ((True, gamma), (False, None)):
        dx, dgamma = torch.full_like(h, float("nan")), torch.full((D,), float("nan"), device="cuda")
        ws = torch.empty(g.rmsnorm_backward_workspace_bytes(rows, D), dtype=torch.uint8, device="cuda")
        ws.fill_(255)
        g.rmsnorm_backward(dy, h, rstd, gm, dx, dgamma, ws, dh=dh if use_dh else None)
        sync()
        check_backward(dy, h, rstd, gm, dh if use_dh else None, dx, dgamma)
        only = torch.empty_like(dx)
        g.rmsnorm_backward(dy, h, rstd, gm, only, dh=dh if use_dh else None)      # gamma frozen
        sync()
        assert torch.equal(only, dx)


@pytest.mark.parametrize("rows,D,ld,at", [
    (1500, 4099, 4099, 0), (5000, 515, 515, 0), (5000, 255, 255, 0), (700, 8195, 8195, 0),      # odd rows, packed
    (1500, 2051, 2056, 3), (1500, 2048, 2051, 0), (5000, 512, 515, 0), (5000, 500, 509, 5), (2500, 16, 17, 0)])
@pytest.mark.parametrize("dt,dyt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
def test_backward_of_many_unaligned_rows(g, rows, D, ld, at, dt, dyt):
    """Several rows to a CTA or warp, off the 16-byte boundaries, all matrices alike: odd widths, odd pitches with even
    widths, odd bases with aligned pitches."""
    def cut(seed, std, t):
        return rand((rows * ld + 16,), seed, std, DT[t])[at:at + rows * ld].view(rows, ld)[:, :D]
    h, dy, dh = cut(80, 2.0, dt), cut(81, 0.5, dyt), cut(82, 0.5, dt)
    gamma = 1 + rand((D,), 83, 0.1)
    rstd = torch.rsqrt((h.double() ** 2).mean(1) + 1e-5).float()
    flat = torch.full((rows * ld + 16,), 3.0, device="cuda", dtype=DT[dt])
    dx, dgamma = flat[at:at + rows * ld].view(rows, ld)[:, :D], torch.full((D,), float("nan"), device="cuda")
    ws = torch.empty(g.rmsnorm_backward_workspace_bytes(rows, D), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    g.rmsnorm_backward(dy, h, rstd, gamma, dx, dgamma, ws, dh=dh)
    sync()
    check_backward(dy, h, rstd, gamma, dh, dx, dgamma)
    assert torch.all(flat[at:at + rows * ld].view(rows, ld)[:, D:] == 3)
    assert torch.all(flat[:at] == 3) and torch.all(flat[at + rows * ld:] == 3)


def check_backward(dy, h, rstd, gamma, dh, dx, dgamma):
    rows, D = h.shape
    dyw, n = f64(dy), f64(h) * f64(rstd)[:, None]
    dn = dyw if gamma is None else dyw * f64(gamma)
    dxw, dgw = O.rmsnorm_grad(dyw, f64(h), f64(rstd), f64(gamma), f64(dh))
    rs = f64(rstd)[:, None]
    # each product and difference rounds its terms; the mean's error is S of its absolute terms
    c_err = (stat(D) + 8 * U) * np.mean(np.abs(dn * n), axis=1, keepdims=True)
    terms = np.abs(rs * dn) + np.abs(rs * n * np.mean(dn * n, axis=1, keepdims=True)) + (0 if dh is None else np.abs(f64(dh)))
    rnd = ROUND["bf16" if dx.dtype == torch.bfloat16 else "f32"]
    assert np.all(np.abs(f64(dx) - dxw) <= 8 * U * terms + rs * np.abs(n) * c_err + rnd * np.abs(dxw) + 1e-40)
    # dγ: a sum over the rows in any grouping, each term of three roundings
    assert np.all(np.abs(f64(dgamma) - dgw) <= (rows + 8) * U * np.sum(np.abs(dyw * n), axis=0) + 1e-40)


@pytest.mark.parametrize("D", [96, 515])
def test_backward_against_differences(g, D):
    """Central differences of Σ w·y over the forward kernel's own fp32 outputs along random directions."""
    rows, e = 6, 2.0 ** -8
    x, w, gamma = rand((rows, D), 11), rand((rows, D), 12), 1 + rand((D,), 13, 0.2)

    def f(x, gamma):
        y = torch.empty_like(x)
        rstd = torch.empty(rows, device="cuda")
        g.rmsnorm_forward(x, gamma, y, 1e-5, rstd_out=rstd)
        return float((y.double() * w.double()).sum()), rstd
    _, rstd = f(x, gamma)
    dx, dgamma = torch.empty_like(x), torch.empty(D, device="cuda")
    ws = torch.empty(g.rmsnorm_backward_workspace_bytes(rows, D), dtype=torch.uint8, device="cuda")
    g.rmsnorm_backward(w, x, rstd, gamma, dx, dgamma, ws)
    for seed in range(4):
        d, dg = rand((rows, D), 20 + seed), rand((D,), 30 + seed)
        num = (f(x + e * d, gamma)[0] - f(x - e * d, gamma)[0]) / (2 * e)
        # rounding: outputs of size ~1 off by ~10u each, n of them added in quadrature, over 2e;
        # truncation: e²/6 of the third derivative, whose size is that of the terms' sum
        size = float((w.double().abs() * (1 + d.double().abs()) ** 3).sum())
        tol = 10 * U * (rows * D) ** 0.5 * 4 / e + e * e * size / (rows * D) ** 0.5
        assert abs(num - float((dx.double() * d.double()).sum())) <= tol
        num = (f(x, gamma + e * dg)[0] - f(x, gamma - e * dg)[0]) / (2 * e)   # linear in gamma
        assert abs(num - float((dgamma.double() * dg.double()).sum())) <= 10 * U * (rows * D) ** 0.5 * 8 / e


@pytest.mark.parametrize("D", [40, 768, 771, 5000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strides_offsets_and_in_place(g, D, dt):
    """Column slices at odd offsets of wider buffers; h on the residual and y on x."""
    rows, wide = 11, 2 * D + 13
    buf = rand((rows, wide), 40, 1.0, DT[dt])
    x, r = buf[:, 3:3 + D], buf[:, D + 7:2 * D + 7]
    x0, r0 = x.clone(), r.clone()
    gamma = 1 + rand((D + 1,), 41, 0.1)[1:]
    out = torch.full((rows, D + 5), 7.0, device="cuda", dtype=DT[dt])
    h, y, rstd = torch.empty_like(x0), out[:, 2:2 + D], torch.empty(rows, device="cuda")
    g.rmsnorm_forward(x, gamma, y, 1e-5, residual=r, h_out=h, rstd_out=rstd)
    sync()
    check_forward(x0, r0, gamma, 1e-5, h, y, rstd)
    assert torch.all(out[:, :2] == 7) and torch.all(out[:, 2 + D:] == 7)
    # both in place, in one buffer: the bits of a call whose outputs lie like x and residual (other layouts may sum
    # in another order)
    other = torch.empty_like(buf)
    y0, h0 = other[:, 3:3 + D], other[:, D + 7:2 * D + 7]
    g.rmsnorm_forward(x, gamma, y0, 1e-5, residual=r, h_out=h0)
    g.rmsnorm_forward(x, gamma, x, 1e-5, residual=r, h_out=r)
    sync()
    assert torch.equal(x, y0) and torch.equal(r, h0)
    check_forward(x0, r0, gamma, 1e-5, r, x, None)
    rest = torch.ones(wide, dtype=torch.bool, device="cuda")
    rest[3:3 + D] = False
    rest[D + 7:2 * D + 7] = False
    assert torch.equal(buf[:, rest], rand((rows, wide), 40, 1.0, DT[dt])[:, rest])
    qb, scale = torch.full((rows, D + 9), 55, device="cuda", dtype=torch.int8), torch.empty(rows, device="cuda")
    g.rmsnorm_forward_q8(x0, gamma, qb[:, 5:5 + D], scale, 1e-5, residual=r0)
    sync()
    check_q8(x0, r0, gamma, 1e-5, qb[:, 5:5 + D], scale)
    assert torch.all(qb[:, :5] == 55) and torch.all(qb[:, 5 + D:] == 55)
    # backward: strided inputs, dx on dy
    dyb = rand((rows, wide), 42, 0.5, DT[dt])
    dy, dh = dyb[:, 1:1 + D], dyb[:, D + 2:2 * D + 2]
    dy0, dh0 = dy.clone(), dh.clone()
    dgamma = torch.empty(D, device="cuda")
    ws = torch.empty(g.rmsnorm_backward_workspace_bytes(rows, D), dtype=torch.uint8, device="cuda")
    g.rmsnorm_backward(dy, h, rstd, gamma, dy, dgamma, ws, dh=dh)
    sync()
    check_backward(dy0, h, rstd, gamma, dh0, dy, dgamma)
    assert torch.equal(dh, dh0)


@pytest.mark.parametrize("D", [16, 100, 4096])
def test_special_rows(g, D):
    """Zeros, subnormals, infinities and NaN stay in their row; zeros give zeros for any eps > 0."""
    x = rand((6, D), 50)
    x[1] = 0
    x[2, D // 2] = float("nan")
    x[3, 0] = float("inf")
    x[4] = 1e-30
    y, rstd = torch.empty_like(x), torch.empty(6, device="cuda")
    g.rmsnorm_forward(x, None, y, 1e-6, rstd_out=rstd)
    q, scale = torch.full((6, D), 77, device="cuda", dtype=torch.int8), torch.empty(6, device="cuda")
    g.rmsnorm_forward_q8(x, None, q, scale, 1e-6)
    sync()
    keep = [0, 1, 4, 5]
    check_forward(x[keep], None, None, 1e-6, None, y[keep], rstd[keep])
    assert torch.all(y[1] == 0) and torch.all(q[1] == 0) and scale[1] == 0
    assert torch.isnan(y[2]).all()
    assert not torch.isfinite(scale[2]) and not torch.isfinite(scale[3]) and torch.all(q[2:4] == 0)
    check_q8(x[[0, 5]], None, None, 1e-6, q[[0, 5]], scale[[0, 5]])


@pytest.mark.parametrize("D", [48, 515, 40000])
def test_q8_of_tiny_and_huge_rows(g, D):
    """Rows whose scale is far from 1: 127 / max would overflow, or the maximum is near the type's end."""
    x = rand((5, D), 51)
    x[1] *= 1e-36
    x[2] *= 1e-33
    x[3] *= 1e16
    gamma = torch.ones(D, device="cuda")
    q, scale = torch.full((5, D), 77, device="cuda", dtype=torch.int8), torch.empty(5, device="cuda")
    g.rmsnorm_forward_q8(x, gamma, q, scale, 1.0)
    sync()
    check_q8(x, None, gamma, 1.0, q, scale)


def test_empty(g):
    x = torch.empty(0, 64, device="cuda")
    g.rmsnorm_forward(x, None, torch.empty_like(x))
    dgamma = torch.full((64,), 5.0, device="cuda")
    ws = torch.empty(g.rmsnorm_backward_workspace_bytes(0, 64), dtype=torch.uint8, device="cuda")
    g.rmsnorm_backward(x, x, torch.empty(0, device="cuda"), None, torch.empty_like(x), dgamma, ws)
    sync()
    assert torch.all(dgamma == 0)


@pytest.mark.parametrize("D", [768, 4099])
def test_other_stream_repeat_and_graph(g, D):
    """The same bits on a side stream, on every repeat and in a graph's replay."""
    rows = 700
    x, r, gamma = rand((rows, D), 60, 1.0, torch.bfloat16), rand((rows, D), 61, 1.0, torch.bfloat16), rand((D,), 62)
    bufs = [torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty_like(x),
            torch.empty(D, device="cuda"), torch.empty_like(x, dtype=torch.int8), torch.empty(rows, device="cuda")]
    ws = torch.empty(g.rmsnorm_backward_workspace_bytes(rows, D), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        y, h, rstd, dx, dgamma, q, scale = bufs
        g.rmsnorm_forward(x, gamma, y, 1e-5, residual=r, h_out=h, rstd_out=rstd, stream=stream)
        g.rmsnorm_forward_q8(x, gamma, q, scale, 1e-5, residual=r, stream=stream)
        g.rmsnorm_backward(y, h, rstd, gamma, dx, dgamma, ws, dh=r, stream=stream)
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


def test_offsets_past_32_bits(g):
    D, rows = 8192, (1 << 31) // 8192 + 3
    x = torch.zeros(rows, D, device="cuda", dtype=torch.bfloat16)
    x[-2:] = rand((2, D), 70, 1.0, torch.bfloat16)
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    g.rmsnorm_forward(x, None, y, 1e-5, rstd_out=rstd)
    sync()
    check_forward(x[-2:], None, None, 1e-5, None, y[-2:], rstd[-2:])
    dgamma = torch.empty(D, device="cuda")
    ws = torch.empty(g.rmsnorm_backward_workspace_bytes(rows, D), dtype=torch.uint8, device="cuda")
    dx = y
    dy = y[-2:].clone()
    g.rmsnorm_backward(y, x, rstd, None, dx, dgamma, ws)
    sync()
    check_backward(dy, x[-2:], rstd[-2:], None, None, dx[-2:], dgamma)
