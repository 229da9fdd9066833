"""Layer norm with the residual's addition on the GPU against the fp64 oracle.

Tolerances, with u = 2^-24 (fp32) and 2^-8 for one bf16 rounding:
  a sum over D elements is a chain of at most D/32 per thread and a tree, so
  its terms' absolute sum bounds its error by S = (D/32 + 64)·u of itself.
  mean: S·mean|h| and the roundings of h = x + residual, u·|h| each.
  h − mean: what the mean is off by (E = S·mean|h| + 2u·max|h|), and its own
  rounding.  The variance about a mean that is off by E is off by E² and, for
  each element's own rounding, by 2·E·sigma at most; rstd by half of that,
  relative to the variance, and by S/2 and a few roundings.
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


def rand(shape, seed, std=1.0, dtype=torch.float32, mean=0.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std + mean).to(dtype)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def stat(D):
    return (D / 32 + 64) * U


def half(t):
    return U if t.dtype == torch.float32 else 2.0 ** -8


def check_forward(x, r, gamma, beta, eps, h, y, mean, rstd):
    D = x.shape[1]
    hw, mw, rw, yw = O.layernorm(f64(x), f64(r), f64(gamma), f64(beta), eps)
    E = stat(D) * np.mean(np.abs(hw), axis=1) + 2 * U * np.max(np.abs(hw), axis=1)
    rel = stat(D) / 2 + 6 * U + E * rw + (E * rw) ** 2
    if mean is not None:
        assert np.all(np.abs(f64(mean) - mw) <= E + 1e-40)
    if rstd is not None:
        assert np.all(np.abs(f64(rstd) - rw) <= rel * rw)
    if h is not None:
        assert np.all(np.abs(f64(h) - hw) <= (half(h) + U) * np.abs(hw) + 1e-40)
    gw = np.ones(D) if gamma is None else np.abs(f64(gamma))
    bw = np.zeros(D) if beta is None else np.abs(f64(beta))
    n = np.abs(hw - mw[:, None]) * rw[:, None]
    off = gw * (E * rw)[:, None] * 2 + gw * n * (rel[:, None] + 4 * U) + 2 * U * bw
    assert np.all(np.abs(f64(y) - yw) <= off * (1 + half(y)) + half(y) * np.abs(yw) + 1e-40)


# one row and many; widths around warps, vectors, CTAs; odd ones; wide ones
SHAPES = [(1, 1), (3, 7), (1, 768), (5, 64), (33, 255), (2, 1000), (7, 1024), (301, 768), (64, 2051), (9, 4096),
          (3, 8200), (2, 16384), (2, 33001), (1, 70000), (700, 1280)]


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
def test_forward(g, rows, D, dt, out):
    x, r = rand((rows, D), 1, 1.0, DT[dt], 0.5), rand((rows, D), 2, 2.0, DT[dt])
    gamma, beta = 1 + rand((D,), 3, 0.1), rand((D,), 4, 0.3)
    y, h = torch.full((rows, D), float("nan"), device="cuda", dtype=DT[out]), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    g.layernorm_forward(x, gamma, beta, y, 1e-5, residual=r, h_out=h, mean_out=mean, rstd_out=rstd)
    sync()
    check_forward(x, r, gamma, beta, 1e-5, h, y, mean, rstd)
    g.layernorm_forward(x, None, None, y, 1e-5)           # nothing that is optional
    sync()
    check_forward(x, None, None, None, 1e-5, None, y, None, None)


@pytest.mark.parametrize("D", [64, 771, 4096, 20000])
def test_rows_far_from_zero(g, D):
    """mean² is 1e6 times the variance: fp32 sums of squares would keep two digits of it."""
    x = rand((5, D), 5, 1.0, mean=1000.0)
    y, mean, rstd = torch.empty_like(x), torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    g.layernorm_forward(x, None, None, y, 1e-5, mean_out=mean, rstd_out=rstd)
    sync()
    check_forward(x, None, None, None, 1e-5, None, y, mean, rstd)
    _, _, rw, _ = O.layernorm(f64(x), None, None, None, 1e-5)
    assert np.all(np.abs(f64(rstd) / rw - 1) <= 1e-3)


def check_backward(dy, h, mean, rstd, gamma, dh, dx, dgamma, dbeta):
    rows, D = h.shape
    rs = f64(rstd)[:, None]
    dyw, n = f64(dy), (f64(h) - f64(mean)[:, None]) * rs
    dn = dyw if gamma is None else dyw * f64(gamma)
    dxw, dgw, dbw = O.layernorm_grad(dyw, f64(h), f64(mean), f64(rstd), f64(gamma), f64(dh))
    # each product and difference rounds its terms; a mean's error is S of its absolute terms
    c1, c2 = (np.mean(np.abs(v), axis=1, keepdims=True) for v in (dn, dn * n))
    off = rs * (stat(D) + 8 * U) * (c1 + np.abs(n) * c2)
    terms = np.abs(rs * dn) + np.abs(rs) * (c1 + np.abs(n) * c2) + (0 if dh is None else np.abs(f64(dh)))
    assert np.all(np.abs(f64(dx) - dxw) <= 8 * U * terms + off + half(dx) * np.abs(dxw) + 1e-40)
    # sums over the rows in any grouping, each term of dγ of four roundings
    if dgamma is not None:
        assert np.all(np.abs(f64(dgamma) - dgw) <= (rows + 8) * U * np.sum(np.abs(dyw * n), axis=0) + 1e-40)
    if dbeta is not None:
        assert np.all(np.abs(f64(dbeta) - dbw) <= (rows + 8) * U * np.sum(np.abs(dyw), axis=0) + 1e-40)


MANY = [(8000, 64), (7500, 130), (7400, 200), (7400, 392), (7400, 515), (7400, 771), (7300, 1000), (7300, 1021)]   # rows after rows per warp


@pytest.mark.parametrize("rows,D", SHAPES + [(1300, 96), (2500, 16), (400, 9000)] + MANY)
@pytest.mark.parametrize("dt,dyt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
def test_backward(g, rows, D, dt, dyt):
    h, dy, dh = rand((rows, D), 7, 2.0, DT[dt], 0.7), rand((rows, D), 8, 0.5, DT[dyt]), rand((rows, D), 9, 0.5, DT[dt])
    gamma = 1 + rand((D,), 10, 0.1)
    mean = h.double().mean(1).float()
    rstd = torch.rsqrt(((h.double() - mean.double()[:, None]) ** 2).mean(1) + 1e-5).float()
    nan = float("nan")
    for use_dh, gm in ((True, gamma), (False, None)):
        dx = torch.full_like(h, nan)
        dgamma, dbeta = torch.full((D,), nan, device="cuda"), torch.full((D,), nan, device="cuda")
        ws = torch.empty(g.layernorm_backward_workspace_bytes(rows, D), dtype=torch.uint8, device="cuda")
        ws.fill_(255)
        d = dh if use_dh else None
        g.layernorm_backward(dy, h, mean, rstd, gm, dx, dgamma, dbeta, ws, dh=d)
        sync()
        check_backward(dy, h, mean, rstd, gm, d, dx, dgamma, dbeta)
        only = torch.empty_like(dx)
        g.layernorm_backward(dy, h, mean, rstd, gm, only, dh=d)                   # no sums over the rows
        one = torch.full((D,), nan, device="cuda")
        g.layernorm_backward(dy, h, mean, rstd, gm, only, None, one, ws, dh=d)    # one of the two
        sync()
        assert torch.equal(only, dx) and torch.equal(one, dbeta)


@pytest.mark.parametrize("D", [64, 255, 512, 768, 1024])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_backward_in_place_of_many_rows(g, D, dt):
    """dx on dy, h or dh: the rows that are fetched ahead are still what they were."""
    rows = 7400
    h, dy, dh = (rand((rows, D), i, 1.0, DT[dt]) for i in (30, 31, 32))
    mean, rstd, gamma = rand((rows,), 33, 0.1), 1 + rand((rows,), 34, 0.1).abs(), 1 + rand((D,), 35, 0.1)
    ws = torch.empty(g.layernorm_backward_workspace_bytes(rows, D), dtype=torch.uint8, device="cuda")
    want, dg, db = torch.empty_like(h), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    g.layernorm_backward(dy, h, mean, rstd, gamma, want, dg, db, ws, dh=dh)
    for on in range(3):
        t = [dy.clone(), h.clone(), dh.clone()]
        dg2, db2 = torch.empty_like(dg), torch.empty_like(db)
        g.layernorm_backward(t[0], t[1], mean, rstd, gamma, t[on], dg2, db2, ws, dh=t[2])
        sync()
        assert torch.equal(t[on], want) and torch.equal(dg2, dg) and torch.equal(db2, db), on


@pytest.mark.parametrize("D", [96, 515])
def test_backward_against_differences(g, D):
    """Central differences of Σ w·y over the forward kernel's own fp32 outputs along random directions."""
    rows, e = 6, 2.0 ** -8
    x, w, gamma, beta = rand((rows, D), 11), rand((rows, D), 12), 1 + rand((D,), 13, 0.2), rand((D,), 14)

    def f(x, gamma, beta):
        y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        g.layernorm_forward(x, gamma, beta, y, 1e-5, mean_out=mean, rstd_out=rstd)
        return float((y.double() * w.double()).sum()), mean, rstd
    _, mean, rstd = f(x, gamma, beta)
    dx, dgamma, dbeta = torch.empty_like(x), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    ws = torch.empty(g.layernorm_backward_workspace_bytes(rows, D), dtype=torch.uint8, device="cuda")
    g.layernorm_backward(w, x, mean, rstd, gamma, dx, dgamma, dbeta, ws)
    for seed in range(4):
        d, dg = rand((rows, D), 20 + seed), rand((D,), 30 + seed)
        num = (f(x + e * d, gamma, beta)[0] - f(x - e * d, gamma, beta)[0]) / (2 * e)
        # rounding: outputs of size up to 5 off by ~10u each, rows·D of them added in quadrature, over 2e;
        # truncation: e²/6 of the third derivative, whose size is that of the terms' sum
        size = float((w.double().abs() * (1 + d.double().abs()) ** 3).sum())
        tol = 10 * U * (rows * D) ** 0.5 * 8 / e + e * e * size / (rows * D) ** 0.5
        assert abs(num - float((dx.double() * d.double()).sum())) <= tol
        # linear in gamma and beta
        for i, got in ((1, dgamma), (2, dbeta)):
            up, down = [x, gamma, beta], [x, gamma, beta]
            up[i], down[i] = up[i] + e * dg, down[i] - e * dg
            num = (f(*up)[0] - f(*down)[0]) / (2 * e)
            assert abs(num - float((got.double() * dg.double()).sum())) <= 10 * U * (rows * D) ** 0.5 * 16 / e


@pytest.mark.parametrize("D", [40, 768, 771, 5000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strides_offsets_and_in_place(g, D, dt):
    """Column slices at odd offsets of wider buffers; h on the residual and y on x; dx on dy, h and dh."""
    rows, wide = 11, 2 * D + 13
    buf = rand((rows, wide), 40, 1.0, DT[dt])
    x, r = buf[:, 3:3 + D], buf[:, D + 7:2 * D + 7]
    x0, r0 = x.clone(), r.clone()
    gamma, beta = 1 + rand((D + 1,), 41, 0.1)[1:], rand((D + 3,), 43, 0.1)[3:]
    out = torch.full((rows, D + 5), 7.0, device="cuda", dtype=DT[dt])
    h, y = torch.empty_like(x0), out[:, 2:2 + D]
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    g.layernorm_forward(x, gamma, beta, y, 1e-5, residual=r, h_out=h, mean_out=mean, rstd_out=rstd)
    sync()
    check_forward(x0, r0, gamma, beta, 1e-5, h, y, mean, rstd)
    assert torch.all(out[:, :2] == 7) and torch.all(out[:, 2 + D:] == 7)
    g.layernorm_forward(x, gamma, beta, x, 1e-5, residual=r, h_out=r)
    sync()
    check_forward(x0, r0, gamma, beta, 1e-5, r, x, None, None)
    rest = torch.ones(wide, dtype=torch.bool, device="cuda")
    rest[3:3 + D] = False
    rest[D + 7:2 * D + 7] = False
    assert torch.equal(buf[:, rest], rand((rows, wide), 40, 1.0, DT[dt])[:, rest])
    ws = torch.empty(g.layernorm_backward_workspace_bytes(rows, D), dtype=torch.uint8, device="cuda")
    for place in range(3):
        dyb = rand((rows, wide), 42, 0.5, DT[dt])
        ins = [dyb[:, 1:1 + D], h.clone(), dyb[:, D + 2:2 * D + 2]]
        dy0, h0, dh0 = (t.clone() for t in ins)
        dgamma, dbeta = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
        g.layernorm_backward(ins[0], ins[1], mean, rstd, gamma, ins[place], dgamma, dbeta, ws, dh=ins[2])
        sync()
        check_backward(dy0, h0, mean, rstd, gamma, dh0, ins[place], dgamma, dbeta)
        for i, old in enumerate((dy0, h0, dh0)):
            assert i == place or torch.equal(ins[i], old)


@pytest.mark.parametrize("D", [16, 100, 4096])
def test_special_rows(g, D):
    """Equal values, subnormals, infinities and NaN stay in their row."""
    x = rand((6, D), 50)
    x[1] = 3.0
    x[2, D // 2] = float("nan")
    x[3, 0] = float("inf")
    x[4] = 1e-40
    y, mean, rstd, beta = torch.empty_like(x), torch.empty(6, device="cuda"), torch.empty(6, device="cuda"), rand((D,), 51)
    g.layernorm_forward(x, None, beta, y, 1e-6, mean_out=mean, rstd_out=rstd)
    sync()
    keep = [0, 1, 4, 5]
    check_forward(x[keep], None, None, beta, 1e-6, None, y[keep], mean[keep], rstd[keep])
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()


def test_empty(g):
    x = torch.empty(0, 64, device="cuda")
    g.layernorm_forward(x, None, None, torch.empty_like(x))
    dgamma, dbeta = torch.full((64,), 5.0, device="cuda"), torch.full((64,), 5.0, device="cuda")
    ws = torch.empty(g.layernorm_backward_workspace_bytes(0, 64), dtype=torch.uint8, device="cuda")
    none = torch.empty(0, device="cuda")
    g.layernorm_backward(x, x, none, none, None, torch.empty_like(x), dgamma, dbeta, ws)
    sync()
    assert torch.all(dgamma == 0) and torch.all(dbeta == 0)


@pytest.mark.parametrize("D", [768, 4099])
def test_other_stream_repeat_and_graph(g, D):
    """The same bits on a side stream, on every repeat and in a graph's replay."""
    rows = 700
    x, r, gamma = rand((rows, D), 60, 1.0, torch.bfloat16), rand((rows, D), 61, 1.0, torch.bfloat16), rand((D,), 62)
    bufs = [torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda"),
            torch.empty(rows, device="cuda"), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")]
    ws = torch.empty(g.layernorm_backward_workspace_bytes(rows, D), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        y, h, dx, mean, rstd, dgamma, dbeta = bufs
        g.layernorm_forward(x, gamma, gamma, y, 1e-5, residual=r, h_out=h, mean_out=mean, rstd_out=rstd, stream=stream)
        g.layernorm_backward(y, h, mean, rstd, gamma, dx, dgamma, dbeta, ws, dh=r, stream=stream)
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
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    g.layernorm_forward(x, None, None, y, 1e-5, mean_out=mean, rstd_out=rstd)
    sync()
    check_forward(x[-2:], None, None, None, 1e-5, None, y[-2:], mean[-2:], rstd[-2:])
    dgamma, dbeta = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    ws = torch.empty(g.layernorm_backward_workspace_bytes(rows, D), dtype=torch.uint8, device="cuda")
    dy = y[-2:].clone()
    g.layernorm_backward(y, x, mean, rstd, None, y, dgamma, dbeta, ws)
    sync()
    check_backward(dy, x[-2:], mean[-2:], rstd[-2:], None, None, y[-2:], dgamma, dbeta)
