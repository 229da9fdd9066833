"""Loss on a teacher's top logits and its gradient on the GPU against the fp64
oracle.

Tolerances, u = 2^-24: an exponent is a product of at most R = (max|z| +
max|teacher|)/τ rounded a few times, an exponential adds 2^-21, a sum over V
positive terms is a chain of at most V/128 and a tree, so probabilities are
off by E = (V/128 + 64)·u + 16·u·R + 2^-20 of themselves and log-probabilities
by E; bf16 rounds the gradient once (2^-8, as in the norm's tests)."""
import numpy as np
import pytest
import torch

from gpu_common import load_library, sync
from oracle import distill_oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def g():
    return load_library()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(T, V, k, dt="bf16", tdt="f32", it=torch.int64, seed=1, std=2.5):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    z = (torch.randn(T, V, generator=gen, device="cuda") * std).to(DT[dt])
    t = (torch.randn(T, k, generator=gen, device="cuda") * 2 + 3).to(DT[tdt])
    index = torch.argsort(torch.rand(T, V, generator=gen, device="cuda"), dim=1)[:, :k]
    index = torch.cat([index, torch.full((T, max(0, k - V)), -1, device="cuda")], 1).to(it).contiguous()
    up = torch.randn(T, generator=gen, device="cuda")
    return z, index, t, up


def all_three(g, z, index, t, up, tau):
    """(loss, lse, gradient): by one call, and by two, which have to agree."""
    T = z.shape[0]
    nan = lambda *s, **k: torch.full(s, float("nan"), device="cuda", **k)  # noqa: E731
    loss, lse, dz = nan(T), nan(T), nan(*z.shape, dtype=z.dtype)
    g.distill_topk_forward_backward(z, index, t, up, loss, lse, dz, temperature=tau)
    loss2, lse2, dz2 = nan(T), nan(T), nan(*z.shape, dtype=z.dtype)
    g.distill_topk_forward(z, index, t, loss2, lse2, temperature=tau)
    g.distill_topk_backward(z, index, t, lse2, up, dz2, temperature=tau)
    sync()
    return (loss, lse, dz), (loss2, lse2, dz2)


def check(z, index, t, up, tau, loss, lse, dz, rows=None):
    if rows is not None:
        z, index, t, up, loss, lse, dz = (None if v is None else v[rows] for v in (z, index, t, up, loss, lse, dz))
    T, V = z.shape
    zw, tw, iw, upw = f64(z), f64(t), index.cpu().numpy(), f64(up)
    fin = lambda a: np.max(np.abs(a[np.isfinite(a)]), initial=0.0)  # noqa: E731
    R = (fin(zw) + fin(tw)) / tau
    E = (V / 128 + 64) * U + 16 * U * R + 2.0 ** -20
    lw, sw, dw = O.distill_topk(zw, iw, tw, tau, upw)
    if loss is not None:
        got = f64(loss)
        ok = np.isfinite(lw)
        assert np.array_equal(got[~ok], lw[~ok])
        # |ln p − ln q| of the entries is at most 2R + ln V; p is off by 2E of itself
        tol = tau * tau * (E + 2 * E * (2 * R + np.log(V + 1.0)))
        assert np.all(np.abs(got[ok] - lw[ok]) <= tol)
    if lse is not None:
        assert np.all(np.abs(f64(lse) - sw) <= E + 4 * U * np.abs(sw))
    if dz is not None:
        gw = np.abs(np.ones(T) if up is None else upw)[:, None] * tau
        # the terms are g·q and g·p: their size is at most that of the gradient and of p
        psum = np.zeros((T, V))
        for r in range(T):
            ok = (iw[r] >= 0) & (iw[r] < V)
            e = tw[r][ok] / tau
            if e.size and np.max(e) > -np.inf:
                p = np.exp(e - np.max(e))
                np.add.at(psum[r], iw[r][ok], p / p.sum())
        q = np.exp(zw / tau - sw[:, None])
        rnd = 2.0 ** -8 if dz.dtype == torch.bfloat16 else U
        # 1e-37: probabilities below fp32's normal range may be flushed
        assert np.all(np.abs(f64(dz) - dw) <= gw * 2 * E * (q + psum) + rnd * np.abs(dw) + 1e-37 * (1 + gw))


# tiny; odd vocabularies; one entry; as many entries as words; few tokens of a large vocabulary; many tokens
SHAPES = [(1, 1, 1), (3, 7, 7), (2, 33, 0), (5, 129, 4), (1, 50257, 50), (4, 4096, 64), (65, 1001, 17), (3, 32003, 256),
          (700, 515, 9), (2, 151936, 1024), (2, 300, 1024), (9, 70001, 33)]


@pytest.mark.parametrize("T,V,k", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_loss_and_gradient(g, T, V, k, dt):
    for tau, tdt, it in ((1.0, "f32", torch.int64), (2.5, "bf16", torch.int32)):
        z, index, t, up = make(T, V, k, dt, tdt, it)
        one, two = all_three(g, z, index, t, up, tau)
        rows = slice(0, 40)
        check(z, index, t, up, tau, *one, rows=rows)
        check(z, index, t, up, tau, *two, rows=rows)


@pytest.mark.parametrize("T,V,k", [(6, 1000, 12), (6, 33, 12), (6, 50257, 12), (200, 2050, 12)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ragged_lists(g, T, V, k, dt):
    """Absent entries, tokens without any, entries past the vocabulary, repeated entries, −infinity and the type's
    lowest value among teacher entries and masked logits."""
    z, index, t, up = make(T, V, k, dt)
    low = torch.finfo(DT[dt]).min
    index[0, 5:] = -1
    index[1, :] = -1
    index[2, 3], index[2, 4] = V, V + 10 ** 12
    index[3, 1], index[3, 7], index[3, 8] = index[3, 0], index[3, 0], index[3, 2]
    t[4, 2:], t[4, 0] = float("-inf"), torch.finfo(torch.float32).min
    t[5, :] = float("-inf")
    hit = torch.zeros(T, V, dtype=torch.bool, device="cuda").scatter_(1, index.clamp(0, V - 1), True)
    masked = (torch.arange(V, device="cuda") % 3 == 1) & ~hit
    for fill in (low, float("-inf")):
        zz = z.masked_fill(masked, fill)
        one, two = all_three(g, zz, index, t, up, 2.0)
        finite = zz.masked_fill(masked, -1e4) if fill == low else zz   # the oracle's R is of the logits that count
        for got in (one, two):
            check(finite, index, t, up, 2.0, *got, rows=slice(0, 40))
            assert got[0][1] == 0 and got[0][5] == 0 and not got[2][1].any() and not got[2][5].any()
            assert not got[2][masked].any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(2, 300), (2, 40000), (700, 300)])
def test_row_masked_whole(g, T, V, dt):
    """Every logit at the type's lowest value: q is uniform, however large the common value."""
    z, index, t, up = make(T, V, 3, dt)
    z[1] = torch.finfo(DT[dt]).min
    loss, lse, dz = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(z)
    for tau in (0.5, 1.0, 2.0):
        g.distill_topk_forward_backward(z, index, t, up, loss, lse, dz, temperature=tau)
        only = torch.empty_like(loss)
        g.distill_topk_forward(z, index, t, only, temperature=tau)
        sync()
        flat = torch.zeros_like(z[1:2])
        check(flat, index[1:2], t[1:2], up[1:2], tau, loss[1:2], None, dz[1:2])
        assert torch.equal(only, loss)
        check(z, index, t, up, tau, loss, lse, dz, rows=slice(0, 1))


def shifted(T, V, dt, common, seed=3):
    """Logits about a large common value, and what is left of them without it (exact: neighbours in the type)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    z = (torch.randn(T, V, generator=gen, device="cuda") * 2.5 + common).to(DT[dt])
    base = torch.tensor(float(common), device="cuda").to(DT[dt])
    return z, (z.double() - base.double())


@pytest.mark.parametrize("common", [2e3, 3e3, -3e3, 1e5, -1e5, 1e6, -1e9, 1e20])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(3, 515), (3, 4096), (2, 40000), (700, 1003)])
def test_large_common_value(g, T, V, dt, common):
    """A shift of all of a token's logits changes neither loss nor gradient, whatever |dloss|.  The logits' differences
    are exact, so only they enter the bound."""
    _, index, t, up = make(T, V, 7, dt)
    z, rest = shifted(T, V, dt, common)
    if rest.abs().amax() > 100:                # the type's spacing there: only rows of one value are left to compare
        z = torch.full_like(z, common)
        rest = torch.zeros_like(rest)
    for tau, w in ((1.0, up), (2.5, up / 8192), (1.0, -up * 2.0 ** -30)):
        loss, lse, dz = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(z)
        g.distill_topk_forward_backward(z, index, t, w, loss, lse, dz, temperature=tau)
        only = torch.empty_like(loss)
        g.distill_topk_forward(z, index, t, only, temperature=tau)
        sync()
        check(rest, index, t, w, tau, loss, None, dz, rows=slice(0, 8))
        assert torch.equal(only, loss)
        want = torch.logsumexp(z.double() / tau, 1)
        # m·c and its product with ln 2 round a few times; E of these sizes is below 1e-4
        assert torch.all((lse.double() - want).abs() <= 8 * U * want.abs() + 1e-4)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("common", [3e3, -3e3, 2e4, -2e4])
def test_kept_lse_of_large_logits(g, dt, common):
    """The gradient from a kept fp32 lse is that of exp(z/τ − lse) with the lse as it was rounded."""
    T, V, k = 5, 1003, 7
    _, index, t, up = make(T, V, k, dt)
    z, rest = shifted(T, V, dt, common)
    for tau in (1.0, 2.5, 3.0):
        exact = torch.logsumexp(z.double() / tau, 1)
        dz = torch.empty_like(z)
        g.distill_topk_backward(z, index, t, exact.float(), up, dz, temperature=tau)
        sync()
        q = torch.exp(z.double() / tau - exact.float().double()[:, None])
        p = torch.zeros_like(q).scatter_add_(1, index, torch.softmax(t.double() / tau, 1))
        gw = up.double()[:, None] * tau
        # as in check, with the size of the exponents' own terms: lse·log2(e) and z·c are rounded as they are
        E = (V / 128 + 64) * U + 16 * U * (float(rest.abs().amax() + t.abs().amax()) + abs(common)) / tau + 2.0 ** -20
        rnd = 2.0 ** -8 if dt == "bf16" else U
        want = gw * (q - p)
        assert torch.all((dz.double() - want).abs() <= gw.abs() * 2 * E * (q + p) + rnd * want.abs() + 1e-37)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(64, 515), (64, 40000), (700, 515)])
def test_kept_lse_that_cannot_carry_the_sum(g, T, V, dt):
    """Rows of one value near -1e9: whatever the fp32 lse rounds to, q stays a probability."""
    _, index, t, up = make(T, V, 5, dt)
    z = (-1e9 - 448.0 * torch.arange(T, device="cuda") * (1 if dt == "f32" else 2.0 ** 14))[:, None].expand(T, V).to(DT[dt]).contiguous()
    loss, lse, dz = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(z)
    for tau in (1.0, 1.5, 3.0):
        g.distill_topk_forward(z, index, t, loss, lse, temperature=tau)
        g.distill_topk_backward(z, index, t, lse, up, dz, temperature=tau)
        sync()
        # g·(q − p) with 0 <= q, p <= 1 lies within |g|, and a rounding
        assert torch.all(dz.double().abs() <= up.double().abs()[:, None] * tau * (1 + 2.0 ** -8))


def low_rows(T, V, dt, mask, slices, seed=5):
    """Rows of low logits: at the start of every slice a masked 16-byte vector and a stretch of -88 on the first vectors
    of a CTA's other threads, then -46 on what the masked one's thread reads and -52 elsewhere; rows of random levels
    and random masked vectors; rows of which a long stretch is masked."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    vec = 8 if dt == "bf16" else 4
    per = -(-(-(-V // slices)) // 128) * 128
    i = torch.arange(V, device="cuda") % per // vec
    z = torch.full((T, V), -52.0, device="cuda")
    z[:, i % 256 == 0] = -46.0
    z[:, (i > 0) & (i < 256)] = -88.0
    z[:, i == 0] = mask
    levels = torch.tensor([-88.0, -52.0, -46.0, -10.0, 0.0, 9.0], device="cuda")
    z[1::4] = levels[torch.randint(0, 6, (V // vec + 1,), generator=gen, device="cuda")].repeat_interleave(vec)[:V]
    z[2::4] = levels[torch.randint(0, 2, (V // vec + 1,), generator=gen, device="cuda")].repeat_interleave(vec)[:V]
    off = torch.rand(V // vec + 1, generator=gen, device="cuda").repeat_interleave(vec)[:V] < 0.3
    z[1:2, off] = mask
    z[2:3, off] = mask
    z[3::4] = torch.randn(V, generator=gen, device="cuda") * 2.5 - 20
    z[3::4, V // 8:V - V // 16] = mask
    return z.to(DT[dt])


@pytest.mark.parametrize("mask", [float("-inf"), -1e4])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,slices", [(320, 50176, 1), (4, 50176, 8), (4, 16384, 4), (320, 2051, 1)])
def test_masked_vectors_among_low_logits(g, T, V, slices, dt, mask):
    _, index, t, up = make(T, V, 5, dt)
    z = low_rows(T, V, dt, mask, slices)
    index = torch.arange(V - 5, V, device="cuda").repeat(T, 1)         # not masked: the loss is finite
    z[:, V - 5:] = -52.0
    for tau in (1.0, 2.0):
        for got in all_three(g, z, index, t, up, tau):
            finite = z.masked_fill(z <= -9e3, -1e3)                    # as far as any mask: R is of the logits that count
            check(finite, index, t, up, tau, *got, rows=slice(0, 4))


@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e10, -1e15, -1e20, -1e30])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(8, 2051), (8, 40000), (700, 2048), (320, 9000)])
def test_finite_masks(g, T, V, dt, mask):
    """Masks that are neither -infinity nor the type's lowest value: over one vector, a thread's or a cluster's whole
    share of the row, all but one logit, the whole row, and over none."""
    _, index, t, up = make(T, V, 4, dt)
    z = (torch.randn(T, V, device="cuda", generator=torch.Generator("cuda").manual_seed(7)) * 2.5).to(DT[dt])
    z[1, 8:16] = mask
    z[2, :V // 2] = mask
    z[3, V // 2:] = mask
    z[4, torch.arange(V, device="cuda") != int(index[4, 1])] = mask
    z[5] = mask
    z[6, torch.arange(V, device="cuda") // 8 % 256 == 3] = mask
    z[7] = mask
    z[7, ::3] = 2 * mask
    index[4] = index[4, 1].clone()
    index[2] = torch.where(index[2] < V // 2, -1, index[2])
    index[3] = torch.where(index[3] < V // 2, index[3], -1)
    index[6] = V - 1 - torch.arange(4, device="cuda") * 8
    index[7] = torch.arange(4, device="cuda") * 3 + 1
    flat = z.masked_fill(z <= -5e3, -1e3)                 # nothing beside the others, where there are others
    flat[5] = 0.0
    flat[7] = 0.0
    flat[7, ::3] = -1e3
    flat[6, index[6]], z[6, index[6]] = 1.0, 1.0
    for tau in (1.0, 2.0):
        (loss, lse, dz), (loss2, lse2, dz2) = all_three(g, z, index, t, up, tau)
        check(flat, index, t, up, tau, loss, None, dz, rows=slice(0, 8))
        check(flat, index, t, up, tau, loss2, None, None, rows=slice(0, 8))
        usual = torch.tensor([0, 1, 2, 3, 4, 6], device="cuda")
        check(flat, index, t, up, tau, loss2, lse2, dz2, rows=usual)
        check(flat, index, t, up, tau, None, lse, None, rows=usual)
        want = torch.logsumexp(z[[5, 7]].double() / tau, 1)
        for got in (lse, lse2):
            assert torch.all((got[[5, 7]].double() - want).abs() <= 8 * U * want.abs() + 1e-4)


def test_zero_weight_and_special_logits(g):
    z, index, t, up = make(5, 700, 8, "f32")
    up[0] = 0.0
    z[0, 3] = float("nan")                     # weight 0: its gradient is 0 all the same
    z[1, int(index[1, 2])] = float("-inf")     # the student gives an entry no probability: infinite loss
    z[2, 9] = float("nan")                     # NaN stays in its token
    index[3, :], z[3, :] = -1, float("nan")    # padding
    for loss, _, dz in all_three(g, z, index, t, up, 1.0):
        assert not dz[0].any() and torch.isinf(loss[1]) and loss[1] > 0
        assert torch.isfinite(dz[1]).all() and torch.isnan(loss[2]) and torch.isnan(dz[2]).any()
        assert loss[3] == 0 and not dz[3].any()
        check(z, index, t, up, 1.0, loss, None, dz, rows=slice(4, 5))
    # no dloss: 1
    dz, one = torch.empty_like(z[4:]), torch.empty_like(z[4:])
    lse = torch.logsumexp(z[4:].double(), 1).float()
    g.distill_topk_backward(z[4:], index[4:], t[4:], lse, None, dz)
    g.distill_topk_backward(z[4:], index[4:], t[4:], lse, torch.ones(1, device="cuda"), one)
    sync()
    assert torch.equal(dz, one)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(6, 515), (6, 40000), (700, 1001)])
def test_infinite_logits(g, T, V, dt):
    """+infinity at a word that is no entry, at an entry, at two words; -infinity throughout: one call and two agree on
    what the formulas leave, q = 0 at finite logits and NaN at the infinite one."""
    z, index, t, up = make(T, V, 4, dt)
    inf = float("inf")
    hit = torch.zeros(T, V, dtype=torch.bool, device="cuda").scatter_(1, index, True)
    word = int((~hit[0]).nonzero()[0])
    z[0, word] = inf
    z[1, int(index[1, 2])] = inf
    z[2, int((~hit[2]).nonzero()[5])], z[2, V - 1] = inf, inf
    z[3], z[4], index[4] = -inf, -inf, -1
    for tau in (1.0, 2.5):
        for loss, lse, dz in all_three(g, z, index, t, up, tau):
            assert torch.all(lse[:3] == inf) and torch.all(lse[3:5] == -inf)
            assert loss[0] == inf and torch.isnan(loss[1]) and torch.isnan(loss[3]) and loss[4] == 0
            p = torch.zeros(T, V, dtype=torch.float64, device="cuda").scatter_(1, index.clamp(0), torch.softmax(t.double() / tau, 1))
            for r in range(3):
                at = z[r] == inf
                want = -(up[r].double() * tau) * p[r]
                # a softmax of four terms; the type's rounding
                tol = (2.0 ** -18 + (2.0 ** -8 if dt == "bf16" else U)) * want.abs()
                assert torch.isnan(dz[r][at]).all() and torch.all(((dz[r].double() - want).abs() <= tol)[~at])
            assert torch.isnan(dz[3]).all() and not dz[4].any()
            check(z, index, t, up, tau, loss, lse, dz, rows=slice(5, 6))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(7, 515), (3, 50257), (300, 1001)])
def test_strides_offsets_and_in_place(g, T, V, dt):
    k = 6
    z, index, t, up = make(T, V, k, dt)
    ref = all_three(g, z, index, t, up, 2.0)[0]
    wide = torch.full((T, V + 11), 5.0, device="cuda", dtype=DT[dt])
    wide[:, 3:3 + V] = z
    ib, tb = torch.full((T, k + 3), -7, device="cuda"), torch.full((T, k + 1), 9.0, device="cuda")
    ib[:, 2:2 + k], tb[:, 1:] = index, t
    out = torch.full((T, V + 6), 8.0, device="cuda", dtype=DT[dt])
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    zs, is_, ts = wide[:, 3:3 + V], ib[:, 2:2 + k], tb[:, 1:]
    g.distill_topk_forward_backward(zs, is_, ts, up, loss, lse, out[:, 1:1 + V], temperature=2.0)
    sync()
    rows = slice(0, 20)
    check(z, index, t, up, 2.0, loss, lse, out[:, 1:1 + V], rows=rows)
    assert torch.all(out[:, :1] == 8) and torch.all(out[:, 1 + V:] == 8)
    g.distill_topk_backward(zs, is_, ts, lse, up, zs, temperature=2.0)            # on the logits themselves
    sync()
    check(z, index, t, up, 2.0, None, None, zs, rows=rows)
    assert torch.all(wide[:, :3] == 5) and torch.all(wide[:, 3 + V:] == 5)
    z2 = z.clone()
    g.distill_topk_forward_backward(z2, index, t, up, loss, lse, z2, temperature=2.0)
    sync()
    assert torch.equal(z2, ref[2]) and torch.equal(loss, ref[0])


def test_gradient_against_differences(g):
    """Central differences of Σ up·loss of the forward kernel along random directions."""
    T, V, k, tau, e = 4, 300, 10, 2.0, 2.0 ** -5
    z, index, t, up = make(T, V, k, "f32")
    _, _, dz = all_three(g, z, index, t, up, tau)[0]

    def f(z):
        loss = torch.empty(T, device="cuda")
        g.distill_topk_forward(z, index, t, loss, temperature=tau)
        return float((loss.double() * up.double()).sum())
    for seed in range(5):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(90 + seed)
        d = torch.randn(T, V, generator=gen, device="cuda")
        num = (f(z + e * d) - f(z - e * d)) / (2 * e)
        # rounding: losses of at most ~100 off by ~2^-17 of themselves at worst, over 2e;
        # truncation: e²/6 times a third cumulant of d/τ under q (|d| <= 4.5), times τ²
        tol = T * 3 * (100 * 2.0 ** -21) / e + T * 3 * tau * tau * e * e / 6 * (4.5 / tau) ** 3
        assert abs(num - float((dz.double() * d.double()).sum())) <= tol


def test_empty(g):
    z, index, t, up = make(4, 50, 3)
    e = torch.empty(0, device="cuda")
    g.distill_topk_forward_backward(z[:0], index[:0], t[:0], e, e, e, z[:0].clone())
    loss = torch.full((4,), 9.0, device="cuda")
    dz = torch.full_like(z, 9.0)
    g.distill_topk_forward_backward(z, index[:, :0], t[:, :0], up, loss, None, dz)      # no entries at all
    sync()
    assert not loss.any() and not dz.any()


@pytest.mark.parametrize("T,V", [(3, 50257), (400, 2003)])
def test_other_stream_repeat_and_graph(g, T, V):
    z, index, t, up = make(T, V, 20)
    index[:, 5] = index[:, 3]
    index[:, 9] = index[:, 3]
    ref = all_three(g, z, index, t, up, 2.0)[0]
    loss, lse, dz = (torch.zeros_like(v) for v in ref)
    side = torch.cuda.Stream()
    sync()
    g.distill_topk_forward_backward(z, index, t, up, loss, lse, dz, temperature=2.0, stream=side)
    sync()
    for a, b in zip((loss, lse, dz), ref):
        assert torch.equal(a, b)
        a.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.distill_topk_forward_backward(z, index, t, up, loss, lse, dz, temperature=2.0)
    graph.replay()
    sync()
    for a, b in zip((loss, lse, dz), ref):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(g):
    T, V, k = 42800, 50257, 4
    z = torch.zeros(T, V, device="cuda", dtype=torch.bfloat16)
    zz, ii, tt, uu = make(3, V, k)
    z[-3:] = zz
    index, t, up = torch.zeros(T, k, dtype=torch.int64, device="cuda"), torch.zeros(T, k, device="cuda"), torch.ones(T, device="cuda")
    index[-3:], t[-3:], up[-3:] = ii, tt, uu
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dz = torch.empty_like(z)
    g.distill_topk_forward_backward(z, index, t, up, loss, lse, dz, temperature=2.0)
    sync()
    check(z, index, t, up, 2.0, loss, lse, dz, rows=slice(T - 3, T))
