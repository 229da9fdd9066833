"""The operators of a distillation step refuse what they cannot run, on the
host and before any CUDA call (the addresses below are never dereferenced),
and take empty requests."""
import ctypes

import pytest
import torch

BASE = 1 << 40


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    __graft_entry__.build()
    import gradient_sync_ddp_gb300 as pkg
    return pkg


def at(i):
    return BASE + (i << 24)


def norm_args(**kw):
    a = dict(x=at(0), ldx=64, res=at(1), ldr=64, dt=1, gamma=at(2), rows=4, D=64, eps=1e-6, h=at(3), ldh=64, y=at(4),
             ldy=64, odt=1, rstd=at(5))
    a.update(kw)
    return a


def norm(g, **kw):
    return g.lib_handle().rmsnorm_forward(*norm_args(**kw).values(), None)


def test_norm_forward(g):
    I, A = g.DDP_ERR_INVALID_ARG, g.DDP_ERR_ALIGNMENT
    assert norm(g, rows=0) == g.DDP_OK
    assert norm(g, rows=0, x=None, res=None, gamma=None, h=None, y=None, rstd=None) == g.DDP_OK
    for bad in (dict(x=None), dict(y=None), dict(dt=2), dict(odt=-1), dict(rows=-1), dict(D=0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(ldx=63), dict(ldr=1), dict(ldh=63), dict(ldy=0),
                dict(y=at(3)),                                   # y on h
                dict(y=at(0) + 16), dict(h=at(1) + 64), dict(y=at(0), odt=0),   # partial or wider overlap
                dict(rstd=at(4)), dict(gamma=at(3) + 4), dict(rstd=at(0)), dict(ldx=1 << 62)):
        assert norm(g, **bad) == I, bad
    for bad in (dict(x=at(0) + 1), dict(y=at(4) + 1), dict(gamma=at(2) + 2), dict(rstd=at(5) + 2)):
        assert norm(g, **bad) == A, bad


def test_norm_q8(g):
    f = g.lib_handle().rmsnorm_forward_q8

    def call(**kw):
        a = dict(x=at(0), ldx=64, res=at(1), ldr=64, dt=1, gamma=at(2), rows=4, D=64, eps=1e-6, h=at(3), ldh=64,
                 q=at(4), ldq=64, scale=at(6), rstd=at(5))
        a.update(kw)
        return f(*a.values(), None)
    assert call(rows=0) == g.DDP_OK
    for bad in (dict(q=None), dict(scale=None), dict(q=at(0)), dict(q=at(3)), dict(scale=at(5)), dict(scale=at(4)),
                dict(ldq=63)):
        assert call(**bad) == g.DDP_ERR_INVALID_ARG, bad
    assert call(scale=at(6) + 1) == g.DDP_ERR_ALIGNMENT


def test_norm_backward(g):
    f = g.lib_handle().rmsnorm_backward
    need = g.rmsnorm_backward_workspace_bytes(4, 64)
    assert need > 0 and g.rmsnorm_backward_workspace_bytes(-1, 64) == 0 == g.rmsnorm_backward_workspace_bytes(4, 0)

    def call(**kw):
        a = dict(dy=at(0), lddy=64, dydt=1, h=at(1), ldh=64, hdt=1, rstd=at(2), gamma=at(3), dh=at(4), lddh=64, rows=4,
                 D=64, dx=at(5), lddx=64, dgamma=at(6), ws=at(7), wsb=need)
        a.update(kw)
        return f(*a.values(), None)
    assert call(rows=0, dgamma=None) == g.DDP_OK
    for bad in (dict(dy=None), dict(h=None), dict(rstd=None), dict(dx=None), dict(ws=None), dict(dydt=9),
                dict(hdt=3), dict(rows=-1), dict(D=0), dict(lddy=1), dict(dx=at(1) + 2), dict(dgamma=at(3)),
                dict(ws=at(5)), dict(ws=at(6)), dict(dx=at(0), dydt=0), dict(dx=at(2))):
        assert call(**bad) == g.DDP_ERR_INVALID_ARG, bad
    assert call(ws=at(7) + 8) == g.DDP_ERR_ALIGNMENT and call(dgamma=at(6) + 2) == g.DDP_ERR_ALIGNMENT
    assert call(wsb=need - 1) == g.DDP_ERR_CAPACITY


def test_product(g):
    f = g.lib_handle().q8_matmul
    need = g.q8_matmul_workspace_bytes(8, 16, 32)
    assert need > 0 and g.q8_matmul_workspace_bytes(-1, 16, 32) == 0 == g.q8_matmul_workspace_bytes(8, 16, 131072)

    def call(**kw):
        a = dict(a=at(0), lda=32, sa=at(1), w=at(2), ldw=32, sw=at(3), M=8, N=16, K=32, out=at(4), ldo=16, dt=1,
                 ws=at(5), wsb=need)
        a.update(kw)
        return f(*a.values(), None)
    assert call(M=0) == g.DDP_OK and call(N=0, ldo=0) == g.DDP_OK
    for bad in (dict(a=None), dict(w=None), dict(sa=None), dict(sw=None), dict(out=None), dict(ws=None), dict(dt=7),
                dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=31), dict(ldw=31), dict(ldo=15), dict(out=at(0)),
                dict(out=at(3)), dict(ws=at(4)), dict(ws=at(2))):
        assert call(**bad) == g.DDP_ERR_INVALID_ARG, bad
    assert call(out=at(4) + 1) == g.DDP_ERR_ALIGNMENT and call(ws=at(5) + 4) == g.DDP_ERR_ALIGNMENT
    assert call(wsb=need - 1) == g.DDP_ERR_CAPACITY
    assert call(K=131072, lda=131072, ldw=131072) == g.DDP_ERR_UNSUPPORTED
    assert call(M=1 << 31) == g.DDP_ERR_UNSUPPORTED


def test_distill(g):
    lib = g.lib_handle()

    def common(**kw):
        a = dict(z=at(0), ldz=100, dt=1, idx=at(1), ldi=5, bits=64, t=at(2), ldt=5, tdt=0, T=3, V=100, k=5, tau=1.0)
        extra = {n: v for n, v in kw.items() if n not in a}
        a.update({n: v for n, v in kw.items() if n in a})
        return list(a.values()), extra

    def fwd(**kw):
        a, e = common(**kw)
        return lib.distill_topk_forward(*a, e.get("loss", at(3)), e.get("lse", at(4)), None)

    def bwd(**kw):
        a, e = common(**kw)
        return lib.distill_topk_backward(*a, e.get("lse", at(4)), e.get("dloss", at(5)), e.get("dz", at(6)),
                                         e.get("lddz", 100), None)

    def both(**kw):
        a, e = common(**kw)
        return lib.distill_topk_forward_backward(*a, e.get("dloss", at(5)), e.get("loss", at(3)), e.get("lse", at(4)),
                                                 e.get("dz", at(6)), e.get("lddz", 100), None)
    for f in (fwd, bwd, both):
        assert f(T=0) == g.DDP_OK
        for bad in (dict(z=None), dict(idx=None), dict(t=None), dict(dt=2), dict(tdt=2), dict(bits=16), dict(T=-1),
                    dict(V=0), dict(k=-1), dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")),
                    dict(tau=float("inf")), dict(ldz=99), dict(ldi=4), dict(ldt=4)):
            assert f(**bad) == g.DDP_ERR_INVALID_ARG, (f, bad)
        assert f(k=1025, ldi=1025, ldt=1025) == g.DDP_ERR_UNSUPPORTED
        assert f(z=at(0) + 1) == g.DDP_ERR_ALIGNMENT and f(idx=at(1) + 4) == g.DDP_ERR_ALIGNMENT
    for f, bad in ((fwd, dict(loss=None)), (fwd, dict(loss=at(0))), (fwd, dict(lse=at(3))), (fwd, dict(loss=at(2))),
                   (bwd, dict(lse=None)), (bwd, dict(dz=None)), (bwd, dict(dz=at(0) + 2)), (bwd, dict(lddz=99)),
                   (bwd, dict(dz=at(1))), (both, dict(dz=at(0), lddz=101)), (both, dict(loss=at(6))),
                   (both, dict(loss=at(5))), (both, dict(dz=at(2)))):
        assert f(**bad) == g.DDP_ERR_INVALID_ARG, (f, bad)


def test_binding_checks_tensors(g):
    x, v = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8)
    with pytest.raises(ValueError):
        g.rmsnorm_forward(x, v, torch.zeros(4, 7, dtype=torch.bfloat16), stream=0)
    with pytest.raises(ValueError):
        g.rmsnorm_forward(x, v, torch.zeros(8, 4, dtype=torch.bfloat16).t(), stream=0)
    with pytest.raises(TypeError):
        g.rmsnorm_forward(x, v.double(), torch.zeros_like(x), stream=0)
    with pytest.raises(TypeError):
        g.rmsnorm_forward(x, v, torch.zeros_like(x), residual=torch.zeros(4, 8), stream=0)
    with pytest.raises(TypeError):
        g.rmsnorm_forward_q8(x, v, torch.zeros(4, 8, dtype=torch.uint8), torch.zeros(4), stream=0)
    with pytest.raises(ValueError):
        g.rmsnorm_backward(x, x, torch.zeros(3), v, torch.zeros_like(x), stream=0)
    a, w, ws = torch.zeros(2, 8, dtype=torch.int8), torch.zeros(3, 7, dtype=torch.int8), torch.zeros(16)
    with pytest.raises(ValueError):
        g.q8_matmul(a, torch.zeros(2), w, torch.zeros(3), torch.zeros(2, 3), ws, stream=0)
    with pytest.raises(TypeError):
        g.q8_matmul(a.float(), torch.zeros(2), w, torch.zeros(3), torch.zeros(2, 3), ws, stream=0)
    z, t = torch.zeros(3, 9), torch.zeros(3, 2)
    with pytest.raises(TypeError):
        g.distill_topk_forward(z, t, t, torch.zeros(3), stream=0)
    with pytest.raises(ValueError):
        g.distill_topk_forward(z, torch.zeros(2, 2, dtype=torch.int64), t, torch.zeros(3), stream=0)
    with pytest.raises(TypeError):
        g.distill_topk_backward(z, torch.zeros(3, 2, dtype=torch.int32), t, torch.zeros(3), None, z.bfloat16(),
                                stream=0)
    with pytest.raises(g.DdpError):
        g.distill_topk_forward(z, torch.zeros(3, 2, dtype=torch.int32), t, torch.zeros(3), temperature=0.0, stream=0)


def test_widths_that_32_bits_cannot_count(g):
    """Column numbers, rounded up to what a CTA takes at a time, would pass 2^31."""
    h, U, wide = g.lib_handle(), g.DDP_ERR_UNSUPPORTED, 2**31 - 65535
    assert norm(g, rows=1, D=wide, ldx=wide, ldr=wide, ldh=wide, ldy=wide) == U
    assert h.rmsnorm_forward_q8(at(0), wide, None, wide, 1, None, 1, wide, 1e-6, None, wide, at(4), wide, at(6), None,
                                None) == U
    assert h.rmsnorm_backward(at(0), wide, 1, at(1), wide, 1, at(2), None, None, wide, 1, wide, at(3), wide, None, None,
                              0, None) == U
    assert h.q8_matmul(at(0), 64, at(1), at(2), 64, at(3), 1, wide, 64, at(4), wide, 0, at(5), 1 << 20, None) == U
    assert h.q8_matmul(at(0), 64, at(1), at(2), 64, at(3), wide, 1, 64, at(4), 1, 0, at(5), 1 << 20, None) == U
    assert h.q8_matmul_workspace_bytes(wide, 64, 64) == h.q8_matmul_workspace_bytes(64, wide, 64) == 0
    assert h.rmsnorm_backward_workspace_bytes(4, wide) == 0
    t = (at(1), 8, 32, at(2), 8, 0, 1, wide, 8, 1.0)
    assert h.distill_topk_forward(at(0), wide, 1, *t, at(3), None, None) == U
    assert h.distill_topk_backward(at(0), wide, 1, *t, at(3), None, at(4), wide, None) == U
    assert h.distill_topk_forward_backward(at(0), wide, 1, *t, None, at(3), None, at(4), wide, None) == U
