"""The operators of a transformer's training step refuse what they cannot run, on the host and before any CUDA call (the
addresses below are never dereferenced), and take empty requests."""
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


def caller(f, **defaults):
    def call(**kw):
        assert set(kw) <= set(defaults)
        return f(*{**defaults, **kw}.values(), None)
    return call


def test_layernorm_forward(g):
    I, A = g.DDP_ERR_INVALID_ARG, g.DDP_ERR_ALIGNMENT
    call = caller(g.lib_handle().layernorm_forward, x=at(0), ldx=64, res=at(1), ldr=64, dt=1, gamma=at(2), beta=at(8),
                  rows=4, D=64, eps=1e-6, h=at(3), ldh=64, y=at(4), ldy=64, odt=1, mean=at(6), rstd=at(5))
    assert call(rows=0) == g.DDP_OK
    assert call(rows=0, x=None, res=None, gamma=None, beta=None, h=None, y=None, mean=None, rstd=None) == g.DDP_OK
    for bad in (dict(x=None), dict(y=None), dict(dt=2), dict(odt=-1), dict(rows=-1), dict(D=0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(ldx=63), dict(ldr=1), dict(ldh=63), dict(ldy=0), dict(y=at(3)),
                dict(y=at(0) + 16), dict(h=at(1) + 64), dict(y=at(0), odt=0), dict(rstd=at(4)), dict(gamma=at(3) + 4),
                dict(beta=at(4) + 8), dict(rstd=at(0)), dict(mean=at(5)), dict(mean=at(8)), dict(ldx=1 << 62)):
        assert call(**bad) == I, bad
    for bad in (dict(x=at(0) + 1), dict(y=at(4) + 1), dict(gamma=at(2) + 2), dict(beta=at(8) + 1), dict(rstd=at(5) + 2),
                dict(mean=at(6) + 2)):
        assert call(**bad) == A, bad
    wide = 2 ** 31 - 65535
    assert call(rows=1, D=wide, ldx=wide, ldr=wide, ldh=wide, ldy=wide) == g.DDP_ERR_UNSUPPORTED


def test_layernorm_backward(g):
    need = g.layernorm_backward_workspace_bytes(4, 64)
    assert need > 0 and g.layernorm_backward_workspace_bytes(-1, 64) == 0 == g.layernorm_backward_workspace_bytes(4, 0)
    assert g.layernorm_backward_workspace_bytes(4, 2 ** 31 - 65535) == 0
    call = caller(g.lib_handle().layernorm_backward, dy=at(0), lddy=64, dydt=1, h=at(1), ldh=64, hdt=1, mean=at(9),
                  rstd=at(2), gamma=at(3), dh=at(4), lddh=64, rows=4, D=64, dx=at(5), lddx=64, dgamma=at(6), dbeta=at(8),
                  ws=at(7), wsb=need)
    assert call(rows=0, dgamma=None, dbeta=None) == g.DDP_OK
    for bad in (dict(dy=None), dict(h=None), dict(mean=None), dict(rstd=None), dict(dx=None), dict(ws=None),
                dict(ws=None, dgamma=None), dict(dydt=9), dict(hdt=3), dict(rows=-1), dict(D=0), dict(lddy=1),
                dict(dx=at(1) + 2), dict(dgamma=at(3)), dict(dbeta=at(6)), dict(dbeta=at(5)), dict(ws=at(5)), dict(ws=at(6)),
                dict(ws=at(8)), dict(dx=at(0), dydt=0), dict(dx=at(2)), dict(dx=at(9))):
        assert call(**bad) == g.DDP_ERR_INVALID_ARG, bad
    assert call(ws=at(7) + 8) == g.DDP_ERR_ALIGNMENT and call(dgamma=at(6) + 2) == g.DDP_ERR_ALIGNMENT
    assert call(dbeta=at(8) + 2) == g.DDP_ERR_ALIGNMENT and call(wsb=need - 1) == g.DDP_ERR_CAPACITY


def test_logprobs_forward(g):
    call = caller(g.lib_handle().token_logprobs_forward, z=at(0), ldz=100, dt=1, target=at(1), bits=64, T=3, V=100,
                  tau=1.0, logp=at(2), ent=at(3), lse=at(4), k=5, ti=at(5), ldti=5, ibits=64, tl=at(6), ldtl=5)
    assert call(T=0) == g.DDP_OK and call(T=0, z=None, target=None, logp=None, ent=None, lse=None, ti=None, tl=None) == g.DDP_OK
    for bad in (dict(z=None), dict(target=None), dict(dt=2), dict(bits=16), dict(ibits=8), dict(T=-1), dict(V=0), dict(k=-1),
                dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")), dict(tau=1e-45), dict(ldz=99),
                dict(ldti=4), dict(ldtl=4), dict(logp=at(0)), dict(ent=at(2)), dict(lse=at(3)), dict(ti=at(6)),
                dict(tl=at(0)), dict(lse=at(1)), dict(ti=at(1))):
        assert call(**bad) == g.DDP_ERR_INVALID_ARG, bad
    for bad in (dict(z=at(0) + 1), dict(target=at(1) + 4), dict(logp=at(2) + 2), dict(ti=at(5) + 4), dict(tl=at(6) + 1)):
        assert call(**bad) == g.DDP_ERR_ALIGNMENT, bad
    assert call(k=g.LOGPROB_MAX_TOP + 1, ldti=500, ldtl=500) == g.DDP_ERR_UNSUPPORTED
    wide = 2 ** 31 - 65535
    assert call(T=1, V=wide, ldz=wide) == g.DDP_ERR_UNSUPPORTED


def test_logprobs_backward(g):
    call = caller(g.lib_handle().token_logprobs_backward, z=at(0), ldz=100, dt=1, target=at(1), bits=64, T=3, V=100,
                  tau=1.0, lse=at(2), ent=at(3), up=at(4), ue=at(5), dz=at(6), lddz=100)
    assert call(T=0) == g.DDP_OK
    for bad in (dict(z=None), dict(target=None), dict(lse=None), dict(ent=None), dict(dz=None), dict(dt=2), dict(bits=16),
                dict(T=-1), dict(V=0), dict(tau=0.0), dict(tau=float("nan")), dict(ldz=99), dict(lddz=99),
                dict(dz=at(0) + 2), dict(dz=at(0), lddz=101), dict(dz=at(1)), dict(dz=at(2)), dict(dz=at(5))):
        assert call(**bad) == g.DDP_ERR_INVALID_ARG, bad
    for bad in (dict(z=at(0) + 1), dict(target=at(1) + 4), dict(lse=at(2) + 2), dict(up=at(4) + 1), dict(dz=at(6) + 1)):
        assert call(**bad) == g.DDP_ERR_ALIGNMENT, bad
    wide = 2 ** 31 - 65535
    assert call(T=1, V=wide, ldz=wide, lddz=wide) == g.DDP_ERR_UNSUPPORTED


def test_binding_checks_tensors(g):
    x, v = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8)
    t, z = torch.zeros(4, dtype=torch.int64), torch.zeros(4, 9)
    for error, call in (
            (ValueError, lambda: g.layernorm_forward(x, v, v, torch.zeros(4, 7, dtype=torch.bfloat16), stream=0)),
            (ValueError, lambda: g.layernorm_forward(x, v, torch.zeros(7), torch.zeros_like(x), stream=0)),
            (TypeError, lambda: g.layernorm_forward(x, v, v.double(), torch.zeros_like(x), stream=0)),
            (ValueError, lambda: g.layernorm_backward(x, x, torch.zeros(4), torch.zeros(3), v, torch.zeros_like(x), stream=0)),
            (TypeError, lambda: g.layernorm_backward(x, x, torch.zeros(4), torch.zeros(4), v, torch.zeros(4, 8), stream=0)),
            (ValueError, lambda: g.token_logprobs_forward(z, None, torch.zeros(4), stream=0)),
            (TypeError, lambda: g.token_logprobs_forward(z, t.float(), torch.zeros(4), stream=0)),
            (ValueError, lambda: g.token_logprobs_forward(z, t[:3], torch.zeros(4), stream=0)),
            (TypeError, lambda: g.token_logprobs_forward(z, t, None, top_index=torch.zeros(4, 2), stream=0)),
            (ValueError, lambda: g.token_logprobs_forward(z, t, None, top_index=torch.zeros(4, 2, dtype=torch.int64),
                                                          top_logprob=torch.zeros(4, 3), stream=0)),
            (ValueError, lambda: g.token_logprobs_forward(z, t, None, top_logprob=torch.zeros(3, 2), stream=0)),
            (TypeError, lambda: g.token_logprobs_backward(z, t, torch.zeros(4), None, z.bfloat16(), stream=0)),
            (ValueError, lambda: g.token_logprobs_backward(z, None, torch.zeros(4), torch.zeros(4), z.clone(), stream=0))):
        with pytest.raises(error):
            call()
    with pytest.raises(g.DdpError):
        g.token_logprobs_forward(z, t, torch.zeros(4), temperature=0.0, stream=0)


def test_sizes_past_32_bits_are_refused(g):
    wide, meta = 2 ** 32 + 64, torch.device("meta")

    def m(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=meta)
    f32, x, v, t = torch.float32, m(2, wide), m(2, dtype=torch.float32), m(2, dtype=torch.int64)
    assert g.layernorm_backward_workspace_bytes(4, wide) == 0
    for call in (lambda: g.layernorm_forward(x, None, None, m(2, wide), stream=0),
                 lambda: g.layernorm_backward(x, m(2, wide), v, v, None, m(2, wide), stream=0),
                 lambda: g.token_logprobs_forward(x, t, v, stream=0),
                 lambda: g.token_logprobs_forward(m(2, 64), t, None, top_logprob=m(2, 2 ** 32 + 4, dtype=f32), stream=0),
                 lambda: g.token_logprobs_backward(x, t, v, v, m(2, wide), stream=0)):
        with pytest.raises(g.DdpError) as e:
            call()
        assert e.value.status == g.DDP_ERR_UNSUPPORTED


def test_newton_schulz(g):
    import ctypes
    need = g.newton_schulz_workspace_bytes(2, 64, 100)
    f = g.newton_schulz_workspace_bytes
    assert need > 0 and f(-1, 4, 4) == f(1, -1, 4) == f(1, 4, -1) == f(1, 65537, 4) == f(1, 4, 65537) == 0
    assert f(0, 4, 4) == 16 and f(64, 8, 8) == f(1000, 8, 8)

    def ptrs(*a):
        return (ctypes.c_void_p * len(a))(*a)
    call = caller(g.lib_handle().newton_schulz, x=ptrs(at(0), at(1)), ldx=100, xdt=0, out=ptrs(at(2), at(3)), ldo=100, odt=1,
                  count=2, rows=64, cols=100, steps=5, eps=1e-7, ws=at(5), wsb=need)
    assert call(count=0) == g.DDP_OK and call(rows=0) == g.DDP_OK and call(cols=0, x=None, out=None, ws=None) == g.DDP_OK
    for bad in (dict(x=None), dict(out=None), dict(ws=None), dict(xdt=2), dict(odt=-1), dict(count=-1), dict(rows=-1),
                dict(cols=-1), dict(steps=0), dict(steps=17), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(ldx=99), dict(ldo=99), dict(x=ptrs(at(0), None)), dict(out=ptrs(None, at(3))),
                dict(out=ptrs(at(2), at(2) + 16)), dict(out=ptrs(at(0), at(3))), dict(out=ptrs(at(1), at(3)), odt=0),
                dict(ws=at(0)), dict(ws=at(3))):
        assert call(**bad) == g.DDP_ERR_INVALID_ARG, bad
    assert call(x=ptrs(at(0) + 2, at(1))) == g.DDP_ERR_ALIGNMENT and call(ws=at(5) + 8) == g.DDP_ERR_ALIGNMENT
    assert call(wsb=need - 1) == g.DDP_ERR_CAPACITY and call(rows=65537) == g.DDP_ERR_UNSUPPORTED


def test_muon(g):
    import ctypes
    need = g.newton_schulz_workspace_bytes(2, 8, 16)
    reps = (ctypes.c_void_p * 2)(at(0), at(1))

    def offs(*a):
        return (ctypes.c_int64 * len(a))(*a)
    call = caller(g.lib_handle().ddp_bucket_allreduce_muon, r=reps, n=2, dt=1, off=offs(0, 128), count=2, rows=8, cols=16,
                  p=at(2), b=at(3), lr=0.1, mu=0.9, wd=0.0, scale=1.0, nest=1, steps=5, eps=1e-7, half=at(4), ws=at(5), wsb=need)
    assert call(count=0) == g.DDP_OK and call(rows=0, r=None, off=None, p=None, b=None, ws=None) == g.DDP_OK
    for bad in (dict(r=None), dict(off=None), dict(p=None), dict(b=None), dict(ws=None), dict(n=0), dict(n=17), dict(dt=3),
                dict(count=-1), dict(rows=-1), dict(steps=0), dict(steps=99), dict(eps=float("nan")), dict(off=offs(0, 127)),
                dict(off=offs(-1, 128)), dict(off=offs(0, 1 << 62)), dict(p=at(0)), dict(b=at(2)), dict(half=at(3)),
                dict(ws=at(1)), dict(p=at(5)), dict(r=(ctypes.c_void_p * 2)(at(0), None))):
        assert call(**bad) == g.DDP_ERR_INVALID_ARG, bad
    for bad in (dict(p=at(2) + 4), dict(b=at(3) + 8), dict(half=at(4) + 2), dict(ws=at(5) + 8),
                dict(r=(ctypes.c_void_p * 2)(at(0), at(1) + 2))):
        assert call(**bad) == g.DDP_ERR_ALIGNMENT, bad
    assert call(wsb=need - 1) == g.DDP_ERR_CAPACITY and call(rows=8, cols=65537) == g.DDP_ERR_UNSUPPORTED


def test_muon_binding(g):
    x, ws = torch.zeros(4, 8), torch.zeros(16)
    flat = torch.zeros(64)
    for error, call in (
            (ValueError, lambda: g.newton_schulz([x], [], ws, stream=0)),
            (ValueError, lambda: g.newton_schulz([x, torch.zeros(4, 9)[:, :8]], [x, x], ws, stream=0)),
            (ValueError, lambda: g.newton_schulz([x], [torch.zeros(8, 4)], ws, stream=0)),
            (TypeError, lambda: g.newton_schulz([x, x.bfloat16()], [x, x], ws, stream=0)),
            (TypeError, lambda: g.newton_schulz([x.double()], [x], ws, stream=0)),
            (ValueError, lambda: g.ddp_bucket_allreduce_muon([], [0], 4, 8, flat, flat, ws, 0.1, 0.9, 0.0, stream=0)),
            (ValueError, lambda: g.ddp_bucket_allreduce_muon([flat], [33], 4, 8, flat, flat, ws, 0.1, 0.9, 0.0, stream=0)),
            (ValueError, lambda: g.ddp_bucket_allreduce_muon([flat], [0], 4, 8, flat[:31], flat, ws, 0.1, 0.9, 0.0, stream=0)),
            (TypeError, lambda: g.ddp_bucket_allreduce_muon([flat], [0], 4, 8, flat.bfloat16(), flat, ws, 0.1, 0.9, 0.0, stream=0)),
            (TypeError, lambda: g.ddp_bucket_allreduce_muon([flat, flat.bfloat16()], [0], 4, 8, flat, flat, ws, 0.1, 0.9, 0.0,
                                                            stream=0)),
            (g.DdpError, lambda: g.newton_schulz([x], [x], ws, steps=0, stream=0))):
        with pytest.raises(error):
            call()
    assert g.newton_schulz_workspace_bytes(1, 2 ** 32 + 4, 4) == 0
