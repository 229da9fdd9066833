"""The binding of the distillation operators on the host: what a first call publishes, and sizes beyond 32 bits."""
import sys

import pytest
import torch


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    __graft_entry__.build()
    import gradient_sync_ddp_gb300 as pkg
    return pkg


def test_first_call_publishes_the_codes_last(g):
    """Another thread takes a filled `codes` for the sign that all the rest is there, at any line of `load`."""
    T, names = g._Torch, ("f32", "bf16", "i8", "i32", "i64")
    T.codes = {}
    for n in names:
        setattr(T, n, None)
    if "stream" in vars(T):
        del T.stream
    seen = []

    def trace(frame, event, arg):
        if frame.f_code is T.load.__func__.__code__ and T.codes:
            seen.append(all(getattr(T, n) is not None for n in names) and hasattr(T, "stream"))
        return trace
    old = sys.gettrace()
    sys.settrace(trace)
    try:
        T.load()
    finally:
        sys.settrace(old)
    assert T.codes and seen and all(seen)


def test_sizes_past_32_bits_are_refused(g):
    """A width of 2^32 + 64 is not one of 64 (tensors without storage: a call that got as far would refuse them as NULL)."""
    wide, meta = 2 ** 32 + 64, torch.device("meta")

    def m(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=meta)
    f32, i8 = torch.float32, torch.int8
    assert g.rmsnorm_backward_workspace_bytes(4, wide) == 0 == g.q8_matmul_workspace_bytes(40, 64, wide)
    x, y, v = m(2, wide), m(2, wide), m(2, dtype=f32)
    idx, t, wide_idx, wide_t = m(2, 4, dtype=torch.int64), m(2, 4), m(2, 2 ** 32 + 4, dtype=torch.int64), m(2, 2 ** 32 + 4)
    for call in (lambda: g.rmsnorm_forward(x, None, y, stream=0),
                 lambda: g.rmsnorm_forward_q8(x, None, m(2, wide, dtype=i8), v, stream=0),
                 lambda: g.rmsnorm_backward(x, y, v, None, y, stream=0),
                 lambda: g.q8_matmul(m(2, wide, dtype=i8), v, m(3, wide, dtype=i8), m(3, dtype=f32), m(2, 3), m(64), stream=0),
                 lambda: g.distill_topk_forward(x, idx, t, v, stream=0),
                 lambda: g.distill_topk_backward(x, idx, t, v, None, y, stream=0),
                 lambda: g.distill_topk_forward_backward(m(2, 64), wide_idx, wide_t, None, v, None, m(2, 64), stream=0)):
        with pytest.raises(g.DdpError) as e:
            call()
        assert e.value.status == g.DDP_ERR_UNSUPPORTED
    # no rows: the call would have been answered with an empty result of another width
    with pytest.raises(g.DdpError):
        g.rmsnorm_forward(m(0, wide), None, m(0, wide), stream=0)
