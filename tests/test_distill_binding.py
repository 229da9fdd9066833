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
