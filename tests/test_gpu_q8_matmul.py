"""Product of 8-bit integers with scales on the GPU against the fp64 oracle.

Tolerance: with u = 2^-24, the sum is exact while partial sums stay below
2^24 in fp32 accumulators (always for K <= 1024); the two scalings and a
conversion round three times, bf16 once more (2^-8 with room for a value at a
rounding boundary).  Above 2^24 each of the K/16 steps of an accumulator may
round or truncate a sum that Σ|a·w| bounds: K/16·2u of it."""
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


def ints(rows, K, seed, low=-128, high=128):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randint(low, high, (rows, K), generator=gen, device="cuda", dtype=torch.int32).to(torch.int8)


def scales(n, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.rand(n, generator=gen, device="cuda") * 0.02 + 1e-3


def run(g, a, sa, w, sw, out):
    ws = torch.empty(g.q8_matmul_workspace_bytes(a.shape[0], w.shape[0], a.shape[1]), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    g.q8_matmul(a, sa, w, sw, out, ws)
    sync()


def check(a, sa, w, sw, out):
    aw, ww = a.cpu().numpy().astype(np.float64), w.cpu().numpy().astype(np.float64)
    saw, sww = sa.double().cpu().numpy(), sw.double().cpu().numpy()
    want = O.q8_matmul(aw, saw, ww, sww)
    size = np.abs(aw) @ np.abs(ww).T
    scale = np.abs(saw)[:, None] * np.abs(sww)
    tol = 4 * U * np.abs(want) + np.where(size >= 2.0 ** 24, a.shape[1] / 16 * 2 * U * size * scale, 0.0)
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    got = out.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


# single tokens; counts around 8, 16, a tile's and a wave's edges; odd K; one channel; long K
SHAPES = [(1, 1, 1), (1, 50257, 768), (2, 130, 64), (3, 5, 7), (5, 1000, 4100), (8, 257, 96), (9, 128, 128),
          (16, 4096, 1024), (17, 129, 65), (37, 300, 4096), (64, 64, 16), (100, 1, 333), (127, 383, 1000),
          (191, 255, 2048), (193, 1025, 48), (400, 700, 100), (513, 640, 513), (1000, 40, 8191), (33, 131, 20000)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_product(g, M, N, K, out):
    a, w, sa, sw = ints(M, K, 1), ints(N, K, 2), scales(M, 3), scales(N, 4)
    o = torch.full((M, N), float("nan"), device="cuda", dtype=DT[out])
    run(g, a, sa, w, sw, o)
    check(a, sa, w, sw, o)


@pytest.mark.parametrize("M,N,K", [(1, 300, 1024), (40, 300, 1024), (300, 300, 1024), (4, 140, 9000), (70, 140, 9000)])
def test_extreme_values(g, M, N, K):
    """All products of one sign and of the largest size: the sums reach (and, for K > 1024, pass) 2^24."""
    for va, vw in ((-128, -128), (127, -128), (127, 127)):
        a = torch.full((M, K), va, device="cuda", dtype=torch.int8)
        w = torch.full((N, K), vw, device="cuda", dtype=torch.int8)
        o = torch.empty(M, N, device="cuda")
        run(g, a, torch.ones(M, device="cuda"), w, torch.ones(N, device="cuda"), o)
        check(a, torch.ones(M), w, torch.ones(N), o)


@pytest.mark.parametrize("M,N,K", [(1, 77, 100), (6, 200, 130), (50, 333, 200), (260, 190, 96), (200, 200, 95)])
def test_strides_and_offsets(g, M, N, K):
    """Column slices of wider buffers at odd offsets, and an output between columns that stay."""
    ab, wb = ints(M, K + 37, 5), ints(N, K + 21, 6)
    sa, sw = scales(M + 1, 7)[1:], scales(N + 3, 8)[3:]
    for oa, ow in ((0, 0), (5, 3), (16, 16)):
        a, w = ab[:, oa:oa + K], wb[:, ow:ow + K]
        for dt in DT.values():
            buf = torch.full((M, N + 9), 3.0, device="cuda", dtype=dt)
            run(g, a, sa, w, sw, buf[:, 4:4 + N])
            check(a, sa, w, sw, buf[:, 4:4 + N])
            assert torch.all(buf[:, :4] == 3) and torch.all(buf[:, 4 + N:] == 3)


@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (30, 200, 256), (300, 200, 256)])
def test_bounds_of_buffers(g, M, N, K):
    """Guard bytes around the output and the workspace stay."""
    a, w, sa, sw = ints(M, K, 9), ints(N, K, 10), scales(M, 11), scales(N, 12)
    ob = torch.full((M * N + 512,), 3.0, device="cuda")
    need = g.q8_matmul_workspace_bytes(M, N, K)
    wsb = torch.full((need + 1024,), 90, dtype=torch.uint8, device="cuda")
    out = ob[256:256 + M * N].view(M, N)
    g.q8_matmul(a, sa, w, sw, out, wsb[512:512 + need])
    sync()
    check(a, sa, w, sw, out)
    assert torch.all(ob[:256] == 3) and torch.all(ob[256 + M * N:] == 3)
    assert torch.all(wsb[:512] == 90) and torch.all(wsb[512 + need:] == 90)


def test_empty_and_scales(g):
    a, w = ints(4, 0, 13), ints(6, 0, 14)
    o = torch.full((4, 6), 9.0, device="cuda")
    run(g, a, scales(4, 15), w, scales(6, 16), o)
    assert torch.all(o == 0)
    o = torch.full((70000, 3), 9.0, device="cuda", dtype=torch.bfloat16)         # more tokens than one launch's rows
    run(g, ints(70000, 0, 13), scales(70000, 15), ints(3, 0, 14), scales(3, 16), o)
    assert torch.all(o == 0)
    run(g, ints(0, 8, 17), scales(0, 1), ints(6, 8, 18), scales(6, 16), torch.empty(0, 6, device="cuda"))
    run(g, ints(4, 8, 17), scales(4, 1), ints(0, 8, 18), scales(0, 16), torch.empty(4, 0, device="cuda"))
    # a scale of 0, a negative one, and a NaN that stays in its token or channel
    for M in (3, 40, 200):
        a, w, sa, sw = ints(M, 64, 19), ints(50, 64, 20), scales(M, 21), scales(50, 22)
        sa[0], sw[1], sw[2] = 0.0, -1.0, float("nan")
        o = torch.empty(M, 50, device="cuda")
        run(g, a, sa, w, sw, o)
        assert torch.isnan(o[:, 2]).all() and torch.isfinite(o[:, :2]).all() and torch.isfinite(o[:, 3:]).all()
        assert torch.all(o[0, 3:] == 0)
        keep = [i for i in range(50) if i != 2]
        check(a, sa, w[keep], sw[keep], o[:, keep])


@pytest.mark.parametrize("M,N,K", [(1, 1000, 768), (20, 512, 2048), (300, 1000, 768)])
def test_other_stream_repeat_and_graph(g, M, N, K):
    a, w, sa, sw = ints(M, K, 23), ints(N, K, 24), scales(M, 25), scales(N, 26)
    ws = torch.empty(g.q8_matmul_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    o = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    g.q8_matmul(a, sa, w, sw, o, ws)
    sync()
    first, side = o.clone(), torch.cuda.Stream()
    o.zero_()
    sync()
    g.q8_matmul(a, sa, w, sw, o, ws, stream=side)
    sync()
    assert torch.equal(o, first)
    o.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.q8_matmul(a, sa, w, sw, o, ws)
    for _ in range(3):
        graph.replay()
    sync()
    assert torch.equal(o, first)


def test_offsets_past_32_bits(g):
    """An output of more than 2^32 bytes and 2^31 elements; its corners are checked."""
    M, N, K = 42800, 50257, 32
    a, w, sa, sw = ints(M, K, 27), ints(N, K, 28), scales(M, 29), scales(N, 30)
    o = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    run(g, a, sa, w, sw, o)
    rows = torch.tensor([0, 1, 21399, M - 200, M - 2, M - 1], device="cuda")
    check(a[rows], sa[rows], w, sw, o[rows])


def test_products_end_before_others_take_their_place(g):
    """Tile kernels of different rings one behind the other and among row kernels, with no wait between them: whatever
    a tile's CTAs still had under way when they end would land in the next one's shared memory and barriers."""
    shapes = [(300, 512, 64), (16, 4096, 1024), (513, 640, 200), (64, 300, 4096), (9, 256, 128), (1000, 257, 48)]
    calls = []
    for i, (M, N, K) in enumerate(shapes):
        a, w, sa, sw = ints(M, K, 40 + i), ints(N, K, 50 + i), scales(M, 60 + i), scales(N, 70 + i)
        ws = torch.empty(g.q8_matmul_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
        calls.append((a, sa, w, sw, torch.empty(M, N, device="cuda"), ws))
    x = torch.ones(600, 768, device="cuda")
    ys = [torch.empty_like(x) for _ in range(3)]
    sync()
    for r in range(12):
        for i in range(len(calls)):
            g.q8_matmul(*calls[(i * (1 + r % 2) + r) % len(calls)])
            if (i + r) % 3 == 0:
                g.rmsnorm_forward(x, None, ys[i % 3], 0.0)
    sync()
    for a, sa, w, sw, out, _ in calls:
        check(a, sa, w, sw, out)
    assert all(torch.equal(y, x) for y in ys)


@pytest.mark.parametrize("M,N,K", [(3, 640, 512), (24, 512, 1024), (40, 2048, 768), (700, 1000, 256)])
def test_operands_written_just_before(g, M, N, K):
    """Norm and product enqueued again and again into the same 8-bit rows and scales, the channels and their scales
    rewritten on the way: every product reads what the calls right before it wrote."""
    steps = 8
    xs = [torch.randn(M, K, device="cuda") * 4.0 ** i for i in range(steps)]
    ws_, sws = [ints(N, K, 80 + i) for i in range(2)], [scales(N, 82 + i) for i in range(2)]
    a, sa = torch.empty(M, K, device="cuda", dtype=torch.int8), torch.empty(M, device="cuda")
    w, sw = ws_[0].clone(), sws[0].clone()
    outs = [torch.empty(M, N, device="cuda") for _ in range(steps)]
    work = torch.empty(g.q8_matmul_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    sync()
    for i in range(steps):
        if i == steps // 2:
            w.copy_(ws_[1])
            sw.copy_(sws[1])
        g.rmsnorm_forward_q8(xs[i], None, a, sa, float(i))           # another eps, another scale, every time
        g.q8_matmul(a, sa, w, sw, outs[i], work)
    sync()
    for i in range(steps):
        g.rmsnorm_forward_q8(xs[i], None, a, sa, float(i))
        sync()
        check(a, sa, ws_[i >= steps // 2], sws[i >= steps // 2], outs[i])
