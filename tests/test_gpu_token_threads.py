"""First calls of the training step's operators from several threads at once, each on a stream of its own, in a fresh
process: what they write is what the same calls write one after another."""
import os
import subprocess
import sys

import pytest

from gpu_common import load_library

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys, threading
sys.path.insert(0, sys.argv[1])
sys.setswitchinterval(1e-6)
import torch
import gradient_sync_ddp_gb300 as g
torch.cuda.init()
n, T, D, V, K = 6, 300, 512, 5003, 9
errors, gate = [], threading.Barrier(n)

def inputs(i):
    r = torch.Generator(device="cuda").manual_seed(i)
    f = lambda *s: torch.randn(*s, device="cuda", generator=r)
    return dict(x=f(T, D), res=f(T, D), gamma=f(D), dy=f(T, D), z=f(T, V).bfloat16(), up=f(T),
                y=torch.randint(0, V, (T,), device="cuda", generator=r), m=[f(200, 136 + 8 * i) for _ in range(3)],
                grads=[f(40 + 3 * 24 * 56) for _ in range(2)], theta=f(40 + 3 * 24 * 56))

def outputs(i):
    e = lambda *s, **k: torch.empty(*s, device="cuda", **k)
    size = 40 + 3 * 24 * 56
    return dict(y=e(T, D), h=e(T, D), mean=e(T), rstd=e(T), dx=e(T, D), dg=e(D), db=e(D), p=e(T), ent=e(T), lse=e(T),
                ti=e(T, K, dtype=torch.int64), tl=e(T, K), dz=e(T, V, dtype=torch.bfloat16),
                o=[e(200, 136 + 8 * i) for _ in range(3)], theta=e(size), buf=torch.zeros(size, device="cuda"),
                ws=[e(max(b, 16), dtype=torch.uint8) for b in (g.layernorm_backward_workspace_bytes(T, D),
                    g.newton_schulz_workspace_bytes(3, 200, 136 + 8 * i), g.newton_schulz_workspace_bytes(3, 24, 56))])

def run(a, o):
    o["theta"].copy_(a["theta"])
    g.layernorm_forward(a["x"], a["gamma"], None, o["y"], residual=a["res"], h_out=o["h"], mean_out=o["mean"], rstd_out=o["rstd"])
    g.token_logprobs_forward(a["z"], a["y"], o["p"], o["ent"], o["lse"], o["ti"], o["tl"])
    g.token_logprobs_backward(a["z"], a["y"], o["lse"], a["up"], o["dz"], o["ent"], a["up"])
    g.layernorm_backward(a["dy"], o["h"], o["mean"], o["rstd"], a["gamma"], o["dx"], o["dg"], o["db"], o["ws"][0])
    g.newton_schulz(a["m"], o["o"], o["ws"][1])
    g.ddp_bucket_allreduce_muon(a["grads"], [0, 24 * 56, 40 + 2 * 24 * 56], 24, 56, o["theta"], o["buf"], o["ws"][2], 0.1, 0.9, 0.01)

a, at_once, in_turn = [inputs(i) for i in range(n)], [outputs(i) for i in range(n)], [outputs(i) for i in range(n)]
torch.cuda.synchronize()

def work(i):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            gate.wait()
            run(a[i], at_once[i])
    except BaseException as e:
        errors.append(repr(e))

threads = [threading.Thread(target=work, args=(i,)) for i in range(n)]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
assert not errors, errors
for i in range(n):
    run(a[i], in_turn[i])
torch.cuda.synchronize()
bits = lambda t: t.contiguous().view(torch.uint8)
for i in range(n):
    for name, want in in_turn[i].items():
        if name == "ws":
            continue
        for p, q in zip(at_once[i][name], want) if name == "o" else [(at_once[i][name], want)]:
            assert torch.equal(bits(p), bits(q)), (i, name)
        assert all(torch.isfinite(q.float()).all() for q in (want if name == "o" else [want])), (i, name)
print("ok")
"""


def test_first_calls_of_six_threads():
    load_library()
    r = subprocess.run([sys.executable, "-c", PROGRAM, ROOT], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]


WIDTHS = """
import sys, threading
sys.path.insert(0, sys.argv[1])
sys.setswitchinterval(1e-6)
import torch
import gradient_sync_ddp_gb300 as g
torch.cuda.init()
errors, gate, widths = [], threading.Barrier(6), [800, 1024, 904, 1000, 864, 960]
f = lambda *s, **k: torch.randn(*s, device="cuda", **k)
sets = [(f(400, D, dtype=torch.bfloat16), f(400, D, dtype=torch.bfloat16), f(400), f(400).abs(), f(D),
         torch.empty(400, D, device="cuda", dtype=torch.bfloat16), f(D), f(D),
         torch.empty(max(g.layernorm_backward_workspace_bytes(400, D), g.rmsnorm_backward_workspace_bytes(400, D)),
                     device="cuda", dtype=torch.uint8)) for D in widths]
torch.cuda.synchronize()

def work(i):
    dy, h, mean, rstd, gamma, dx, dg, db, ws = sets[i]
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            gate.wait()
            for _ in range(1500):
                g.rmsnorm_backward(dy, h, rstd, gamma, dx, dg, ws)
            g.layernorm_backward(dy, h, mean, rstd, gamma, dx, dg, db, ws)
    except BaseException as e:
        errors.append(repr(e))

threads = [threading.Thread(target=work, args=(i,)) for i in range(6)]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
assert not errors, errors
print("ok")
"""


def test_widths_of_one_kernel_at_once():
    """Calls of one kernel that take different amounts of shared memory, at once: none lowers what another is allowed."""
    load_library()
    r = subprocess.run([sys.executable, "-c", WIDTHS, ROOT], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]
