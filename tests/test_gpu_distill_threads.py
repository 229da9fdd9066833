"""First calls of the distillation operators from several threads at once, in a fresh process."""
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
n, errors, gate = 8, [], threading.Barrier(8)
x = [torch.full((40, 512), float(i + 1), device="cuda") for i in range(n)]
y = [torch.empty_like(v) for v in x]
rstd = [torch.empty(40, device="cuda") for _ in x]
q = [torch.empty(40, 512, dtype=torch.int8, device="cuda") for _ in x]
scale = [torch.empty(40, device="cuda") for _ in x]
torch.cuda.synchronize()

def work(i):
    try:
        gate.wait()
        g.rmsnorm_forward(x[i], None, y[i], 0.0, rstd_out=rstd[i])
        g.rmsnorm_forward_q8(x[i], None, q[i], scale[i], 0.0)
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
    assert torch.all((y[i] - 1).abs() <= 2e-6) and torch.all((rstd[i] * (i + 1) - 1).abs() <= 2e-6)
    assert torch.all(q[i] == 127) and torch.all((scale[i] * 127 - 1).abs() <= 2e-6)
print("ok")
"""


def test_first_calls_of_eight_threads():
    load_library()
    r = subprocess.run([sys.executable, "-c", PROGRAM, ROOT], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]
