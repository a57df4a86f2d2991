"""First calls from many threads at once: whichever comes last, every later call of every shape still launches."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

# Shapes whose launches take different amounts of shared memory, so that the threads' first calls raise
# the kernels' limits in any order (the C calls release the interpreter's lock).
CODE = """
import threading, torch
import bit_quantized_linear_q8_gb300 as B

dev = "cuda"
k = 4096
jobs = []
one = torch.ones(4096, device=dev)
for m, n in ((1, 64), (16, 4096), (40, 512), (48, 4096), (64, 130), (80, 4096), (100, 300), (128, 2048),
             (129, 64), (160, 4096), (200, 512), (256, 4096), (300, 130), (384, 640), (500, 4096), (700, 2048)):
    a = torch.ones((m, k), dtype=torch.int8, device=dev)
    w = torch.ones((n, k), dtype=torch.int8, device=dev)
    jobs.append((lambda a=a, w=w, m=m, n=n: B.int8_gemm(a, one[:m], w, one[:n]), float(k)))
for group in (128, 512):
    for n, kk in ((96, 512), (256, 4096), (1024, 8192)):
        # codes of 1 with scales of one: the value that the packed weight expands to
        q2 = B.q2_pack(torch.ones((n, kk), dtype=torch.uint8, device=dev),
                       torch.ones((n, kk // group), dtype=torch.bfloat16, device=dev), group)
        value = B.dequant_q2_to_bf16(q2)[0, 0].item()
        for m in (1, 2, 4, 8):
            x = torch.ones((m, kk), dtype=torch.bfloat16, device=dev)
            jobs.append((lambda x=x, q2=q2: B.q2_gemv_batchm(x, q2), value * kk))
torch.cuda.synchronize()
start = threading.Barrier(len(jobs))
errors = []

def run(f, want):
    start.wait()
    try:
        for _ in range(3):
            out = f()
        torch.cuda.synchronize()
        if not bool((out.float() == want).all()):
            errors.append("values")
    except Exception as e:
        errors.append(str(e))

for attempt in range(2):  # the first calls, then every shape again
    threads = [threading.Thread(target=run, args=j) for j in jobs]
    [t.start() for t in threads]
    [t.join() for t in threads]
assert not errors, errors
print("ok")
"""


def test_first_calls_from_many_threads():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
