"""Calls of the packed-layer blocks from several threads at once, the very first ones of a process among them (GPU)."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import threading
import torch
from diffusion_transformer_denoiser_dit_b200 import Rotary, attention_packed, linear_fused

g = torch.Generator(device="cuda").manual_seed(0)
x = torch.randn(600, 256, device="cuda", generator=g).bfloat16()
w = torch.randn(512, 256, device="cuda", generator=g).bfloat16()
big = torch.cat([x] * 9)
q = x.unflatten(1, (4, 64))
cu, one, pos = torch.tensor([0, 600], device="cuda").int(), torch.tensor([0, 1], device="cuda").int(), torch.arange(600, device="cuda")
rot = Rotary(64)
calls = [lambda: linear_fused(x, w), lambda: linear_fused(big, w, out_dtype=torch.float32), lambda: linear_fused(x[:1], w),
         lambda: linear_fused(x[:, 1:251], w[:, 1:251]), lambda: attention_packed(q, q, q, cu, cu, 600, 600, causal=True),
         lambda: attention_packed(q[:1], q, q, one, cu, 1, 600), lambda: rot.apply(q, pos), lambda: linear_fused(x.half(), w.half())]
torch.cuda.synchronize()
got, start, errors = [None] * 16, threading.Barrier(16), []

def work(i):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            got[i] = [calls[(i + n) % len(calls)]() for n in range(len(calls))]
            torch.cuda.current_stream().synchronize()
    except BaseException as e:
        errors.append(repr(e))

threads = [threading.Thread(target=work, args=(i,)) for i in range(16)]
for t in threads: t.start()
for t in threads: t.join()
assert not errors, errors
want = [c() for c in calls]
for i in range(16):
    for n in range(len(calls)):
        assert torch.equal(got[i][n], want[(i + n) % len(calls)]), (i, n)
print("same")
"""


def test_first_calls_from_many_threads():
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=200)
        assert r.returncode == 0 and "same" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]
