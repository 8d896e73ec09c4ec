"""The first calls of a process from several threads at once, each with its own stream and buffers, have the bits of later ones."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()

CHILD = """
import threading, torch
import activation_sparse_transformer_tcgen05_gb300 as tw

BF, SIZES = torch.bfloat16, [(512, 2048, 2048), (256, 1024, 4096), (777, 264, 2696), (300, 1024, 1024), (3, 520, 2048), (64, 1000, 4096)]

class Work:
    def __init__(self, i):
        M, N, K = SIZES[i % len(SIZES)]
        g = torch.Generator(device="cuda").manual_seed(i)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(BF)
        self.x, self.W, self.dy = rand(M, K), rand(N, K), rand(M, N)
        self.out = [torch.empty(M, N, device="cuda", dtype=BF), torch.empty(M, K, device="cuda", dtype=BF), torch.empty(N, K, device="cuda")]
        self.ws = torch.empty(tw.twell_linear_bwd_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
        self.st, self.stream = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cuda.Stream()

    def run(self):
        y, dx, dW = self.out
        tw.twell_linear_fwd(self.x, self.W, False, None, tw.ACT_NONE, None, None, y, self.st, stream=self.stream)
        tw.twell_linear_bwd(self.dy, self.x, self.W, False, tw.ACT_NONE, None, dx, dW, False, None, self.ws, self.st, stream=self.stream)

works = [Work(i) for i in range(12)]
torch.cuda.synchronize()
start = threading.Barrier(len(works))
errors = []

def body(w):
    try:
        start.wait()
        w.run()
    except Exception as e:
        errors.append(e)

threads = [threading.Thread(target=body, args=(w,)) for w in works]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not errors, errors
first = [[t.clone() for t in w.out] for w in works]
for w, was in zip(works, first):
    for t in w.out:
        t.fill_(5)
    torch.cuda.synchronize()
    w.run()
    torch.cuda.synchronize()
    assert tw.twell_check(w.st) == 0
    assert all(torch.equal(a, b) for a, b in zip(w.out, was))
print("same")
"""


def test_first_calls_of_a_process():
    for _ in range(2):
        r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300,
                           cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
        assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
