"""Tensors that have no memory to point to (the values that torch.vmap hands to its function) are
refused with a Python error by the calls that ask their tensors in C++. In a child process: where
the error is raised without the interpreter's lock, the process dies."""
from __future__ import annotations

import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parents[1]

CHILD = r"""
import sys, threading
import torch
sys.path.insert(0, sys.argv[1])
import fp8_weight_only_gemm_gb300 as w8

w8.load()
bf = dict(dtype=torch.bfloat16, device="cuda")
W = torch.zeros(64, 128, dtype=torch.uint8, device="cuda")
S = torch.zeros(64, 4, device="cuda")
C = torch.zeros(2, 64, **bf)
cache = w8.KVCache.empty(4, 16, 1, 64)
table, lens = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
out = torch.zeros(2, 2, 64, **bf)
ws = torch.empty(w8.kv_attention_workspace_bytes(cache, 2, 1, 2), dtype=torch.uint8, device="cuda")
k = torch.zeros(2, 1, 64, **bf)

calls = {
    "gemm_w4": (lambda x: w8.gemm_w4(x, W, S, C), torch.zeros(3, 2, 256, **bf)),
    "kv_attention": (lambda x: w8.kv_attention(cache, x, table, lens, out, workspace=ws), torch.zeros(3, 2, 2, 64, **bf)),
    "kv_append": (lambda x: w8.kv_append(cache, x, k, table, lens), torch.zeros(3, 2, 1, 64, **bf)),
}
call, x = calls[sys.argv[2]]
stop = threading.Event()
busy = threading.Thread(target=lambda: [sum(range(100)) for _ in iter(stop.is_set, True)])   # wants the lock all the time
busy.start()
try:
    for _ in range(100):
        try:
            torch.vmap(call)(x)
        except RuntimeError as e:
            assert "storage" in str(e) or "data pointer" in str(e), e
        else:
            raise AssertionError("not refused")
finally:
    stop.set()
    busy.join()
print("refused")
"""


@pytest.mark.parametrize("name", ["gemm_w4", "kv_attention", "kv_append"])
def test_tensors_without_memory_are_refused(name):
    from fp8_weight_only_gemm_gb300.build import build_library
    build_library()
    r = subprocess.run([sys.executable, "-c", CHILD, str(ROOT), name], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("refused"), (r.returncode, r.stdout[-2000:] + r.stderr[-3000:])
