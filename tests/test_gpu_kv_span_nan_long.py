"""NaN values among many keys of a window or a shared prefix: the rows that see them get them and no others, and marking them takes
less than the other warps' waits may last (40 ms here, in a child process), also where an item has a hundred units of keys and
all of them hold one. Against the same call with finite values in their places: what is not NaN has the same bits."""
from __future__ import annotations

import json
import os
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parents[1]

CHILD = r"""
import json, sys
import torch
sys.path.insert(0, sys.argv[1])
import fp8_weight_only_gemm_gb300 as w8

w8.load()
w8.device_status(clear=True)
P, results = 64, []

def run(name, lens, T, Hq, Hkv, D, spots, prefix=0, window=None, sinks=0):
    # spots: (sequence, position, dim) of a NaN value; those of the prefix are every sequence's
    g = torch.Generator("cuda").manual_seed(len(lens) + T)
    B, first = len(lens), prefix // P if prefix else 0
    width = -(-max(lens) // P)
    own = [max(0, -(-n // P) - first) for n in lens]
    shared = -(-prefix // P)
    total = shared + sum(own)
    cache = w8.KVCache.empty(total, P, Hkv, D)
    for c in (cache.k_codes, cache.v_codes):
        for i in range(0, total, 256):
            c[i:i + 256] = (torch.randn(c[i:i + 256].shape, generator=g, device="cuda") * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    cache.k_scale.fill_(2.0 ** -8), cache.v_scale.fill_(2.0 ** -6)
    table, at = torch.full((B, width), -1, dtype=torch.int32), shared
    for b in range(B):
        table[b, first:first + own[b]] = torch.arange(at, at + own[b])
        at += own[b]
    pages = torch.arange(shared, dtype=torch.int32, device="cuda")
    q = torch.randn(B * T, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    kw = dict(prefix_pages=pages, prefix_len=prefix) if prefix else dict(window=window, sinks=sinks)
    args = (cache, q, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    clean = w8.kv_attention(*args, **kw)
    want = torch.zeros(B * T, D, dtype=torch.bool)
    for b, pos, d in spots:
        page = pos // P if pos < prefix else int(table[b, pos // P])
        cache.v_codes[page, :, pos % P, d] = 0x7F if pos % 2 else 0xFF
        for s in range(B) if pos < prefix else (b,):
            p = torch.arange(lens[s] - T, lens[s])
            want[s * T:(s + 1) * T, d] |= (pos <= p) & ((pos > p - window) | (pos < sinks) if window else True)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    got = w8.kv_attention(*args, **kw)
    end.record()
    torch.cuda.synchronize()
    nan = got.isnan()
    results.append(dict(name=name, status=w8.device_status(clear=True)[0], nan=torch.equal(nan.cpu(), want[:, None].expand(-1, Hq, -1)),
                        bits=torch.equal(got.masked_fill(nan, 0), clean.masked_fill(nan, 0)), marked=int(want.sum()), ms=begin.elapsed_time(end)))

L = 8000
lens = [3000] + [L + 9 + 3 * i for i in range(39)]
few = [(0, 2990, 1), (0, 0, 2), (1, L - 1, 3), (2, L + 2, 4)]
many = [(0, i, i % 63) for i in range(5, L, 97)]
for T, what in ((8, "the kernel for few rows behind it"), (12, "the kernel for many")):
    run(f"prefix, one value, {what}", lens, T, 256, 32, 64, few[:1], prefix=L)
    run(f"prefix, {what}", lens, T, 256, 32, 64, few, prefix=L)
    run(f"prefix, all units, {what}", lens, T, 256, 32, 64, many, prefix=L)
n, W = 24000, 20000
for D, Hkv in ((64, 32), (128, 24)):
    spots = [(0, n - 5, 0), (0, n - 590, 7), (0, n - W - 300, 8), (0, n - W - 2, 9), (0, 100, 10), (0, 3, 11), (0, n - 10000, 12)]
    run(f"window, {D}", [n], 600, 4 * Hkv, Hkv, D, spots, window=W, sinks=70)
    run(f"window, one value, {D}", [n], 600, 4 * Hkv, Hkv, D, spots[1:2], window=W, sinks=70)
    run(f"window of everything, {D}", [n], 600, 4 * Hkv, Hkv, D, spots[:3], window=1 << 30)
print(json.dumps(results))
"""


def test_nan_among_many_keys():
    from fp8_weight_only_gemm_gb300.build import build_library
    build_library()
    env = dict(os.environ, W8A16_WAIT_TIMEOUT_MS="40")
    r = subprocess.run([sys.executable, "-c", CHILD, str(ROOT)], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    results = json.loads(r.stdout.strip().splitlines()[-1])
    assert len(results) == 12
    for x in results:
        assert x["status"] == 0 and x["nan"] and x["bits"] and x["marked"] > 0, x
