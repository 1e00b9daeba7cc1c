"""Guard bands around what the decode-step operators write (the stand-in for a memory checker):
outputs, cache pages and scales, and workspaces of exactly the stated size live in the middle of
larger buffers whose bands hold a fixed pattern, checked byte for byte after the calls, with the
rows' and pages' own gaps. An output that a call leaves unwritten shows as a difference between two
calls (they are deterministic) into buffers with different patterns. Inputs must come back as they were, and the status must be clear."""
from __future__ import annotations

import pytest
import torch

from test_gpu_guard import _bands_intact, _guarded

pytestmark = pytest.mark.gpu
FILLS = (0x5A, 0xA5)


@pytest.fixture(scope="module")
def w8():
    import fp8_weight_only_gemm_gb300 as w8
    from fp8_weight_only_gemm_gb300.build import build_library
    build_library()
    w8.load()
    w8.device_status(clear=True)
    return w8


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", [(1, 67, 384), (2, 4097, 640), (8, 300, 2048), (16, 129, 1024), (31, 1000, 512), (33, 9763, 1664), (16, 9763, 640)])
def test_gemm_w4(w8, M, N, K, dtype, group):
    g = torch.Generator("cuda").manual_seed(M + N + K)
    A = torch.randn(M, K + 24, generator=g, device="cuda").to(dtype)
    W = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    S = torch.rand(N, K // group, generator=g, device="cuda").to(dtype)
    Z = torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8, device="cuda")
    inputs = [t.clone() for t in (A, W, S, Z)]
    ldc = N + 5
    for zeros in (None, Z):
        for flags in (0, w8.FLAG_PDL):
            got = []
            for fill in FILLS:
                buf, v = _guarded(M * ldc * 2, fill)
                C = v.view(dtype).view(M, ldc)
                w8.gemm_w4(A[:, :K], W, S, C[:, :N], zeros=zeros, flags=flags)
                torch.cuda.synchronize()
                assert _bands_intact(buf, M * ldc * 2, fill), "wrote outside C"
                assert bool((C[:, N:].contiguous().view(torch.uint8) == fill).all()), "wrote the gaps of C's rows"
                got.append(C[:, :N].contiguous().view(torch.int16))
            assert torch.equal(*got), "left outputs unwritten"
    assert all(torch.equal(a, b) for a, b in zip(inputs, (A, W, S, Z)))
    assert w8.device_status(clear=True)[0] == 0


def guarded_cache(w8, pages, P, H, D, gap, seed):
    """A cache whose pages have `gap` unused bytes behind each token, its buffers and their views."""
    g = torch.Generator("cuda").manual_seed(seed)
    bufs, views = [], []
    for _ in range(2):
        n = pages * H * P * (D + gap)
        buf, v = _guarded(n)
        v.copy_(torch.randint(0, 0x7E, (n,), generator=g, dtype=torch.uint8, device="cuda"))
        bufs.append((buf, n))
        views.append(v.view(pages, H, P, D + gap))
    for _ in range(2):
        buf, v = _guarded(pages * H * 4)
        s = v.view(torch.float32).view(pages, H)
        s.copy_(2.0 ** torch.randint(-9, -5, (pages, H), generator=g, device="cuda").float())
        bufs.append((buf, pages * H * 4))
        views.append(s)
    cache = w8.KVCache(views[0][..., :D], views[1][..., :D], views[2], views[3])
    return cache, bufs, views


LENS, COUNTS = [1, 16, 130, 77, 0, 300], [1, 5, 33, 0, 2, 17]


def sequences(P, seed):
    used = [max(1, -(-n // P)) for n in LENS]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.zeros(len(LENS), max(used), dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    cu = torch.tensor([0] + COUNTS).cumsum(0).to(torch.int32)
    return pages, table, cu


@pytest.mark.parametrize("D,gap,P,Hq,H,dtype", [(128, 0, 16, 8, 2, torch.bfloat16), (64, 16, 32, 3, 3, torch.float16), (80, 48, 64, 4, 1, torch.bfloat16),
                                                 (256, 0, 16, 2, 2, torch.float16)])
def test_kv_append(w8, D, gap, P, Hq, H, dtype):
    pages, table, cu = sequences(P, D)
    cache, bufs, views = guarded_cache(w8, pages, P, H, D, gap, D)
    before = [v.clone() for v in views]
    g = torch.Generator("cuda").manual_seed(D)
    n = int(cu[-1])
    q, k, v = (torch.randn(n, h, D, generator=g, device="cuda").to(dtype) for h in (Hq, H, H))
    cos, sin = (torch.rand(300, D // 2, generator=g, device="cuda") for _ in range(2))
    inputs = [t.clone() for t in (q, k, v, cos, sin)]
    nbytes = n * Hq * (D + 8) * 2
    qbuf, qv = _guarded(nbytes)
    qo = qv.view(dtype).view(n, Hq, D + 8)
    w8.kv_append(cache, k, v, table.cuda(), torch.tensor(LENS, dtype=torch.int32).cuda(), cos, sin, q=q, q_out=qo[..., :D], cu_q=cu.cuda(),
                 max_q=max(COUNTS))
    torch.cuda.synchronize()
    assert _bands_intact(qbuf, nbytes) and bool((qo[..., D:].contiguous().view(torch.uint8) == 0x5A).all())
    for (buf, size) in bufs:
        assert _bands_intact(buf, size)
    assert all(torch.equal(a, b) for a, b in zip(inputs, (q, k, v, cos, sin)))
    # slots and scales that may change: the new tokens', and older ones in the page where they begin
    slots = torch.zeros(pages, P, dtype=torch.bool)
    for b, (length, count) in enumerate(zip(LENS, COUNTS)):
        first = max(length - count, 0)
        if first < length:
            for pos in range(first // P * P, length):
                slots[int(table[b, pos // P]), pos % P] = True
    touched = slots.any(1).cuda()
    slots = slots.cuda()
    for old, new in zip(before[:2], views[:2]):
        same = (old == new).transpose(1, 2)                       # [pages, P, H, D + gap]
        assert bool(same[~slots].all()), "wrote slots of other tokens"
        assert bool(same[..., D:].all()), "wrote the gaps between tokens"
    for old, new in zip(before[2:], views[2:]):
        assert bool((old == new)[~touched].all()), "wrote scales of other pages"
    assert w8.device_status(clear=True)[0] == 0


@pytest.mark.parametrize("D,gap,P,Hq,H,dtype", [(128, 0, 16, 4, 4, torch.bfloat16), (128, 16, 64, 32, 4, torch.bfloat16), (64, 0, 32, 2, 2, torch.float16),
                                                 (80, 48, 16, 8, 1, torch.float16), (256, 0, 16, 2, 1, torch.bfloat16), (16, 0, 128, 6, 2, torch.float16)])
@pytest.mark.parametrize("tokens", ["one", "ragged"])
def test_kv_attention(w8, D, gap, P, Hq, H, dtype, tokens):
    pages, table, cu = sequences(P, D)
    cache, bufs, views = guarded_cache(w8, pages, P, H, D, gap, D)
    before = [v.clone() for v in views]
    g = torch.Generator("cuda").manual_seed(D + Hq)
    most = 1 if tokens == "one" else max(COUNTS)
    n = len(LENS) if tokens == "one" else int(cu[-1])
    q = torch.randn(n, Hq, D, generator=g, device="cuda").to(dtype)
    q0 = q.clone()
    nbytes = n * Hq * (D + 8) * 2
    need = w8.kv_attention_workspace_bytes(cache, len(LENS), most, Hq)
    rows = {} if tokens == "one" else {"cu_q": cu.cuda(), "max_q": most}
    got = []
    for fill in FILLS:
        obuf, ov = _guarded(nbytes, fill)
        out = ov.view(dtype).view(n, Hq, D + 8)
        wbuf, ws = _guarded(need, fill)
        w8.kv_attention(cache, q, table.cuda(), torch.tensor(LENS, dtype=torch.int32).cuda(), out[..., :D], workspace=ws, **rows)
        torch.cuda.synchronize()
        assert _bands_intact(obuf, nbytes, fill), "wrote outside the outputs"
        assert _bands_intact(wbuf, need, fill), "wrote outside the workspace"
        assert bool((out[..., D:].contiguous().view(torch.uint8) == fill).all()), "wrote the gaps of the outputs' rows"
        got.append(out[..., :D].contiguous().view(torch.int16))
    assert torch.equal(*got), "left rows unwritten"
    assert torch.equal(q, q0) and all(torch.equal(a, b) for a, b in zip(before, views))
    for (buf, size) in bufs:
        assert _bands_intact(buf, size)
    assert w8.device_status(clear=True)[0] == 0
