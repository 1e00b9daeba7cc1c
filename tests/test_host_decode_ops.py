"""The host-side checks of the paged-cache calls and the 4-bit product (no GPU, no launch):
every refusal with its own code and a message that names the value, and what the binding
refuses before a pointer reaches the library."""
from __future__ import annotations

import ctypes

import pytest
import torch

import fp8_weight_only_gemm_gb300 as w8
from fp8_weight_only_gemm_gb300 import binding
from fp8_weight_only_gemm_gb300.build import build_library

M_ZERO, K_BLOCK, PITCH, A_PITCH, N_ZERO, NULL, ALIGN, RANGE, DEVICE, ARG = -1, -2, -3, -4, -5, -6, -7, -8, -9, -13
P = 0x10000   # a placeholder: every call here is refused before it is used


@pytest.fixture(scope="module")
def lib():
    build_library()
    return binding.load()


def cache(**over):
    d = dict(k_codes=P, v_codes=P, k_scale=P, v_scale=P, page_stride=64 * 128, head_stride=64 * 128 * 9, token_stride=128,
             scale_page_stride=2, scale_head_stride=1, num_pages=9, page_size=64, kv_heads=2, head_dim=128)
    d.update(over)
    return binding.KvCacheDesc(*(d[f] for f, _ in binding.KvCacheDesc._fields_))


def batch(**over):
    d = dict(page_table=P, lens=P, cu_q=None, page_table_stride=4, max_pages=4, batch=3, tokens=6, max_q=2)
    d.update(over)
    return binding.KvBatchDesc(*(d[f] for f, _ in binding.KvBatchDesc._fields_))


def heads(n=2, ptr=P, token=256, head=128):
    return binding.HeadsDesc(ptr, token, head, n)


def rope(**over):
    d = dict(cos=P, sin=P, rows=100, rotary_dim=64, interleaved=0)
    d.update(over)
    return binding.RopeDesc(*(d[f] for f, _ in binding.RopeDesc._fields_))


def append(lib, c=None, b=None, act=0, k=None, v=None, q=None, q_out=None, r=None):
    ref = lambda x: None if x is None else ctypes.byref(x)
    return lib.w8a16_kv_append(ref(c or cache()), ref(b or batch()), act, ref(k or heads()), ref(v or heads()), ref(q), ref(q_out),
                               ref(r or rope()), None)


def attention(lib, c=None, b=None, act=0, q=None, out=None, scale=0.1, ws=P, ws_bytes=1 << 40):
    return lib.w8a16_kv_attention(ctypes.byref(c or cache()), ctypes.byref(b or batch()), act, ctypes.byref(q or heads(8, token=1024)),
                                  ctypes.byref(out or heads(8, token=1024)), scale, ws, ws_bytes, None)


CACHE_AND_BATCH = [
    (dict(c=dict(k_codes=None)), NULL, "NULL cache pointer"),
    (dict(c=dict(head_dim=8)), ARG, "head_dim=8"),
    (dict(c=dict(head_dim=136)), ARG, "head_dim=136"),
    (dict(c=dict(head_dim=272)), ARG, "head_dim=272"),
    (dict(c=dict(page_size=48)), ARG, "page_size=48"),
    (dict(c=dict(page_size=512)), ARG, "page_size=512"),
    (dict(c=dict(kv_heads=0)), ARG, "kv_heads=0"),
    (dict(c=dict(num_pages=0)), RANGE, "num_pages=0"),
    (dict(c=dict(v_codes=P + 8)), ALIGN, "16-byte"),
    (dict(c=dict(token_stride=136)), ALIGN, "strides"),
    (dict(c=dict(head_stride=-16)), RANGE, "negative"),
    (dict(c=dict(token_stride=(1 << 22) + 16)), RANGE, "2^22"),
    (dict(b=dict(batch=0)), M_ZERO, "batch=0"),
    (dict(b=dict(tokens=0)), M_ZERO, "tokens=0"),
    (dict(b=dict(lens=None)), NULL, "lens"),
    (dict(b=dict(page_table=P + 2)), ALIGN, "page_table"),
    (dict(b=dict(max_q=7, cu_q=P)), RANGE, "max_q=7"),
    (dict(b=dict(tokens=7)), ARG, "tokens=7"),
    (dict(b=dict(max_pages=0)), RANGE, "max_pages=0"),
    (dict(b=dict(max_pages=1 << 26)), RANGE, "max_pages"),
]


@pytest.mark.parametrize("over,code,needle", CACHE_AND_BATCH)
@pytest.mark.parametrize("call", [append, attention])
def test_cache_and_batch(lib, call, over, code, needle):
    kw = {k: (cache if k == "c" else batch)(**v) for k, v in over.items()}
    assert call(lib, **kw) == code
    assert needle in binding.last_error()


@pytest.mark.parametrize("kw,code,needle", [
    (dict(act=7), ARG, "activation type 7"),
    (dict(k=heads(3)), ARG, "k has 3 heads, not 2"),
    (dict(v=heads(ptr=None)), NULL, "v is NULL"),
    (dict(k=heads(token=260)), ALIGN, "k needs"),
    (dict(q=heads(8, token=1024)), NULL, "q_out is NULL"),
    (dict(q=heads(8, token=1024), q_out=heads(4, token=1024)), ARG, "q_out has 4 heads, not 8"),
    (dict(q_out=heads(8, token=1024)), NULL, "q_out without q"),
    (dict(r=rope(rotary_dim=24)), ARG, "rotary_dim=24"),
    (dict(r=rope(rotary_dim=144)), ARG, "rotary_dim=144"),
    (dict(r=rope(sin=None)), NULL, "sin"),
    (dict(r=rope(cos=P + 4)), ALIGN, "cos"),
    (dict(r=rope(rows=0)), RANGE, "rows=0"),
])
def test_append(lib, kw, code, needle):
    assert append(lib, **kw) == code
    assert needle in binding.last_error()


@pytest.mark.parametrize("kw,code,needle", [
    (dict(act=2), ARG, "activation type 2"),
    (dict(q=heads(7, token=1024), out=heads(7, token=1024)), ARG, "7 query heads"),
    (dict(out=heads(4, token=1024)), ARG, "out has 4 heads, not 8"),
    (dict(scale=0.0), ARG, "softmax_scale"),
    (dict(scale=float("nan")), ARG, "softmax_scale"),
    (dict(scale=float("inf")), ARG, "softmax_scale"),
])
def test_attention(lib, kw, code, needle):
    assert attention(lib, **kw) == code
    assert needle in binding.last_error()


def w4(lib, A=P, lda=256, act=0, W=P, scale=P, sdt=0, zeros=None, group=64, C=P, ldc=96, M=2, N=96, K=256, flags=0):
    return lib.w8a16_gemm_w4(A, lda, act, W, scale, sdt, zeros, group, C, ldc, M, N, K, flags, None)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(flags=8), ARG, "flag bits 8"),
    (dict(M=0), M_ZERO, "m=0"),
    (dict(group=16), ARG, "group=16"),
    (dict(K=0), K_BLOCK, "K=0"),
    (dict(K=224), K_BLOCK, "K=224"),
    (dict(lda=255), PITCH, "a=255"),
    (dict(ldc=95), PITCH, "c=95"),
    (dict(lda=260), A_PITCH, "a_row_stride=260"),
    (dict(N=0), N_ZERO, "n=0"),
    (dict(M=1 << 31), RANGE, "out of range"),
    (dict(N=1 << 29, ldc=1 << 29), RANGE, "out of range"),
    (dict(act=9), ARG, "activation type 9"),
    (dict(sdt=5), ARG, "scale type 5"),
    (dict(W=None), NULL, "NULL"),
    (dict(A=P + 8), ALIGN, "alignment"),
    (dict(zeros=P + 1), ALIGN, "alignment"),
])
def test_gemm_w4(lib, kw, code, needle):
    assert w4(lib, **kw) == code
    assert needle in binding.last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are placeholders that no GPU may be given")
def test_well_formed_calls_without_a_device_are_errors(lib):
    assert append(lib) == DEVICE and attention(lib) == DEVICE and w4(lib) == DEVICE
    assert lib.w8a16_kv_attention_workspace_bytes(ctypes.byref(cache()), 3, 2, 8) == 0


def test_binding_refuses_host_tensors(lib):
    kv = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    s = torch.zeros(4, 2)
    with pytest.raises(ValueError):
        w8.KVCache(kv, kv, s, s)
    A, W, scale = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.uint8), torch.ones(8, 2)
    with pytest.raises(ValueError, match="CUDA"):
        w8.gemm_w4(A, W, scale)
    with pytest.raises(TypeError):
        w8.gemm_w4(A.float(), W, scale, torch.empty(2, 8))
    with pytest.raises(ValueError, match="W must be"):
        w8.gemm_w4(A, W[:, :31], scale)
    with pytest.raises(ValueError, match="scale"):
        w8.gemm_w4(A, W, scale[:5])
    with pytest.raises(TypeError, match="scale"):
        w8.gemm_w4(A, W, scale.half())
    with pytest.raises(ValueError, match="zeros"):
        w8.gemm_w4(A, W, scale, zeros=torch.zeros(8, 2))
    with pytest.raises(ValueError, match="C must be"):
        w8.gemm_w4(A, W, scale, torch.empty(2, 7, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="tensor"):
        w8.gemm_w4(A, W, None, torch.empty(2, 8, dtype=torch.bfloat16))
