"""Appending to the 8-bit paged cache against the plain 64-bit form.

Tolerances, from the arithmetic: the kernel rotates in FP32 with three roundings per
element (two products, one sum of terms up to |a| + |b| with |cos|, |sin| <= 1), so a
rotated value is off by at most 2^-22 (|a| + |b|). Queries then round once to the
activation type (unit roundoff 2^-p of a p-bit significand: 2^-8 for BF16, 2^-11 for
FP16, relative). A code may
differ from the 64-bit form's only where the value lies within that rotation error of
the midpoint between two codes: then it is the neighbouring code. Page scales are powers
of two and must be equal (the inputs keep every page maximum away from 448 * 2^n by more
than the error). Values are not rotated: their codes and scales are equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def w8():
    import fp8_weight_only_gemm_gb300 as w8
    from fp8_weight_only_gemm_gb300.build import build_library
    build_library()
    w8.load()
    w8.device_status(clear=True)
    yield w8
    assert w8.device_status(clear=True)[0] == 0


class Case:
    """Random cache, page table (pages in random order), and ragged rows."""

    def __init__(self, lens, counts, Hq, Hkv, D, P, dtype, seed, slot_major=False, fused=False, spread=False):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.counts, self.D, self.P, self.dtype = lens, counts, D, P, dtype
        self.cu = np.concatenate([[0], np.cumsum(counts)]).tolist()
        N = self.cu[-1]
        used = [max(1, -(-n // P)) for n in lens]
        pages = sum(used) + 2
        order = torch.randperm(pages, generator=g).tolist()
        self.table = np.zeros((len(lens), max(used)), dtype=np.int32)
        for b, n in enumerate(used):
            self.table[b, :n] = [order.pop() for _ in range(n)]
        shape = (pages, P, Hkv, D) if slot_major else (pages, Hkv, P, D)

        def codes():
            c = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)     # NaN codes among them
            return c
        self.kc, self.vc = codes(), codes()
        self.ks = 2.0 ** torch.randint(-9, -5, (pages, Hkv), generator=g).float()
        self.vs = 2.0 ** torch.randint(-9, -5, (pages, Hkv), generator=g).float()
        self.slot_major = slot_major
        qkv = torch.randn(N, Hq + 2 * Hkv, D, generator=g)
        if spread:
            qkv *= 2.0 ** torch.randint(-6, 7, (N, 1, 1), generator=g).float()
        self.qkv = qkv.to(DT[dtype])
        self.Hq, self.Hkv, self.fused = Hq, Hkv, fused

    def split(self, x):
        return x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]

    def to_gpu(self, w8):
        kc, vc = self.kc.cuda(), self.vc.cuda()
        if self.slot_major:
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
        self.cache = w8.KVCache(kc, vc, self.ks.cuda(), self.vs.cuda())
        qkv = self.qkv.cuda()
        q, k, v = self.split(qkv)
        if not self.fused:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        self.q, self.k, self.v = q, k, v
        self.dtable = torch.from_numpy(self.table).cuda()
        self.dlens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.dcu = torch.tensor(self.cu, dtype=torch.int32).cuda()
        return self

    def state(self):
        def np_codes(c):
            return (c.transpose(1, 2) if self.slot_major else c).contiguous().numpy().copy()
        return {"k": np_codes(self.kc), "v": np_codes(self.vc), "k_scale": self.ks.double().numpy().copy(),
                "v_scale": self.vs.double().numpy().copy()}

    def np_qkv(self):
        return [t.double().numpy() for t in self.split(self.qkv)]

    def gpu_state(self):
        c = self.cache
        return {"k": c.k_codes.cpu().contiguous().numpy(), "v": c.v_codes.cpu().contiguous().numpy(),
                "k_scale": c.k_scale.cpu().double().numpy(), "v_scale": c.v_scale.cpu().double().numpy()}


def same_codes_or_neighbours(got, want, share):
    """Codes equal, but for at most `share` of them one step apart."""
    bad = np.argwhere(got != want)
    if len(bad) == 0:
        return
    order = np.where(np.arange(256) < 128, np.arange(256), 128 - np.arange(256)).astype(int)   # monotone index
    step = np.abs(order[got[tuple(bad.T)]] - order[want[tuple(bad.T)]])
    assert step.max() <= 1, f"codes differ by {step.max()} steps"
    assert len(bad) <= max(2, share * got.size), f"{len(bad)} of {got.size} codes differ"


def check(case, w8, rot, interleaved, uniform=False, in_place=False):
    case.to_gpu(w8)
    cos, sin = ref.rope_table(max(max(case.lens), 1) + 3, rot) if rot else (None, None)
    if rot:
        dc, ds = cos.cuda(), sin.cuda()
    else:
        dc = ds = None
    kw = {} if uniform else {"cu_q": case.dcu, "max_q": max(case.counts)}
    qo = w8.kv_append(case.cache, case.k, case.v, case.dtable, case.dlens, dc, ds, q=case.q,
                      q_out=case.q if in_place else None, interleaved=interleaved, **kw)
    torch.cuda.synchronize()
    st = case.state()
    q, k, v = case.np_qkv()
    want_q = ref.append(st, k, v, q, case.table, case.lens, case.cu, cos.double().numpy() if rot else None,
                        sin.double().numpy() if rot else None, rot, interleaved)
    got = case.gpu_state()
    assert np.array_equal(got["v_scale"], st["v_scale"])
    assert np.array_equal(got["v"], st["v"])
    assert np.array_equal(got["k_scale"], st["k_scale"])
    # midpoints hit within 2^-22 (|a|+|b|): spacing of codes is >= 2^-4 of the value, so
    # the chance per element is below 2^-15
    same_codes_or_neighbours(got["k"], st["k"], 2.0 ** -13)
    gq = qo.double().cpu().numpy()
    big = np.abs(q).max(axis=-1, keepdims=True)
    assert np.all(np.abs(gq - want_q) <= EPS[case.dtype] * np.abs(want_q) + 2.0 ** -21 * big + 2.0 ** -25)
    if rot < case.D:
        assert np.array_equal(gq[..., rot:], q[..., rot:])
    return case


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 64, True), (64, 64, True), (80, 32, False),
                                               (96, 96, False), (256, 128, False), (16, 16, True), (128, 0, False)])
def test_single_tokens(w8, D, rot, interleaved, dtype):
    # first token of all, first and last slot of a page, mid-page; an empty sequence
    case = Case([1, 17, 32, 33, 250, 0], [1, 1, 1, 1, 1, 1], 4, 2, D, 16, dtype, seed=D + rot)
    check(case, w8, rot, interleaved, uniform=True)


@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("slot_major,fused", [(False, False), (True, True)])
def test_chunks(w8, P, slot_major, fused):
    # odd chunks that begin and end inside pages, one longer than its sequence (padding), one empty
    case = Case([201, 77, 33, 300, 5], [75, 77, 1, 131, 0], 6, 3, 64, P, "bf16", seed=P, slot_major=slot_major, fused=fused)
    check(case, w8, 64, False)
    pad = Case([40, 3], [41, 9], 2, 1, 128, P, "f16", seed=P + 1, slot_major=slot_major, fused=fused)
    check(pad, w8, 128, True)


def test_growing_scales_and_in_place(w8):
    case = Case([20, 40, 60, 16], [3, 3, 3, 3], 2, 2, 128, 32, "bf16", seed=5, spread=True)
    check(case, w8, 128, False, in_place=True)


def test_token_by_token_equals_values_held(w8):
    """A page filled one token at a time holds, for each token, its value rounded once at
    the page's final scale, where that scale's normal range covers it."""
    P, H, D = 16, 2, 64
    g = torch.Generator().manual_seed(3)
    cache = w8.KVCache.empty(2, P, H, D)
    x = (torch.randn(P, H, D, generator=g) * 2.0 ** torch.randint(-2, 3, (P, 1, 1), generator=g).float()).bfloat16().cuda()
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    for t in range(P):
        w8.kv_append(cache, x[t:t + 1], x[t:t + 1], table, torch.tensor([t + 1], dtype=torch.int32, device="cuda"))
    whole = w8.KVCache.empty(2, P, H, D)
    w8.kv_append(whole, x, x, table, torch.tensor([P], dtype=torch.int32, device="cuda"))
    assert torch.equal(cache.k_scale, whole.k_scale) and torch.equal(cache.v_codes, cache.k_codes)
    a = cache.k_codes[1].view(torch.float8_e4m3fn).float()
    b = whole.k_codes[1].view(torch.float8_e4m3fn).float()
    normal = b.abs() >= 2.0 ** -6
    assert torch.equal(a[normal], b[normal])
    assert (a - b).abs().max() <= 2.0 ** -9            # one step of the subnormal range
    assert cache.k_codes[0].sum() == 0


def test_nonfinite_and_zero_tokens(w8):
    case = Case([16, 16], [16, 2], 2, 2, 64, 16, "bf16", seed=9)
    case.qkv[3, 2, 5] = float("inf")
    case.qkv[4, 3, 6] = float("-inf")
    case.qkv[5, 4, 7] = float("nan")
    case.qkv[16:, 2:] = 0.0                             # zero keys and values
    check(case, w8, 0, False)


def test_another_stream_and_no_queries(w8):
    case = Case([70, 9], [1, 1], 2, 2, 128, 16, "bf16", seed=11).to_gpu(w8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w8.kv_append(case.cache, case.k, case.v, case.dtable, case.dlens, stream=s)
    s.synchronize()
    st = case.state()
    _, k, v = case.np_qkv()
    ref.append(st, k, v, None, case.table, case.lens, case.cu, None, None, 0, False)
    got = case.gpu_state()
    assert all(np.array_equal(got[n], st[n]) for n in st)


def test_bad_indices_are_skipped_and_reported(w8):
    case = Case([20, 40], [2, 2], 2, 1, 64, 16, "bf16", seed=13).to_gpu(w8)
    before = case.gpu_state()
    cos, sin = (t.cuda() for t in ref.rope_table(10, 64))
    for table, lens, rope in ((case.dtable + 1000, case.dlens, (None, None)), (case.dtable - 1000, case.dlens, (None, None)),
                              (case.dtable, case.dlens + 100000, (None, None)), (case.dtable, case.dlens, (cos, sin))):
        w8.kv_append(case.cache, case.k, case.v, table, lens, *rope)
        assert w8.device_status(clear=True)[0] == 2
    cu = torch.tensor([0, 7, 4], dtype=torch.int32, device="cuda")
    w8.kv_append(case.cache, case.k, case.v, case.dtable, case.dlens, cu_q=cu, max_q=2)
    assert w8.device_status(clear=True)[0] == 2
    after = case.gpu_state()
    assert all(np.array_equal(before[n], after[n]) for n in before)
    assert w8.device_status()[0] == 0


def test_refusals(w8):
    case = Case([20, 40], [1, 1], 2, 2, 64, 16, "bf16", seed=15).to_gpu(w8)
    c, k, v, t, n = case.cache, case.k, case.v, case.dtable, case.dlens
    cos, sin = (x.cuda() for x in ref.rope_table(50, 64))
    with pytest.raises(TypeError):
        w8.kv_append(c, k.float(), v.float(), t, n)
    with pytest.raises(TypeError):
        w8.kv_append(c, k, v.half(), t, n)
    with pytest.raises(ValueError):
        w8.kv_append(c, k, v, t.long(), n)
    with pytest.raises(ValueError):
        w8.kv_append(c, k, v, t, n[:1])
    with pytest.raises(ValueError):
        w8.kv_append(c, k, v, t.cpu(), n)
    with pytest.raises(ValueError):
        w8.kv_append(c, k[:, :, :32], v, t, n)
    with pytest.raises(ValueError):
        w8.kv_append(c, k, v, t, n, cos, sin[:-1])
    with pytest.raises(ValueError):
        w8.kv_append(c, k, v, t, n, q_out=case.q)
    with pytest.raises(w8.W8A16Error):
        w8.kv_append(c, k[:, :1], v, t, n)                              # heads
    with pytest.raises(w8.W8A16Error):
        w8.kv_append(c, k, v, t, n, *(x.cuda() for x in ref.rope_table(50, 24)))   # rotary_dim % 16
    with pytest.raises(w8.W8A16Error):
        w8.kv_append(c, k, v, t, n, *(x.cuda() for x in ref.rope_table(50, 80)))   # above head_dim
    odd = torch.empty(2 * 2 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 2, 64)
    with pytest.raises(w8.W8A16Error):
        w8.kv_append(c, odd, v, t, n)                                   # alignment
    with pytest.raises(ValueError):
        w8.KVCache(c.k_codes, c.v_codes[:, :1], c.k_scale, c.v_scale)
    with pytest.raises(ValueError):
        w8.KVCache(c.k_codes, c.v_codes, c.k_scale.double(), c.v_scale)
    bad = w8.KVCache.empty(4, 24, 2, 64)                                # page size
    with pytest.raises(w8.W8A16Error):
        w8.kv_append(bad, k, v, t, n)
