"""Calls behind a kernel that lets them start at once and, milliseconds later, reads their outputs and workspace and writes their operands:
no call reads or writes anything before that kernel is done. Until then the operands hold other, valid values. Each call has to give the
bits that it gives alone, and the kernel has to find outputs and workspace as they were. (That dependents do start early is tested with
one that notes the time.)"""
from __future__ import annotations

import ctypes
import subprocess
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parent.parent
DELAY_NS = 3_000_000


@pytest.fixture(scope="module")
def w8():
    import fp8_weight_only_gemm_gb300 as w8
    from fp8_weight_only_gemm_gb300.build import build_library
    build_library()
    w8.load()
    w8.device_status(clear=True)
    yield w8
    assert w8.device_status(clear=True)[0] == 0


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    from fp8_weight_only_gemm_gb300 import build
    so = tmp_path_factory.mktemp("probe") / "late_writer_probe.so"
    r = subprocess.run([build._nvcc(), *build.ARCH, "-O3", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
                        str(ROOT / "tests" / "late_writer_probe.cu"), "-o", str(so)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(str(so))


def late_copies(probe, pairs, done_at):
    n = len(pairs)
    assert all(a.is_contiguous() and b.is_contiguous() and a.nbytes == b.nbytes for a, b in pairs)
    src = (ctypes.c_void_p * n)(*(a.data_ptr() for a, _ in pairs))
    dst = (ctypes.c_void_p * n)(*(b.data_ptr() for _, b in pairs))
    size = (ctypes.c_ulonglong * n)(*(a.nbytes for a, _ in pairs))
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert probe.late_writer_launch(src, dst, size, ctypes.c_uint(n), ctypes.c_ulonglong(DELAY_NS), ctypes.c_void_p(done_at.data_ptr()), stream) == 0


def bits(t):
    return t.contiguous().view(torch.uint8)


def behind(probe, call, operands, outputs):
    """operands: (tensor, what it holds until the predecessor writes it); outputs: what the call writes, workspace included. One that is
    both is held to its result alone."""
    true = [t.clone() for t, _ in operands]
    call()
    torch.cuda.synchronize()
    alone = [t.clone() for t in outputs]
    inout = [any(t is o for o, _ in operands) for t in outputs]
    for (t, early) in operands:
        t.copy_(early) if torch.is_tensor(early) else t.fill_(early)
    for t, both in zip(outputs, inout):
        if not both:
            bits(t).fill_(0x3A)
    kept = [torch.zeros_like(t) for t in outputs]
    done_at = torch.zeros(1, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    late_copies(probe, [(t, k) for t, k, both in zip(outputs, kept, inout) if not both] + [(a, t) for a, (t, _) in zip(true, operands)], done_at)
    call()
    torch.cuda.synchronize()
    for i, (t, a, k, both) in enumerate(zip(outputs, alone, kept, inout)):
        if t.dtype != torch.uint8 or both:          # (uint8: a workspace, which need not come out the same)
            assert torch.equal(bits(t), bits(a)), f"output {i} differs"
        assert both or bool((bits(k) == 0x3A).all()), f"output {i} was written early"


def rand(*shape, dtype=torch.bfloat16, seed=0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def test_dependents_start_early(probe):
    times = torch.zeros(2, dtype=torch.int64, device="cuda")
    a, b = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    early = False
    for _ in range(10):     # the first may be late, its code being loaded, or one whose launch this process was slow to make
        torch.cuda.synchronize()
        late_copies(probe, [(a, b)], times[:1])
        assert probe.early_start_launch(ctypes.c_void_p(times[1:].data_ptr()), stream) == 0
        torch.cuda.synchronize()
        early = early or 0 < int(times[1]) < int(times[0])
    assert torch.equal(a, b) and early


@pytest.mark.parametrize("M,H", [(1, 4096), (70, 512), (400, 8192)])
@pytest.mark.parametrize("quantize", [False, True])
def test_norms(w8, probe, M, H, quantize):
    x, r, w, h, gate = rand(M, H), rand(M, H, dtype=torch.float32), rand(H, dtype=torch.float32), torch.zeros(M, H, device="cuda"), rand(M, H, seed=1)
    y = (torch.zeros(M, H, dtype=torch.uint8, device="cuda"), torch.zeros(H // 128, (M + 3) // 4 * 4, device="cuda")) if quantize else torch.zeros_like(x)
    for flags, late in ((0, [(w, 1.0)]), (w8.FLAG_PDL, [])):        # with the flag no earlier work may write the weights
        outputs = [h, y[0].view(torch.int8) if quantize else y]
        behind(probe, lambda: w8.norm_residual(x, r, w, post_weight=w, gate=gate, out=y, residual_out=h, quantize=quantize, flags=flags),
               [(x, 0.5), (r, 0.25), (gate, 2.0)] + late, outputs)


class Served:
    """Three sequences in a paged cache, the operands of a call, and what they hold before they are written."""

    def __init__(self, w8, T, heads, D, kv_heads=2, P=32, length=1500):
        self.D, pages = D, 3 * -(-length // P)
        self.cache = w8.KVCache.empty(pages, P, kv_heads, D)
        g = torch.Generator("cuda").manual_seed(T + D)
        for c in (self.cache.k_codes, self.cache.v_codes):
            c.copy_((torch.randn(c.shape, generator=g, device="cuda") * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        self.cache.k_scale.copy_(2.0 ** torch.randint(-9, -6, self.cache.k_scale.shape, generator=g, device="cuda"))
        self.cache.v_scale.copy_(2.0 ** torch.randint(-9, -6, self.cache.v_scale.shape, generator=g, device="cuda"))
        self.table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(3, -1).contiguous()
        self.lens = torch.tensor([length, length - 601, length - 77], dtype=torch.int32, device="cuda")
        self.q = torch.randn(3 * T, heads, D, generator=g, device="cuda").to(torch.bfloat16)
        self.out = torch.zeros_like(self.q)
        self.operands = [(self.q, 0.5), (self.lens, T + 40), (self.table, 0), (self.cache.k_codes, 0), (self.cache.v_codes, 0),
                         (self.cache.k_scale, 1.0), (self.cache.v_scale, 1.0)]


@pytest.mark.parametrize("T,heads,D", [(1, 8, 128), (3, 4, 64), (30, 8, 128), (5, 4, 256)])
@pytest.mark.parametrize("span", [{}, dict(window=200, sinks=4)])
def test_attention(w8, probe, T, heads, D, span):
    s = Served(w8, T, heads, D)
    ws = torch.empty(w8.kv_attention_workspace_bytes(s.cache, 3, T, heads), dtype=torch.uint8, device="cuda")
    behind(probe, lambda: w8.kv_attention(s.cache, s.q, s.table, s.lens, s.out, workspace=ws, **span), s.operands, [s.out, ws])


# rows a key/value head, of the prefix pass and of the sequences' own keys: both on the kernel for few; the first on the kernel for
# many; both on it; there with the launch between them that joins many parts; heads that only the kernel for few takes
@pytest.mark.parametrize("T,heads,D,prefix", [(1, 8, 128, 500), (2, 8, 64, 500), (5, 8, 128, 800), (30, 8, 128, 100), (17, 8, 64, 890), (12, 8, 256, 500)])
def test_attention_over_a_prefix(w8, probe, T, heads, D, prefix):
    s = Served(w8, T, heads, D)
    pages = s.table[0, :-(-prefix // 32)].contiguous()
    ws = torch.empty(w8.kv_attention_workspace_bytes(s.cache, 3, T, heads, prefix_tokens=3 * T), dtype=torch.uint8, device="cuda")
    behind(probe, lambda: w8.kv_attention(s.cache, s.q, s.table, s.lens, s.out, workspace=ws, prefix_pages=pages, prefix_len=prefix),
           s.operands + [(pages, 1)], [s.out, ws])


@pytest.mark.parametrize("several", [False, True])
@pytest.mark.parametrize("T", [1, 40])
def test_append(w8, probe, T, several):
    s = Served(w8, T, 8, 128)
    k, v = rand(3 * T, 2, 128, seed=3), rand(3 * T, 2, 128, seed=4)
    cos, sin = rand(1600, 64, dtype=torch.float32, seed=5), rand(1600, 64, dtype=torch.float32, seed=6)
    positions = torch.randint(0, 1600, (2, 3 * T), generator=torch.Generator().manual_seed(7), dtype=torch.int32).cuda()
    kw = dict(positions=positions, axes=w8.RopeAxes.sections((30, 34), cyclic=True)) if several else {}
    c = s.cache
    # (the sequences' pages are read as no others' here: the table stays, or the poison's page would be all sequences')
    operands = [o for o in s.operands if o[0] is not s.table] + [(k, 1.0), (v, 1.0), (cos, 1.0), (sin, 0.0)] + ([(positions, 0)] if several else [])
    behind(probe, lambda: w8.kv_append(c, k, v, s.table, s.lens, cos, sin, q=s.q, q_out=s.out, **kw), operands,
           [s.out, c.k_codes, c.v_codes, c.k_scale, c.v_scale])
