"""What the kernels do about copies on their way when a wait gives up: ring_drain waits for all
of them before the ring is read, reused or left, also where the phases have wrapped, and it
ends at its own limit. (That no wait of a healthy call gives up is why the function is tested by
itself; the kernels' calls of it cover the steps that they have asked for and not yet taken.)"""
from __future__ import annotations

import ctypes
import subprocess
import time
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parent.parent
STAGES, BYTES = 3, 8192


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    from fp8_weight_only_gemm_gb300 import build
    so = tmp_path_factory.mktemp("probe") / "ring_drain_probe.so"
    r = subprocess.run([build._nvcc(), *build.ARCH, "-O3", "-std=c++17", "--expt-relaxed-constexpr", "-shared", "-Xcompiler", "-fPIC", "-I", str(build.INCLUDE),
                        "-I", str(build.CSRC), str(ROOT / "tests" / "ring_drain_probe.cu"), "-o", str(so)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(str(so))
    lib.ring_drain_probe.argtypes = [ctypes.c_void_p, ctypes.c_uint, ctypes.c_uint, ctypes.c_void_p]
    lib.ring_drain_limit.argtypes = [ctypes.c_uint64]
    return lib


def status(lib):
    w = (ctypes.c_uint * 3)()
    assert lib.ring_drain_status(w) == 0
    return tuple(w)


@pytest.mark.parametrize("taken,steps", [(0, 1), (0, 3), (1, 3), (2, 9), (3, 6), (5, 20), (7, 8), (4, 4)])
def test_all_copies_have_landed(probe, taken, steps):
    g = torch.Generator("cuda").manual_seed(taken + 31 * steps)
    src = torch.randint(0, 256, (steps, BYTES), generator=g, dtype=torch.uint8, device="cuda")
    out = torch.zeros(STAGES, BYTES, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert probe.ring_drain_probe(src.data_ptr(), taken, steps, out.data_ptr()) == 0
    left = min(STAGES, steps - taken)
    assert torch.equal(out[:left], src[taken:taken + left]) and not out[left:].any()
    assert status(probe)[0] == 0


def test_the_limit_is_its_own(probe):   # last: it leaves the probe's status set
    begin = time.perf_counter()
    assert probe.ring_drain_limit(50_000_000) == 0
    assert time.perf_counter() - begin < 5.0
    code, _, detail = status(probe)
    assert (code, detail) == (1, 7)
