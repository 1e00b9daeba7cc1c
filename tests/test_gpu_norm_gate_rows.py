"""A gate without rows is refused: its pointer is NULL, which for the library means a call without a gate."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_gate_without_rows_is_refused():
    import fp8_weight_only_gemm_gb300 as w8
    x, w = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for gate in (x[:0], torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")):
        with pytest.raises(ValueError, match="gate"):
            w8.norm_residual(x, x, w, gate=gate)
