"""The code-generation guard on the sources of the fused layer, the expert products and the router: no register-spill
store between a buffer-to-LDS load and its barrier, nor while a vector-memory load may still be in flight."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from bit_weight_only_awq_amd import build as B
from tests.test_codegen_guard import SOURCES, lds_dma_spill_hazards, spill_stores_with_loads_in_flight


def kernel_sources():
    return [s for s in B.SOURCES if s not in SOURCES and s not in ("awq_api.hip", "awq_noalloc.hip", "awq_fused_api.hip")]


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"), reason="needs hipcc")
@pytest.mark.parametrize("src", kernel_sources())
def test_no_spill_store_while_loads_are_in_flight(src, tmp_path):
    out = tmp_path / (src + ".s")
    cmd = [B.hipcc(), *(f for f in B.COMMON_FLAGS if f != "-fPIC"), "--cuda-device-only", "-S",
           os.path.join(B.CSRC, src), "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    asm = out.read_text()
    assert not lds_dma_spill_hazards(asm)
    assert not spill_stores_with_loads_in_flight(asm)
