"""The code-generation guard on the sources of the fused layer, the expert products and the router: no register-spill
store between a buffer-to-LDS load and its barrier, nor while a vector-memory load may still be in flight; and no matrix
instruction of 8 passes whose result overlaps its operands, or part of another's result.

Why the last: with the upper half of a 16-row tile's sums unused, the compiler gave two such results overlapping
registers (v[2:17] and v[10:25]), and the weight-stream kernel returned wrong sums, NaN among them, from the variants
compiled so and from no others."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

from bit_weight_only_awq_amd import build as B
from tests.test_codegen_guard import SOURCES, lds_dma_spill_hazards, spill_stores_with_loads_in_flight


def kernel_sources():
    return [s for s in B.SOURCES if s not in SOURCES and s not in ("awq_api.hip", "awq_noalloc.hip", "awq_fused_api.hip")]


def overlapping_results(asm: str):
    """(function, instruction, registers) of every 32x32 matrix instruction whose result overlaps an operand, and every
    pair of results that share some registers but not all."""
    bad, fn, results = [], None, {}
    span = lambda t: (m.group(1), int(m.group(2)), int(m.group(3))) if (m := re.match(r"([va])\[(\d+):(\d+)\]", t)) else None  # noqa: E731
    over = lambda p, q: p is not None and q is not None and p[0] == q[0] and p[1] <= q[2] and q[1] <= p[2]  # noqa: E731
    for line in asm.splitlines():
        if m := re.match(r"^(_Z\S+):", line):
            fn = m.group(1)
        m = re.match(r"\s+(v_mfma_f32_32x32\S+) (\S+), (\S+), (\S+), ", line)
        if not m:
            continue
        d, a, b = (span(t) for t in m.groups()[1:4])
        if over(d, a) or over(d, b):
            bad.append((fn, m.group(1), d))
        for other in results.setdefault(fn, set()):
            if other != d and over(other, d):
                bad.append((fn, m.group(1), other, d))
        results[fn].add(d)
    return bad


def test_guard_flags_overlapping_results():
    lines = ["_Zk:", "\tv_mfma_f32_32x32x16_f16 v[2:17], v[34:37], v[30:33], 0",
             "\tv_mfma_f32_32x32x16_f16 v[10:25], v[34:37], v[30:33], 0",
             "\tv_mfma_f32_32x32x16_f16 v[40:55], v[52:55], v[30:33], 0",
             "\tv_mfma_f32_32x32x16_f16 a[2:17], v[2:5], v[30:33], a[2:17]"]
    assert len(overlapping_results("\n".join(lines))) == 2
    assert not overlapping_results("\n".join(lines[:2] + lines[4:]))


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
    assert not overlapping_results(asm)
