"""The compiled variants of the 8-bit row kernel are those that a call can reach, by the rule that launches them."""
import re
import shutil
import subprocess

import pytest

TYPES = {"f": 4, "13__nv_bfloat16": 2, "6__half": 2}
QUANTIZE, NORM, NORM_RESIDUAL, GATE = range(4)


def _launched(op, size):
    """(eights a thread holds, team, threads, blocks an SM) for up to 128, 1024, 4096 columns and more."""
    if op in (NORM, NORM_RESIDUAL):
        long = (2, 0, 640, 2) if op == NORM else (3, 0, 416, 2) if size == 2 else (2, 0, 512, 2)
        return {(4, 32, 128, 6), (2, 0, 256, 3 if op == NORM_RESIDUAL and size == 4 else 4), long}
    middle = (4, 0, 128, 6) if op == QUANTIZE else (2, 0, 256, 4)
    return {(2, 8, 128, 8), (4, 32, 128, 8), middle, (4, 0, 320, 3) if size == 2 else (2, 0, 640, 2)}


@pytest.mark.skipif(shutil.which("nm") is None, reason="no nm")
def test_row_variants():
    from dual_ar_tts_gb300 import build
    names = subprocess.run(["nm", build.build()], capture_output=True, text=True, check=True).stdout
    found = {(t, int(op), *map(int, rest.split("ELi")))
             for t, op, rest in re.findall(r"k_q8_rowsI(f|13__nv_bfloat16|6__half)LNS\d*_2OpE(\d)ELi((?:\d+ELi)*\d+)EEEv", names)}
    want = {(t, op, *v) for t, size in TYPES.items() for op in range(4) for v in _launched(op, size)}
    assert found == want, (found - want, want - found)
