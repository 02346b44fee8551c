"""What the f16 warp MMA drops over one chain of MMAs (a hardware property), on which the page selection's
bound on a score's error rests: each product that is not zero and each running sum is cut below 2^-25 of the
largest addend's leading bit, and each MMA's result to fp32's 24 bits.  The probe holds the MMA to the sum of
these, also on data whose dropped parts add up."""
import os
import subprocess

import pytest

from fp8_attention_forward_gb300 import build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_a_chain_drops_no_more_than_the_selection_allows(tmp_path):
    exe = str(tmp_path / "probe")
    subprocess.run([build.nvcc(), *build.ARCH, "-O2", "-std=c++17", "--expt-relaxed-constexpr", "-I",
                    os.path.join(build.ROOT, "include"), "-I", build.CSRC, "-o", exe,
                    os.path.join(HERE, "mma_chain_probe.cu")], check=True, capture_output=True, timeout=600)
    out = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=300).stdout
    rows = [line.split("|") for line in out.strip().splitlines()]
    assert len(rows) == 7 + 4 * 10 * 2
    for kind, worst in rows:
        print(kind, worst)
        assert float(worst) <= 1.0, (kind, worst)
