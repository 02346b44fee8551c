"""What the f16 warp MMA drops when it sums E4M3 products (a hardware property): the page
selection takes 2^-23 A per MMA step as the bound on a score's error, A = sum |q| * max |bound|;
the probe holds the MMA to half of that."""
import os
import subprocess

import pytest

from fp8_attention_forward_gb300 import build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_dropped_bits_stay_within_the_selection_bound(tmp_path):
    exe = str(tmp_path / "probe")
    subprocess.run([build.nvcc(), *build.ARCH, "-O2", "-std=c++17", "--expt-relaxed-constexpr", "-I",
                    os.path.join(build.ROOT, "include"), "-I", build.CSRC, "-o", exe,
                    os.path.join(HERE, "mma_accumulation_probe.cu")], check=True, capture_output=True, timeout=600)
    out = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=300).stdout
    rows = [line.split("|") for line in out.strip().splitlines()]
    assert len(rows) == 5
    for kind, worst in rows:
        print(kind, worst)
        assert float(worst) <= 0.5, (kind, worst)
