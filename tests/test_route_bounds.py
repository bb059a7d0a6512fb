"""Host check of the bounds of routing by scores (csrc/route_bounds.hpp): a token whose
choice hangs on two values closer than they say is chosen again in double precision, so
they have to hold for every rounding at its worst.  tests/route_bounds_check.cpp gives
each one its largest error over grids of logits, biases and ranges."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "bit_quantized_linear_rotate_amd", "csrc")


def test_bounds_hold_at_the_worst(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "route_bounds_check")
    subprocess.check_call([gxx, "-std=c++17", "-O2", "-ffp-contract=off", "-I", CSRC,
                           os.path.join(HERE, "route_bounds_check.cpp"), "-o", exe])
    out = subprocess.run([exe], capture_output=True, text=True)
    print(out.stdout)
    assert out.returncode == 0, out.stdout + out.stderr
    assert len(out.stdout.splitlines()) == 30
