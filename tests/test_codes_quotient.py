"""The 8-bit codes' quotients by two products and a residue: rounded like the division's."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_rounded_like_the_quotient(tmp_path):
    exe = str(tmp_path / "codes_check")
    r = subprocess.run(["gcc", "-O2", "-std=c11", "-ffp-contract=off", os.path.join(HERE, "codes_check.c"), "-o", exe, "-lm"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        pytest.skip("no C compiler")
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
