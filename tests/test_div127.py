"""The division of a largest magnitude by 127 as two products: correctly rounded for every significand."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_significand(tmp_path):
    exe = str(tmp_path / "div127_check")
    r = subprocess.run(["gcc", "-O2", "-std=c11", "-ffp-contract=off", os.path.join(HERE, "div127_check.c"), "-o", exe, "-lm"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        pytest.skip("no C compiler")
    assert subprocess.run([exe]).returncode == 0
