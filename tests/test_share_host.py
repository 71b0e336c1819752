"""The grouped products' blocks take every quarter of every tile exactly once."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("share") / "share_driver")
    subprocess.run(["g++", "-O2", "-std=c++17", os.path.join(HERE, "share_driver.cpp"), "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("units, most", [(1, 20), (2, 30), (3, 40), (4, 60), (7, 100), (64, 700), (256, 1600)])
def test_every_quarter_once(driver, units, most):
    r = subprocess.run([driver, str(units), str(most)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
