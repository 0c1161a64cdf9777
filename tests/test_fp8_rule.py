"""Which kernel takes a call of the e4m3 linear layer, on the host (no GPU):
compiles and runs tests/host/fp8_rule.cu (see its header).  A GB300 has 152 SMs."""
import os
import shutil
import subprocess

import pytest

from test_fp8_wide_gpu import SIZES

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    out = str(tmp_path_factory.mktemp("rule") / "fp8_rule")
    r = subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", "-o", out,
                        os.path.join(HERE, "host", "fp8_rule.cu")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return out


def run(exe, *args):
    r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    return r.stdout.split("\n")


def test_choices_fit_a_launch(exe):
    assert run(exe)[-2].endswith(" 0 failed checks")


def test_the_sizes_of_the_many_row_tests_go_to_that_kernel(exe):
    got = run(exe, 152, *(x for size in SIZES for x in size))[:-1]
    assert dict(zip(SIZES, got)) == SIZES
    assert set(got) == {"narrow", "wide"}
