"""How a ragged step is cut into pieces, on the host: a driver over the library's
own `kv8_step.cuh` with the undefined-behaviour sanitizer, over random steps of up to
2^20 rows, 1024 kv heads and 2^31 - 1 positions."""

import importlib
import os
import subprocess

import pytest

build = importlib.import_module("bit_moe_decode_w4a16_gb300.build")   # the package's own `build` is a function

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("cut") / "driver")
    cmd = [build.nvcc(), *build.ARCH, "-std=c++17", "-O1", "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"), "--expt-relaxed-constexpr",
           os.path.join(HERE, "host_kv8_cut_driver.cu"), "-o", exe]
    checked = ["-Xcompiler", "-fsanitize=undefined,-fno-sanitize-recover=all", "-lubsan"]
    made = subprocess.run(cmd + checked, capture_output=True, text=True)
    if made.returncode != 0 and "ubsan" in made.stderr + made.stdout:   # no sanitizer runtime: the driver's own checks alone
        made = subprocess.run(cmd, capture_output=True, text=True)
    assert made.returncode == 0, made.stderr
    return exe


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_pieces_cover_every_tile_once_and_fit(driver, seed):
    run = subprocess.run([driver, "20000", str(seed)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout + run.stderr[-2000:]
