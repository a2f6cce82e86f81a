"""The choice of a kernel for an FP8 product, on the host (no GPU)."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "nvfp4_block_scaled_quantize_amd", "csrc")
STREAM, T64X32, T64X64, T64X128, T128X128, T256X256 = range(6)


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    """[(kernel, workgroups, threads of one)] of pairs (B, N)."""
    exe = tmp_path_factory.mktemp("tiles") / "fp8_tiles"
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, os.path.join(HERE, "host_fp8_tiles.cpp"), "-o", str(exe)], check=True,
                   capture_output=True)

    def run(pairs):
        out = subprocess.run([str(exe)] + [str(x) for p in pairs for x in p], check=True, capture_output=True, text=True)
        return [tuple(int(x) for x in line.split()) for line in out.stdout.splitlines()]
    return run


def test_every_product_fits_a_launch(choose):
    """The entry point takes ceil(B / 128) ceil(N / 128) <= 2^22 tiles; a launch takes fewer than 2^32 threads.  2^29 - 63
    rows and more by up to 64 columns are 2^23 workgroups of 64 x 64, 2^32 threads."""
    most = 1 << 22
    pairs = [(1 << 29, 64), (1 << 29, 1), ((1 << 29) - 63, 33), ((1 << 29) - 64, 64), (1 << 29, 128), (64, 1 << 29), (1, 1 << 29)]
    for e in range(1, 23):
        for rows, cols in ((1 << e, most >> e), ((1 << e) - 1, most // ((1 << e) - 1))):
            pairs += [(128 * rows - i, 128 * cols - j) for i in (0, 63, 64, 127) for j in (0, 63, 64, 127)]
    for (b, n), (kernel, groups, threads) in zip(pairs, choose(pairs)):
        assert groups * threads < 1 << 32, (b, n, kernel, groups)


def test_sizes_and_kernels(choose):
    want = {(1, 4096): STREAM, (8, 4096): STREAM, (9, 4096): T64X32, (1, 8192): T64X32, (64, 8192): T64X32,
            (128, 8192): T64X64, (777, 2120): T64X128, (400, 8192): T64X128, (512, 8192): T64X128, (1000, 8192): T128X128, (2048, 4096): T128X128, (2048, 2048): T64X128,
            (1500, 2700): T128X128, (4096, 8192): T256X256, (4096, 4096): T256X256}
    assert dict(zip(want, (c[0] for c in choose(list(want))))) == want
