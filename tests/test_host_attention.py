"""Host checks of address arithmetic that the attention kernels share with the host (no GPU)."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "nvfp4_block_scaled_quantize_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def test_offsets_inside_a_page_pass_32_bits(tmp_path):
    """A page may have 2^30 places: the byte offset of a row passes 2^31 from place 2^23 on at 256 bytes
    a row (2^24 at 128), where a product in 32 bits turns negative."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc unavailable")
    exe = tmp_path / "page_offset"
    subprocess.run([HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-I", CSRC,
                    os.path.join(HERE, "host_page_offset.cpp"), "-o", str(exe)], check=True, capture_output=True)
    pairs = [(p, b) for b in (16, 128, 192, 256) for n in (23, 24, 27, 30) for p in ((1 << n) - 1, (1 << n) % (1 << 30))]
    out = subprocess.run([str(exe)] + [str(x) for pair in pairs for x in pair], check=True, capture_output=True, text=True)
    assert [int(x) for x in out.stdout.split()] == [p * b for p, b in pairs]
