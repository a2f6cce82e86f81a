"""Host checks of address arithmetic that the attention kernels share with the host, and of the limits of
a launch (no GPU)."""
import ctypes
import os
import subprocess

import pytest
import torch

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


# never dereferenced: a call that is not refused must not find a device to launch on
@pytest.mark.skipif(torch.cuda.is_available(), reason="refusals only, without a GPU")
@pytest.mark.parametrize("tokens,seqs,q_heads,kv_heads", [(1 << 20, 1 << 20, 32, 32), (1 << 20, 1 << 19, 64, 32),
                                                          (1 << 26, 1, 32, 32), (128, (1 << 19) - 2, 32, 32)])
def test_prompts_of_more_workgroups_than_a_launch_takes(tokens, seqs, q_heads, kv_heads):
    """A launch takes fewer than 2^32 threads, 2^24 workgroups of 256."""
    import nvfp4_block_scaled_quantize_amd as nv
    assert (tokens * (q_heads // kv_heads) // 128 + seqs + 1) * kv_heads >= 1 << 24
    p = ctypes.c_void_p(4096)
    fn = nv.lib().nvfp4_prompt_attn

    def call(n):
        return fn(p, p, p, nv.NVFP4_BF16, p, n, tokens, q_heads, kv_heads, 64, 0, 64, 0, 64, 0, 64, 0.125, 0, p, p, None)

    assert call(seqs) == nv.NVFP4_EUNSUPPORTED
    if tokens == 128:   # one workgroup of each head fewer: accepted up to the question for a device
        assert call(seqs - 1) not in (nv.NVFP4_OK, nv.NVFP4_EINVAL, nv.NVFP4_EUNSUPPORTED)
