"""Buffers that workgroups of a call read while others already write: an output overlaps nothing else that is passed, but
for the output of the MoE layer that is its input.  Refusals need no GPU."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="refusals only, without a GPU: the addresses are none")

SEE = 1 << 22    # far apart
# sizes in bytes: fp8_quantize 4 x 256 (SwiGLU: 4 x 512 in), fp8_gemm 5 x 300 x 272, moe_decode 3 tokens
QUANT = dict(x=4 * 512 * 2, codes=4 * 256, scale=4 * 2 * 4)
GEMM = dict(a=5 * 272, sa=5 * 3 * 4, w=300 * 272, sw=3 * 3 * 4, y=5 * 300 * 2)
E, T, K, H, M = 16, 3, 4, 256, 128
MOE = dict(x=T * H * 2, router=E * H * 2, bias=E * 4, w1=E * 2 * M * H // 2, w1_sf=E * 2 * M * H // 16, w1_g=E * 4, w2=E * H * M // 2,
           w2_sf=E * H * M // 16, w2_g=E * 4, out=T * H * 2, ids=T * K * 4, weights=T * K * 4, ws=None)


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    return nv


def quant(nv, at):
    p = {n: ctypes.c_void_p(a) for n, a in at.items()}
    return nv.lib().nvfp4_fp8_quantize(p["x"], 0, 4, 256, 1, 1, p["codes"], p["scale"], None)


def gemm(nv, at):
    p = {n: ctypes.c_void_p(a) for n, a in at.items()}
    return nv.lib().nvfp4_fp8_gemm(p["a"], p["sa"], p["w"], p["sw"], p["y"], 0, 5, 300, 272, None)


def moe(nv, at):
    p = {n: ctypes.c_void_p(a) for n, a in at.items()}
    need = nv.moe_decode_workspace_size(T, E, K, H, M)
    return nv.lib().nvfp4_moe_decode(p["x"], 1, p["router"], p["bias"], p["w1"], p["w1_sf"], p["w1_g"], p["w2"], p["w2_sf"],
                                     p["w2_g"], 0, p["out"], p["ids"], p["weights"], T, E, K, H, M, 1, 1, 1, 1, 1.0, p["ws"],
                                     need, None)


CALLS = [(quant, QUANT, "codes scale".split()), (gemm, GEMM, ["y"]), (moe, MOE, "out ids weights ws".split())]


@pytest.mark.parametrize("call,sizes,written", CALLS)
def test_overlaps_are_refused(nv, call, sizes, written):
    sizes = {n: s or nv.moe_decode_workspace_size(T, E, K, H, M) for n, s in sizes.items()}
    assert max(sizes.values()) < SEE
    at = {n: SEE * (i + 1) for i, n in enumerate(sizes)}
    assert call(nv, at) not in (nv.NVFP4_OK, nv.NVFP4_EINVAL)      # apart: accepted up to the question for a device
    for one in written:
        for two in sizes:
            if one == two:
                continue
            # one's last bytes are two's first, and the other way round, at an alignment that everything has
            for a, b in ((one, two), (two, one)):
                place = at[a] + (sizes[a] - 1) // 256 * 256
                want = nv.NVFP4_EINVAL
                if {one, two} == {"out", "x"} and place == at[a]:
                    continue
                assert call(nv, dict(at, **{b: place})) == want, (a, b)
                # one byte behind it, rounded up: apart
                behind = at[a] + -(-sizes[a] // 256) * 256
                assert call(nv, dict(at, **{b: behind})) != want, (a, b)


def test_the_output_may_be_the_input(nv):
    sizes = {n: s or nv.moe_decode_workspace_size(T, E, K, H, M) for n, s in MOE.items()}
    at = {n: SEE * (i + 1) for i, n in enumerate(sizes)}
    at["out"] = at["x"]
    assert moe(nv, at) not in (nv.NVFP4_OK, nv.NVFP4_EINVAL)
    for other in ("ids", "weights", "ws"):
        assert moe(nv, dict(at, **{other: at["x"]})) == nv.NVFP4_EINVAL
