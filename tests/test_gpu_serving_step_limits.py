"""The largest sizes that the header allows, as far as they fit: rows, columns and tokens whose offsets pass 32 bits, the
longest rows, the most heads."""
import pytest
import torch

import strict_checks as strict
import test_gpu_fp8 as fp8
import test_gpu_moe_decode as moe
import test_gpu_moe_decode_kernels as kernels
import test_gpu_rope_kv as rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return nv


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantizer_of_many_rows(nv, block_rows):
    """6.4 billion values: rows that repeat (in whole blocks), so that the result does."""
    rows, k, period = (1 << 27) + 77, 48, 128 * 8191
    x = torch.randn((period, k), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    want = nv.fp8_quantize(x, block_rows=block_rows)
    codes, scale = fp8.quantize_ref(x.cpu()[:1280], block_rows)
    assert torch.equal(want["codes"][:1280].cpu().view(torch.uint8), codes.view(torch.uint8))
    got = nv.fp8_quantize(x.repeat(-(-rows // period), 1)[:rows], block_rows=block_rows)
    for at in range(0, rows - rows % 128, period):   # the last block, that is short, below
        n = min(period, rows - rows % 128 - at)
        assert torch.equal(got["codes"][at:at + n].view(torch.uint8), want["codes"][:n].view(torch.uint8)), at
        assert torch.equal(got["scale"][at // block_rows:(at + n) // block_rows], want["scale"][:n // block_rows]), at
    codes, scale = fp8.quantize_ref(x.cpu()[(rows - rows % 128) % period:][:rows % 128], block_rows)
    assert torch.equal(got["codes"][-(rows % 128):].cpu().view(torch.uint8), codes.view(torch.uint8))
    assert (got["scale"][-len(scale):].cpu().numpy() == scale).all()


def test_the_most_columns(nv):
    """2^29 rows of w for one of a."""
    N, period = 1 << 29, 128 * 8191
    a, sa, w, sw = fp8.exact_operands(1, period, 16, seed=5)
    want = fp8.binary64(a, sa, w, sw)[0].half().view(-1)
    times = -(-N // period)
    y = nv.fp8_gemm(a, sa, w.view(torch.uint8).repeat(times, 1)[:N].view(fp8.FP8), sw.repeat(times, 1)[:N // 128]).view(-1)
    for at in range(0, N, period):
        part = y[at:at + period]
        assert torch.equal(part, want[:len(part)]), at


@pytest.mark.parametrize("B,N", [(2, 3), (9, 20)])
def test_the_longest_rows(nv, B, N):
    K = (1 << 24) - 16
    ops = fp8.operands(B, N, K, seed=B)
    strict.fp8_check(nv.fp8_gemm(*ops, out_dtype=torch.bfloat16), *fp8.binary64(*ops), K)


def test_the_most_tokens(nv):
    """2^24 - 1 tokens of a workgroup each, all of them the same row, few with a slot."""
    T, d = (1 << 24) - 1, 512
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((1, 1, d), generator=g).half() for _ in range(2))
    freq = 10000.0 ** (-torch.arange(d // 2) / (d // 2))
    positions = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    at = [0, 1, 65535, 65536, T // 2, T - 2, T - 1]
    slots[at] = torch.arange(len(at), device="cuda") + 3
    kc, vc = (torch.zeros((3, 1, 5, d), dtype=torch.float16, device="cuda") for _ in range(2))
    nv.rope_kv_write(None, k.cuda().expand(T, 1, d), v.cuda().expand(T, 1, d), positions, freq.cuda(), slots, kc, vc)
    want, room = rope.turned(k.expand(len(at), 1, d), torch.tensor(at, dtype=torch.int32), freq, False, 1.0)
    rope.near(kc.view(15, 1, d)[3:3 + len(at)].cpu(), want, room, torch.float16)
    assert torch.equal(vc.view(15, 1, d)[3:3 + len(at)].cpu(), v.expand(len(at), 1, d))
    for c in (kc, vc):
        assert not c.view(15, d)[:3].any() and not c.view(15, d)[3 + len(at):].any()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hk,d,r", [(65536, 1, 64, 64), (1, 1, 32768, 512), (1, 1, 32766, 510), (3, 65536, 32, 8)])
def test_the_most_heads_and_the_widest(nv, hq, hk, d, r, interleaved):
    rope.run(nv, "bf16", 3, hq, hk, d, r, interleaved, 2, 5000, seed=hq, pad=0)


@pytest.mark.parametrize("act", ["relu2", "swiglu"])
@pytest.mark.parametrize("tokens,hidden,inter", [(1, 65536, 64), (3, 65536, 64), (1, 64, 65536), (3, 64, 65536), (32, 65536, 128)])
def test_the_longest_expert_rows(nv, tokens, hidden, inter, act):
    layer = moe.Layer("bf16", tokens, 3, hidden, inter, act, seed=tokens)
    kernels.full(nv, layer, 2)
    if inter % 128 == 0 and hidden % 128 == 0:
        kernels.full(nv, layer, 2, tiled=True)
