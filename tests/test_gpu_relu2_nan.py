"""NaN through ReLU^2: it stays NaN, where max(NaN, 0) = 0 would hide it."""
import pytest
import torch

import test_gpu_fp8 as fp8
import test_gpu_moe_decode as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return nv


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantizer(nv, block_rows, dtype):
    """The NaN's code is NaN; its block's scale and the other codes are those of a block with 0 in its place."""
    x = torch.randn((130, 400), generator=torch.Generator().manual_seed(block_rows)).to(dtype).cuda()
    x[3, 7], x[129, 399], x[:, 64] = 0, 0, -0.0
    want = nv.fp8_quantize(x, block_rows=block_rows, act="relu2")
    x[3, 7], x[129, 399] = float("nan"), float("nan")
    got = nv.fp8_quantize(x, block_rows=block_rows, act="relu2")
    assert torch.equal(got["scale"], want["scale"])
    at = got["codes"].float().isnan()
    assert at.nonzero().tolist() == [[3, 7], [129, 399]]
    assert torch.equal(got["codes"].view(torch.uint8)[~at], want["codes"].view(torch.uint8)[~at])
    assert torch.equal(want["codes"].float(), fp8.quantize_ref(torch.clamp(torch.nan_to_num(x.cpu().float()), min=0) ** 2,
                                                               block_rows)[0].float().cuda())


@pytest.mark.parametrize("act", ["relu2", "swiglu"])
@pytest.mark.parametrize("tokens", [1, 9, 32])
def test_experts(nv, tokens, act):
    """An expert with a NaN in one row of fc1: the tokens that chose it are NaN, the others have their bits."""
    layer = moe.Layer("bf16", tokens, 16, 256, 128, act, seed=tokens)
    want, ids, _ = moe.run(nv, layer, 3, 1, 1)
    bad = int(ids[0, 1])
    layer.w1[1][bad, 77, 3] = 0x7F    # an E4M3 scale that is NaN
    got, i2, _ = moe.run(nv, layer, 3, 1, 1)
    assert torch.equal(i2, ids)
    chose = (ids == bad).any(1)
    assert chose.any() and got[chose].isnan().all()
    assert torch.equal(got[~chose], want[~chose])
