"""Numbers that the C entry points take in 32 bits, and that ctypes would cut: an activation of 2^32 + 1 ran as SwiGLU on
operands that were checked for none, and read behind them.  No GPU: refused before a device is asked for."""
import pytest
import torch


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    return nv


def z(*s, dtype=torch.float16):
    return torch.zeros(s, dtype=dtype)


@pytest.mark.parametrize("act", [(1 << 32) + 1, (1 << 32) + 2, 1 << 32, -(1 << 32) + 1, 1 << 31])
def test_activations(nv, act):
    u8, f32 = torch.uint8, torch.float32
    for call in (lambda: nv.act_quant(z(4, 256), act=act), lambda: nv.mx_quantize(z(4, 256), act=act),
                 lambda: nv.fp8_quantize(z(4, 256), act=act),
                 lambda: nv.moe_decode(z(4, 256), z(16, 256), z(16, dtype=f32), z(16, 128, 128, dtype=u8), z(16, 128, 16, dtype=u8),
                                       z(16, dtype=f32), z(16, 256, 64, dtype=u8), z(16, 256, 8, dtype=u8), z(16, dtype=f32), 4,
                                       act=act)):
        with pytest.raises(ValueError, match="act must fit 32 bits"):
            call()


def test_workspace_size(nv):
    good = [4, 16, 4, 256, 128]
    assert nv.moe_decode_workspace_size(*good) > 0
    for i in range(5):
        with pytest.raises(ValueError, match="must fit 32 bits"):
            nv.moe_decode_workspace_size(*good[:i], good[i] + (1 << 32), *good[i + 1:])
