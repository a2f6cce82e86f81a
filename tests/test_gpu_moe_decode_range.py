"""The MoE layer at the ends of binary32: activations of an expert that overflow, and small ones whose scales' product
leaves the normal range though the result does not."""
import numpy as np
import pytest
import torch

import test_gpu_moe_decode as moe
import test_gpu_moe_decode_kernels as kernels

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return nv


def one_large_row(tokens, hidden, inter, act, seed):
    """BF16 tokens of 2^57 times a normal number; of every expert's h a few rows are beyond binary32, the others not."""
    layer = moe.Layer("bf16", tokens, 4, hidden, inter, act, seed=seed, x_scale=2.0 ** 57)
    layer.router = torch.zeros_like(layer.router)
    layer.bias = torch.zeros(4)
    codes, sf, glob = layer.w1
    sf = torch.full(sf.shape, 2.0 ** -6).to(moe.FP8).view(torch.uint8)
    at = torch.randperm(inter, generator=torch.Generator().manual_seed(seed))[:3]
    for rows in ((at, at + inter) if act == "swiglu" else (at,)):
        sf[:, rows] = torch.tensor(448.0).to(moe.FP8).view(torch.uint8)
    layer.w1 = (codes, sf, glob * 2.0 ** 7)
    return layer


def by_definition(layer, ids, wts):
    """h in binary32 (overflow is an infinity), then products and sums of the definition: 0 * inf and inf - inf are NaN."""
    x = layer.x.double()
    out = torch.zeros(x.shape, dtype=torch.float64)
    few = 0
    for t in range(len(ids)):
        for e, w in zip(ids[t], wts[t]):
            w1, w2 = (moe.values(m[0][e], m[1][e], m[2][e]) for m in (layer.w1, layer.w2))
            y = w1 @ x[t]
            if layer.act == "swiglu":
                gate, up = y[:layer.inter], y[layer.inter:]
                h = gate * torch.sigmoid(gate) * up
            else:
                h = torch.clamp(y, min=0) ** 2
            # none so near the border that the sum's roundings decide
            border = 2.0 ** 128
            assert ((h.abs() < border / 4) | (h.abs() > border * 4)).all()
            h = h.to(torch.float32).double()
            few += int(torch.isinf(h).sum())
            out[t] += w * (w2 * h).sum(1)
    assert few > 0
    return out


@pytest.mark.parametrize("act", ["relu2", "swiglu"])
@pytest.mark.parametrize("size", [(1, 256, 128), (6, 256, 128), (3, 192, 2112), (1, 192, 2112), (20, 64, 1088)])
def test_infinite_activations(nv, size, act):
    """An output is an infinity where the definition has one, and NaN only where it has NaN."""
    tokens, hidden, inter = size
    for seed in range(2):
        layer = one_large_row(tokens, hidden, inter, act, seed)
        out, ids, wts = moe.run(nv, layer, 2, 1, 1)
        want = by_definition(layer, ids.tolist(), wts.double().tolist()).numpy()
        got = out.double().cpu().numpy()
        assert np.isinf(want).any()
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])


def tiny(tokens):
    """h of about 2^-84, fc2 of one large value everywhere, and globals that bring the sum to about 2^-125."""
    layer = moe.Layer("bf16", tokens, 8, 256, 2048, "relu2", seed=21, x_scale=2.0 ** -50)
    layer.w1 = (layer.w1[0], (layer.w1[1].view(moe.FP8).float() * 256).to(moe.FP8).view(torch.uint8), layer.w1[2])
    codes, sf, glob = layer.w2
    largest = torch.tensor(448.0).to(moe.FP8).view(torch.uint8)
    layer.w2 = (torch.full_like(codes, 0x77), torch.full_like(sf, int(largest)), glob * 2.0 ** -58)
    return layer


@pytest.mark.parametrize("tokens", [1, 6])
def test_scales_whose_product_is_subnormal(nv, tokens):
    """Outputs that are normal numbers of BF16, though h times the global, and the global over the power of two that h is
    scaled by, are not."""
    out = kernels.full(nv, tiny(tokens), 8)
    assert out.abs().median() > 2.0 ** -126


@pytest.mark.parametrize("tokens", [1, 6])
def test_small_activations_beside_a_large_one(nv, tokens):
    """One h is some 2^29 times the others, and fc2 has zeros for it: the others are held to 2^-38 of the large one."""
    layer = moe.Layer("bf16", tokens, 8, 256, 512, "relu2", seed=5)
    layer.w1[1][:] = torch.tensor(2.0 ** -6).to(moe.FP8).view(torch.uint8)
    layer.w1[1][:, 77] = torch.tensor(448.0).to(moe.FP8).view(torch.uint8)
    layer.w2[0][:, :, 77 // 2] &= 0x0F      # the odd one of the pair
    kernels.full(nv, layer, 3)
