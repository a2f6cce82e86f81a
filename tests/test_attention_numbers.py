"""Numbers that do not fit the C entry points' 32-bit arguments are refused by the binding instead of being
cut to their low bits."""
import pytest
import torch

BF16 = torch.bfloat16
WIDE = [(1 << 32) + 5, 1 << 32, 1 << 31, -(1 << 32), -(1 << 31) - 1]


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    return nv


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


@pytest.mark.parametrize("number", WIDE)
def test_wide_numbers_are_refused(nv, number):
    q, kv, cache = (torch.zeros(s, dtype=BF16) for s in ((4, 4, 64), (4, 2, 64), (3, 2, 16, 64)))
    with pytest.raises(ValueError, match="window must fit 32 bits"):
        nv.prompt_attn(q, kv, kv, i32(2), window=number)
    with pytest.raises(ValueError, match="window must fit 32 bits"):
        nv.paged_attn(q, cache, cache, i32(2, 4), i32(3), i32(2), window=number)
    with pytest.raises(ValueError, match="page_size must fit 32 bits"):
        nv.page_maps(i32(2), i32(2), i32(2, 4), i32(3), number, 8)


@pytest.mark.gpu
def test_wide_shapes_are_refused(nv):
    # 64 GiB that nothing touches
    cache = torch.empty((1, 1, (1 << 32) + 16, 8), dtype=BF16, device="cuda")
    q, slots, ints = torch.zeros((2, 1, 8), dtype=BF16, device="cuda"), torch.zeros(2, dtype=torch.int64).cuda(), i32(3).cuda()
    try:
        with pytest.raises(ValueError, match="page_size must fit 32 bits"):
            nv.kv_write(q, q, slots, cache, cache)
        with pytest.raises(ValueError, match="page_size must fit 32 bits"):
            nv.paged_attn(q, cache, cache, i32(2, 1).cuda(), ints, i32(2).cuda())
    finally:
        del cache
        torch.cuda.empty_cache()


@pytest.mark.gpu
def test_head_dimension_of_zero_is_refused(nv):
    q, cache = torch.zeros((2, 1, 0), dtype=BF16, device="cuda"), torch.zeros((1, 1, 4, 0), dtype=BF16, device="cuda")
    with pytest.raises(nv.Nvfp4Error):
        nv.prompt_attn(q, q, q, i32(2).cuda())
    with pytest.raises(nv.Nvfp4Error):
        nv.paged_attn(q, cache, cache, i32(2, 1).cuda(), i32(3).cuda(), i32(2).cuda())
