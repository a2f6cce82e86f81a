"""Attention at the ends of what it accepts: pages of several GiB."""
import numpy as np
import pytest
import torch

import attention_checks as ac
from test_gpu_attention import f64, normal

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return nv


@pytest.mark.parametrize("news", [1, 40])
@pytest.mark.parametrize("dim", [64, 80, 128])
def test_places_past_32_bit_offsets_in_a_page(nv, dim, news):
    # one page holds the whole cache; a window keeps the keys that are read on both sides of 2^31 bytes
    # from the page's start
    dtype, window, tail = torch.bfloat16, 200, 300
    keys = (1 << 31) // (dim * 2) // 8 * 8 + 130
    page = keys + 6 + (-(keys + 6)) % 8
    rng = np.random.default_rng([41, dim, news])
    q = normal(rng, (news, 2, dim), dtype)
    k, v = normal(rng, (tail, 1, dim), dtype), normal(rng, (tail, 1, dim), dtype)
    kc = torch.empty((1, 1, page, dim), dtype=dtype, device="cuda")
    vc = torch.empty((1, 1, page, dim), dtype=dtype, device="cuda")
    nv.kv_write(k.cuda(), v.cuda(), torch.arange(keys - tail, keys).cuda(), kc, vc)
    out, lse = nv.paged_attn(q.cuda(), kc, vc, torch.zeros((1, 1), dtype=torch.int32).cuda(), ac.starts([news]).cuda(),
                             torch.tensor([keys], dtype=torch.int32).cuda(), window=window, want_lse=True)
    refs = [ac.attend(f64(q), f64(k), f64(v), dim ** -0.5, window)]
    ac.check(out.cpu(), lse.cpu(), refs, dtype, window, 8.0)
