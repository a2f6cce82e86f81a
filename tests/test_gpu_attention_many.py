"""Attention of many requests at once: how a workgroup finds its rows and its share changes with the
number of requests (up to 63 and 64, up to 256, more), and lengths of every kind are mixed."""
import numpy as np
import pytest
import torch

import attention_checks as ac
from test_gpu_attention import TYPES, normal, packed, paged, paged_refs, prompt_refs, run_paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return nv


def mixed_lens(rng, seqs):
    lens = rng.integers(0, 12, seqs)
    lens[rng.permutation(seqs)[:4]] = [150, 64, 65, 33]
    return [int(n) for n in lens]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("seqs", [5, 62, 63, 64, 65, 128, 255, 256, 257, 600])
def test_prompts(nv, seqs, dtype):
    rng = np.random.default_rng([31, seqs])
    lens = mixed_lens(rng, seqs)
    hq, hk, dim, pad = 4, 2, (128 if seqs % 2 else 64), 37
    q, k, v = packed(rng, lens + [pad], hq, hk, dim, dtype)
    n = sum(lens)
    out, lse = nv.prompt_attn(q.cuda(), k.cuda(), v.cuda(), ac.starts(lens).cuda(), want_lse=True)
    refs = prompt_refs(q[:n], k[:n], v[:n], lens, dim ** -0.5)
    ac.check(out[:n].cpu(), lse[:n].cpu(), refs, dtype, max(lens), float(v.abs().max()))
    # rows that follow the last prompt
    assert torch.count_nonzero(out[n:]).item() == 0 and torch.all(lse[n:] == -float("inf")).item()


@pytest.mark.parametrize("order", ["rising", "falling", "one long first", "one long last"])
def test_prompts_in_any_order(nv, order):
    # blocks are taken by their number in the request; every row has to be written once
    lens = {"rising": list(range(1, 90, 4)), "falling": list(range(90, 1, -4)), "one long first": [700] + [3] * 30,
            "one long last": [3] * 30 + [700]}[order]
    rng = np.random.default_rng(32)
    dtype, hq, hk, dim = torch.bfloat16, 6, 2, 128
    q, k, v = packed(rng, lens, hq, hk, dim, dtype)
    out = torch.full((sum(lens), hq, dim), float("nan"), dtype=dtype, device="cuda")
    lse = torch.full((sum(lens), hq), float("nan"), device="cuda")
    nv.prompt_attn(q.cuda(), k.cuda(), v.cuda(), ac.starts(lens).cuda(), out=out, lse=lse)
    ac.check(out.cpu(), lse.cpu(), prompt_refs(q, k, v, lens, dim ** -0.5), dtype, max(lens), float(v.abs().max()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("seqs,chunks", [(62, 0), (63, 2), (64, 0), (64, 2), (65, 1), (130, 3), (300, 0), (300, 4)])
def test_paged(nv, seqs, chunks, dtype):
    rng = np.random.default_rng([33, seqs, chunks])
    news = [1] * seqs
    lens = [int(x) for x in rng.integers(1, 60, seqs)]
    lens[seqs // 2], lens[0] = 900, 1
    for i in range(chunks):
        at = int(rng.integers(0, seqs))
        news[at] = int(rng.integers(20, 60))
        lens[at] = news[at] + int(rng.integers(0, 300))
    news[3], lens[5] = 0, 2
    dim = 64 if chunks == 2 else 128
    x = paged(rng, news, lens, 4, 1, dim, 16, dtype, float("nan"))
    out, lse = run_paged(nv, x)
    ac.check(out.cpu(), lse.cpu(), paged_refs(x[0], x[1], x[2], news, dim ** -0.5), dtype, max(lens), 8.0)


def test_more_free_rows_than_requests(nv):
    # a batch with room for 200 tokens of which 70 requests use 70: the rest is written as 0 / -inf
    rng = np.random.default_rng(34)
    lens = [int(x) for x in rng.integers(1, 40, 70)]
    x = list(paged(rng, [1] * 70, lens, 4, 2, 64, 16, torch.float16, 0.0))
    q = torch.cat([x[0], normal(rng, (130, 4, 64), torch.float16)])
    out, lse = run_paged(nv, [q] + x[1:])
    refs = paged_refs(x[0], x[1], x[2], [1] * 70, 0.125)
    ac.check(out[:70].cpu(), lse[:70].cpu(), refs, torch.float16, max(lens), 8.0)
    assert torch.count_nonzero(out[70:]).item() == 0 and torch.all(lse[70:] == -float("inf")).item()
