"""Attention at the ends of what it accepts: pages of several GiB, scores of any size, values at the ends of
their type and weights far below the largest."""
import numpy as np
import pytest
import torch

import attention_checks as ac
from test_gpu_attention import f64, normal, paged_refs, prompt_refs

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


# ---------------------------------------------------------------- large scores
#
# Scores are whole numbers below 2^24 here (two channels of q and k are whole numbers, the others 0), so
# binary32 forms them exactly whatever the order, and what is left is the exponent's argument: (s_j - top)
# scale log2 e with a relative error of at most 3 x 2^-24.  Keys further than 2^21 below the top in weight do
# not count; for the others that is at most 21 x 3 x 2^-24 < 2^-18 of the weight.
ARGUMENT = 2.0 ** -18

# the large part of key j's score, in units of 2048
PATTERNS = {
    "level": lambda j: 2000 + 0 * j,
    "negative": lambda j: -2000 + 0 * j,
    "rising": lambda j: 8 * (j % 250),
    "falling": lambda j: 8 * (249 - j % 250),
    "rises late": lambda j: np.where(j % 256 == 150, 2000, 0),
    "from far below": lambda j: np.where(j < 70, -2000, np.where(j < 140, 0, 3)),
    "signs": lambda j: np.where(j % 3 == 0, 2000, -2000),
}
SCALES = [0, 2, 6, 10, 30, 60, 90]   # log2


def whole_numbers(rng, rows, hq, keys, hk, dim, dtype, pattern):
    q, k = np.zeros((rows, hq, dim)), np.zeros((keys, hk, dim))
    # large scores of both signs in one wave, and rows without them
    q[..., 3], q[..., dim - 1] = rng.choice([2048, 2048, 2048, -2048, 0], (rows, hq)), rng.choice([-1, 1, 2], (rows, hq))
    k[..., 3] = PATTERNS[pattern](np.arange(keys))[:, None]
    k[..., dim - 1] = rng.integers(-8, 9, (keys, hk))
    return torch.from_numpy(q).to(dtype), torch.from_numpy(k).to(dtype), normal(rng, (keys, hk, dim), dtype)


def exact_scores(refs):
    return [(o, lse, big, np.where(np.isfinite(lse), ARGUMENT, 0.0)) for o, lse, big, _ in refs]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pattern", PATTERNS)
def test_prompt_with_large_scores(nv, pattern, dtype):
    n = 330
    for dim in (64, 128):
        rng = np.random.default_rng([42, dim])
        q, k, v = whole_numbers(rng, n, 4, n, 2, dim, dtype, pattern)
        for e in SCALES:
            out, lse = nv.prompt_attn(q.cuda(), k.cuda(), v.cuda(), ac.starts([n]).cuda(), scale=2.0 ** e, want_lse=True)
            ac.check(out.cpu(), lse.cpu(), exact_scores(prompt_refs(q, k, v, [n], 2.0 ** e)), dtype, n, 8.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("news,lens", [([1, 5], [2000, 333]), ([1, 70], [300, 900])])
def test_paged_with_large_scores(nv, news, lens, pattern, dtype):
    # split over workgroups, whose parts have references of their own
    dim, page = 64, 16
    rng = np.random.default_rng([43, sum(news)])
    parts = [whole_numbers(rng, m, 4, n, 2, dim, dtype, pattern) for m, n in zip(news, lens)]
    q, ks, vs = torch.cat([x[0] for x in parts]), [x[1] for x in parts], [x[2] for x in parts]
    table, total = ac.pages_of(lens, page, 3, rng)
    kc, vc = (ac.fill_cache(x, table, page, total, float("nan")).cuda() for x in (ks, vs))
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    for e in SCALES:
        out, lse = nv.paged_attn(q.cuda(), kc, vc, table.cuda(), ac.starts(news).cuda(), ln, scale=2.0 ** e, want_lse=True)
        ac.check(out.cpu(), lse.cpu(), exact_scores(paged_refs(q, ks, vs, news, 2.0 ** e)), dtype, max(lens), 8.0)


def winners(q, k, scale):
    """The key of each row's largest score, that score, and whether no rounding of binary32 can change who
    wins: the next one is further below than both scores' bounds (see attention_checks) and 2^60 in weight."""
    n, hq, dim = q.shape
    best, top, sure, bound = (np.zeros((n, hq), t) for t in (int, float, bool, float))
    for i in range(n):
        for h in range(hq):
            kk = k[:i + 1, h * k.shape[1] // hq]
            s = scale * (kk @ q[i, h])
            d = 2.0 ** -24 * (dim + 4) * scale * (np.abs(kk) @ np.abs(q[i, h])).max()
            best[i, h], top[i, h], bound[i, h] = s.argmax(), s.max(), d
            sure[i, h] = i == 0 or s.max() - np.partition(s, -2)[-2] > 4 * d + 42
    return best, top, sure, bound


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size,scale", [(1.0, 2.0 ** 24), (1.0, 2.0 ** 30), (1.0, 2.0 ** 90), (2e4, 128 ** -0.5)])
def test_one_key_takes_all(nv, size, scale, dtype):
    # ordinary numbers with a large scale, and large finite numbers with an ordinary one
    n, dim = 200, 128
    rng = np.random.default_rng(44)
    q, k = (torch.from_numpy(np.clip(rng.standard_normal((n, h, dim)) * size, -6e4, 6e4)).to(dtype) for h in (4, 2))
    v = normal(rng, (n, 2, dim), dtype)
    out, lse = nv.prompt_attn(q.cuda(), k.cuda(), v.cuda(), ac.starts([n]).cuda(), scale=scale, want_lse=True)
    best, top, sure, bound = winners(f64(q), f64(k), scale)
    assert sure.mean() > 0.9
    want = f64(v)[best, np.arange(4)[None] // 2]
    u = ac.UNIT[dtype]
    g, x = out.cpu().double().numpy(), lse.cpu().double().numpy()
    assert np.isfinite(g).all() and np.isfinite(x).all()
    # one rounding of the weight and one of the result
    assert np.all(np.abs(g - want)[sure] <= (2 * u * 1.01 * np.abs(want) + 2.0 ** -24)[sure])
    assert np.all(np.abs(x - top) <= bound + 2.0 ** -22 * np.abs(top) + np.log(n))


# ---------------------------------------------------------------- values and weights at the ends of their types

def both_ways(nv, q, k, v, scale):
    """The last row of a prompt (with all its keys) and the same row as a decode step, and the rows before
    them as one chunk over the cache."""
    n, hk, dim = k.shape
    page = 16
    table, total = ac.pages_of([n], page, 1, np.random.default_rng(45))
    kc, vc = (ac.fill_cache([x], table, page, total, 0.0).cuda() for x in (k, v))
    yield n, nv.prompt_attn(q.cuda(), k.cuda(), v.cuda(), ac.starts([n]).cuda(), scale=scale, want_lse=True)
    for m in (1, 100):
        yield m, nv.paged_attn(q[-m:].cuda(), kc, vc, table.cuda(), ac.starts([m]).cuda(),
                               torch.tensor([n], dtype=torch.int32).cuda(), scale=scale, want_lse=True)


@pytest.mark.parametrize("size", [3e38, 2.0 ** -118])
@pytest.mark.parametrize("dim", [64, 128])
def test_bf16_values_at_the_ends_of_the_range(nv, dim, size):
    # one value per channel near the largest of the type, and a later key that outweighs all before it by a
    # factor of 220: less than makes the running maximum follow.  The weighted sum stays below the largest
    # binary32 as long as no weight exceeds 1.
    dtype, n = torch.bfloat16, 300
    rng = np.random.default_rng([46, dim])
    q, k = torch.zeros((n, 4, dim), dtype=dtype), torch.zeros((n, 2, dim), dtype=dtype)
    q[:, :, 5] = 1.0
    k[160, :, 5] = 5.375
    if size > 1:
        v = normal(rng, (n, 2, dim), dtype, 1e30)
        v[160] = torch.from_numpy(rng.choice([-3e38, 3e38], (2, dim))).to(dtype)
    else:
        v = normal(rng, (n, 2, dim), dtype, size)
    for m, (out, lse) in both_ways(nv, q, k, v, 1.0):
        refs = [ac.attend(f64(q)[-m:], f64(k), f64(v), 1.0)]
        ac.check(out.cpu(), lse.cpu(), refs, dtype, n, 0.0)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("first", [True, False])
def test_fp16_weights_far_below_the_largest(nv, first, dim):
    # 4000 keys whose weight is 2^-25.6 of the largest, which is on a value of 0: together they are the
    # result.  The rounding of a weight to the type is at most 2^-31 of the largest each.
    dtype, n = torch.float16, 4000
    rng = np.random.default_rng([47, dim])
    q, k = torch.zeros((n, 4, dim), dtype=dtype), torch.zeros((n, 2, dim), dtype=dtype)
    q[:, :, 7] = 1.0
    k[:, :, 7] = -25.6
    top = 0 if first else n - 200
    k[top, :, 7] = 0.0
    v = torch.from_numpy(rng.uniform(0.5, 1.0, (n, 2, dim))).to(dtype)
    v[top] = 0.0
    u, scale = ac.UNIT[dtype], float(np.log(2.0))
    for m, (out, lse) in both_ways(nv, q, k, v, scale):
        rows = min(m, 50)     # the last ones
        want, want_lse, big, d = ac.attend(f64(q)[-rows:], f64(k), f64(v), scale)
        tol = 1.05 * (u * np.abs(want) + (u + 2 * d[..., None] + 2.0 ** -21 + 2 * n * 2.0 ** -24) * big) + n * 2.0 ** -31 + \
            2.0 ** -25
        assert np.all(np.abs(out[-rows:].cpu().double().numpy() - want) <= tol)
        assert np.all(np.abs(lse[-rows:].cpu().double().numpy() - want_lse) <= 2 * d + 2.0 ** -20 + n * 2.0 ** -24)
