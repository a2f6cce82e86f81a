"""Attention over the paged cache where a workgroup's share holds many tiles: the steady state of the
kernels' loops, their rings of buffers, refills of the window of page ids, items that are split and items
of several tiles that are not.  Every row is compared with a binary64 evaluation; the tolerances are those
of tests/attention_checks.py."""
import numpy as np
import pytest
import torch

import attention_checks as ac

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]
HQ, HK = 16, 4


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return nv


def shares(news, lens, window):
    """Units of (few rows, many rows) in a workgroup's share and, for each kind, how many units the items of
    each request have: the split that the kernels make of a call with both kinds."""
    got = []
    for few, block, unit, count in ((True, 32, 64, 512), (False, 256, 64, 256)):
        total, cost = 0, {}
        for i, (m, n) in enumerate(zip(news, lens)):
            rows = m * (HQ // HK)
            if rows == 0 or (rows <= 32) != few:
                continue
            lo = max(0, n - m + 1 - window) if window else 0
            cost[i] = max(1, -(-n // unit) - lo // unit) + 4
            total += -(-rows // block) * cost[i] * HK
        got.append((-(-total // count), cost))
    return got


def attend(q, k, v, scale, window):
    """attention_checks.attend on the GPU: q [m, HQ, D], k and v [L, HK, D]."""
    m, length, dim = q.shape[0], k.shape[0], q.shape[2]
    back = torch.arange(length - m, length, device="cuda")[:, None] - torch.arange(length, device="cuda")
    hidden = (back < 0) | (back >= window) if window else back < 0
    out, lse, big, d = [], [], [], []
    for h in range(HQ):
        a, b, c = q[:, h].double(), k[:, h * HK // HQ].double(), v[:, h * HK // HQ].double()
        x = ((a @ b.t()) * scale).masked_fill(hidden, -np.inf)
        size = (a.abs() @ b.abs().t()).masked_fill(hidden, 0.0).amax(1)
        top = x.amax(1, keepdim=True)
        w = torch.exp(x - top)
        total = w.sum(1, keepdim=True)
        lse.append((top + total.log()).squeeze(1))
        out.append(w @ c / total)
        big.append(w @ c.abs() / total)
        d.append(2.0 ** -24 * (dim + 4) * scale * size + 2.0 ** -23 * x.masked_fill(hidden, 0.0).abs().amax(1))
    return tuple(torch.stack(t, 1).cpu().numpy() for t in (out, lse, big, d))


def run(nv, news, lens, dim, page, window, dtype, whole_scale=0.0):
    gen = torch.Generator(device="cuda").manual_seed(61)

    def normal(*shape):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)

    table, total = ac.pages_of(lens, page, 3, np.random.default_rng(62))
    table = table.cuda()
    def whole(t, large, small):
        """Two channels of whole numbers, the others 0."""
        pick = torch.randint(0, 1 << 30, t.shape[:2], device="cuda", generator=gen)
        t.zero_()
        t[..., 3], t[..., dim - 1] = large[pick % len(large)].to(dtype), small[pick // 64 % len(small)].to(dtype)

    kc, vc = (torch.full((total, HK, page, dim), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    ks, vs = [], []
    for i, n in enumerate(lens):
        p = torch.arange(n, device="cuda")
        ks.append(normal(n, HK, dim))
        vs.append(normal(n, HK, dim))
        if whole_scale:
            whole(ks[-1], torch.tensor([2000, 1992, -2000, 0], device="cuda"), torch.arange(-8, 9, device="cuda"))
        kc[table[i, p // page].long(), :, p % page], vc[table[i, p // page].long(), :, p % page] = ks[-1], vs[-1]
    q, scale, at, refs = normal(sum(news), HQ, dim) * 1.5, whole_scale or dim ** -0.5, 0, []
    if whole_scale:
        whole(q, torch.tensor([2048, -2048, 0], device="cuda"), torch.tensor([-1, 1, 2], device="cuda"))
    for m, k, v in zip(news, ks, vs):
        refs.append(attend(q[at:at + m], k, v, scale, window))
        if whole_scale:   # binary32 forms the scores exactly: see test_gpu_attention_range.py
            refs[-1] = refs[-1][:3] + (np.full_like(refs[-1][3], 2.0 ** -18),)
        at += m
    out, lse = nv.paged_attn(q, kc, vc, table, ac.starts(news).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                             scale=scale, window=window, want_lse=True)
    ac.check(out.cpu(), lse.cpu(), refs, dtype, max(lens), 8.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window", [0, 5000])
@pytest.mark.parametrize("page", [16, 7, 32])
@pytest.mark.parametrize("dim", [64, 80, 128])
def test_many_rows(nv, dim, page, window, dtype):
    news, lens = [300, 70, 90, 333, 150], [12000, 400, 700, 9001, 611]
    (_, none), (share, cost) = shares(news, lens, window)
    assert share >= 8 and not none
    # items of all tiles in one share, and items split over several
    assert cost[1] <= share and cost[4] <= share and cost[0] > 3 * share and cost[3] > 3 * share
    run(nv, news, lens, dim, page, window, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window", [0, 3000])
@pytest.mark.parametrize("page", [16, 7, 1])
@pytest.mark.parametrize("dim", [64, 80, 128])
def test_few_rows(nv, dim, page, window, dtype):
    # with page 1 a share runs through more page ids than a wave keeps
    news, lens = [1, 2, 8] * 8 + [1] * 20, [8000, 9000, 7777] * 8 + [300] * 20
    (share, cost), (_, none) = shares(news, lens, window)
    assert share >= 5 and not none
    assert cost[30] <= share + 4 and cost[0] > 3 * share
    assert window or share * 64 > 256 * 2
    run(nv, news, lens, dim, page, window, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 80, 128])
def test_both_kinds(nv, dim, dtype):
    news, lens = [1, 300, 4] * 5, [30000, 9000, 20000] * 5
    (few, _), (many, _) = shares(news, lens, 0)
    assert few >= 8 and many >= 20
    run(nv, news, lens, dim, 16, 0, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [1.0, 8.0, 2.0 ** 40])
@pytest.mark.parametrize("dim", [64, 80, 128])
def test_large_scores(nv, dim, scale, dtype):
    # rows that count from a reference, over shares of many tiles, beside rows that do not
    news, lens = [1, 300, 4] * 5, [9000, 3000, 7001] * 5
    (few, _), (many, _) = shares(news, lens, 0)
    assert few >= 8 and many >= 16
    run(nv, news, lens, dim, 16, 0, dtype, scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_a_chunk_among_idle_requests(nv, dim, dtype):
    # no more tokens than requests: the chunk's 240 rows go through the kernel of few rows, in blocks
    news, lens = [0] * 60 + [60] + [1, 0] * 10, [9] * 60 + [5000] + [900, 33] * 10
    assert sum(news) <= len(news) and max(news) * HQ // HK > 32 * 7
    run(nv, news, lens, dim, 16, 0, dtype)
    run(nv, news, lens, dim, 16, 700, dtype)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("news", [1, 40])
def test_a_query_that_is_not_finite_stays_in_its_row(nv, news, bad):
    gen = torch.Generator(device="cuda").manual_seed(63)
    kc, vc = (torch.empty((40, HK, 16, 64), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(2))
    q = torch.empty((news, HQ, 64), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    table, cu = torch.arange(40, dtype=torch.int32, device="cuda")[None], ac.starts([news]).cuda()
    n = torch.tensor([633], dtype=torch.int32).cuda()
    want, want_lse = nv.paged_attn(q, kc, vc, table, cu, n, want_lse=True)
    q[news // 2, 5, 7] = bad
    out, lse = nv.paged_attn(q, kc, vc, table, cu, n, want_lse=True)
    row = torch.zeros((news, HQ), dtype=torch.bool, device="cuda")
    row[news // 2, 5] = True
    assert torch.isnan(out[row]).all() and torch.isnan(lse[row]).all()
    # the others may have had their maximum raised at other keys: equal up to the roundings
    close = (out.float() - want.float()).abs() <= 2.0 ** -7 * (want.float().abs() + vc.float().abs().max())
    assert close[~row].all() and ((lse - want_lse).abs() <= 1e-4)[~row].all()
