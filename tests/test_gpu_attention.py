"""Attention of whole packed prompts and of new tokens over the paged cache against a plain
binary64 evaluation, at the lengths, heads, strides, masks and values where a tiled kernel can go
wrong.  Tolerances: tests/attention_checks.py."""
import ctypes

import numpy as np
import pytest
import torch

import attention_checks as ac

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return nv


def normal(rng, shape, dtype, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(dtype)


def f64(t):
    return t.double().numpy()


def packed(rng, lens, hq, hk, dim, dtype):
    t = sum(lens)
    return normal(rng, (t, hq, dim), dtype, 1.5), normal(rng, (t, hk, dim), dtype), normal(rng, (t, hk, dim), dtype)


def prompt_refs(q, k, v, lens, scale, window=0):
    refs, at = [], 0
    for n in lens:
        refs.append(ac.attend(f64(q[at:at + n]), f64(k[at:at + n]), f64(v[at:at + n]), scale, window))
        at += n
    return refs


# one token; odd and empty lengths; a block of rows and one more; tile edges
PROMPTS = [
    ([1], 1, 1, 64), ([1], 8, 1, 128), ([2, 0, 1, 3], 4, 2, 64), ([63], 4, 4, 64), ([64], 2, 1, 128),
    ([65], 7, 1, 128), ([31, 33, 1, 0, 130], 8, 2, 128), ([257], 4, 2, 64), ([128, 129], 6, 2, 80),
    ([200, 7], 4, 1, 96), ([100], 3, 3, 8), ([97], 2, 2, 40), ([300], 16, 1, 104), ([5] * 40, 4, 2, 64),
    ([0, 0, 0], 2, 1, 64), ([70], 40, 1, 64),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,hq,hk,dim", PROMPTS)
def test_prompt_attention(nv, lens, hq, hk, dim, dtype):
    rng = np.random.default_rng([1, sum(lens), hq, dim])
    q, k, v = packed(rng, lens, hq, hk, dim, dtype)
    out, lse = nv.prompt_attn(q.cuda(), k.cuda(), v.cuda(), ac.starts(lens).cuda(), want_lse=True)
    refs = prompt_refs(q, k, v, lens, dim ** -0.5)
    ac.check(out.cpu(), lse.cpu(), refs, dtype, max(lens), float(v.abs().max()) if v.numel() else 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 1000])
def test_prompt_window(nv, window, dtype):
    lens = [150, 1, 37, 260]
    rng = np.random.default_rng([2, window])
    q, k, v = packed(rng, lens, 4, 2, 64, dtype)
    out, lse = nv.prompt_attn(q.cuda(), k.cuda(), v.cuda(), ac.starts(lens).cuda(), scale=0.2, window=window,
                              want_lse=True)
    ac.check(out.cpu(), lse.cpu(), prompt_refs(q, k, v, lens, 0.2, window), dtype, max(lens), float(v.abs().max()))


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_rounding_is_all(nv, dtype):
    # a longer prompt with peaked and flat rows: the error is that of the two documented roundings
    lens = [700]
    rng = np.random.default_rng(3)
    q, k, v = packed(rng, lens, 4, 2, 128, dtype)
    q[::2] *= 4
    out, lse = nv.prompt_attn(q.cuda(), k.cuda(), v.cuda(), ac.starts(lens).cuda(), want_lse=True)
    refs = prompt_refs(q, k, v, lens, 128 ** -0.5)
    ac.check(out.cpu(), lse.cpu(), refs, dtype, 700, float(v.abs().max()))
    assert ac.rounding_only(out.cpu(), refs, dtype) <= (2 / 3) ** 0.5 * 1.05


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_strided_views(nv, dtype):
    # q, k, v as slices of one fused projection, and as [heads, tokens, dim] transposed
    lens, hq, hk, dim = [70, 45], 6, 2, 64
    t = sum(lens)
    rng = np.random.default_rng(4)
    qkv = normal(rng, (t, hq + 2 * hk, dim), dtype)
    refs = prompt_refs(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], lens, dim ** -0.5)
    vmax = float(qkv.abs().max())
    d = qkv.cuda()
    cu = ac.starts(lens).cuda()
    out, lse = nv.prompt_attn(d[:, :hq], d[:, hq:hq + hk], d[:, hq + hk:], cu, want_lse=True)
    ac.check(out.cpu(), lse.cpu(), refs, dtype, 70, vmax)
    turned = d.transpose(0, 1).contiguous().transpose(0, 1)
    again = nv.prompt_attn(turned[:, :hq], turned[:, hq:hq + hk], turned[:, hq + hk:], cu)
    assert torch.equal(again, out)
    wide = torch.zeros((t, hq + 2 * hk, dim + 24), dtype=dtype, device="cuda")   # rows with gaps
    wide[:, :, 8:8 + dim] = d
    w = wide[:, :, 8:8 + dim]
    assert torch.equal(nv.prompt_attn(w[:, :hq], w[:, hq:hq + hk], w[:, hq + hk:], cu), out)


def test_prompt_padding_rows_are_zero(nv):
    # a batch padded to 100 tokens: the rows after the last prompt are 0 / -inf
    rng = np.random.default_rng(5)
    q, k, v = packed(rng, [100], 4, 2, 64, torch.bfloat16)
    k[40:] = float("nan")
    v[40:] = float("inf")
    cu = torch.tensor([0, 13, 40], dtype=torch.int32).cuda()
    out = torch.full((100, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    _, lse = nv.prompt_attn(q.cuda(), k.cuda(), v.cuda(), cu, out=out, want_lse=True)
    refs = prompt_refs(q[:40], k[:40], v[:40], [13, 27], 0.125)
    ac.check(out[:40].cpu(), lse[:40].cpu(), refs, torch.bfloat16, 27, float(v[:40].abs().max()))
    assert torch.count_nonzero(out[40:]).item() == 0
    assert torch.all(lse[40:] == -float("inf")).item()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_prompt_hidden_values_do_not_leak(nv, dtype, bad):
    # a later token's key and value are not finite, at the start, middle and end of a tile
    lens, hq, hk, dim = [150], 4, 2, 64
    rng = np.random.default_rng(6)
    for at in (0, 1, 40, 63, 64, 100, 149):
        q, k, v = packed(rng, lens, hq, hk, dim, dtype)
        v[at, 0, 5] = bad
        v[at, 1, 63] = -bad
        out, lse = nv.prompt_attn(q.cuda(), k.cuda(), v.cuda(), ac.starts(lens).cuda(), want_lse=True)
        refs = prompt_refs(q, k, v, lens, dim ** -0.5)
        ac.check(out.cpu(), lse.cpu(), refs, dtype, 150, float(v[torch.isfinite(v)].abs().max()))
        k[at, 0, 3] = bad
        out, lse = nv.prompt_attn(q.cuda(), k.cuda(), v.cuda(), ac.starts(lens).cuda(), want_lse=True)
        assert torch.isfinite(out[:at]).all() and torch.isfinite(lse[:at]).all()
        refs = prompt_refs(q[:at], k[:at], v[:at], [at], dim ** -0.5) if at else []
        if at:
            ac.check(out[:at].cpu(), lse[:at].cpu(), refs, dtype, 150, 8.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_scores_of_minus_infinity(nv, dtype):
    # keys of -inf where q is positive: those keys have weight 0, a row with no other key is empty
    lens, dim = [90], 64
    rng = np.random.default_rng(7)
    q, k, v = packed(rng, lens, 2, 1, dim, dtype)
    q[:, :, 0] = q[:, :, 0].abs() + 0.5
    k[:70, 0, 0] = -float("inf")
    out, lse = nv.prompt_attn(q.cuda(), k.cuda(), v.cuda(), ac.starts(lens).cuda(), want_lse=True)
    refs = prompt_refs(q, k, v, lens, dim ** -0.5)
    refs = [tuple(np.nan_to_num(x, nan=0.0, posinf=0.0) if i == 3 else x for i, x in enumerate(r)) for r in refs]
    clean = k.clone()
    clean[:70, 0, 0] = 0
    d = ac.attend(f64(q), f64(clean), f64(v), dim ** -0.5)[3]
    refs = [(refs[0][0], refs[0][1], refs[0][2], d)]
    ac.check(out.cpu(), lse.cpu(), refs, dtype, 90, float(v.abs().max()))
    assert torch.count_nonzero(out[:70]).item() == 0


def test_prompt_large_scores_and_growing_maxima(nv):
    # the running maximum rises in every tile, falls off, and jumps by less and by more than 2^8
    dtype, dim = torch.bfloat16, 64
    rng = np.random.default_rng(8)
    q, k, v = packed(rng, [400], 2, 1, dim, dtype)
    q[:, :, 0] = 8.0
    for step in (0.5, 4.0, 30.0, -4.0):
        k[:, 0, 0] = torch.arange(400).to(dtype) * step / 8
        out, lse = nv.prompt_attn(q.cuda(), k.cuda(), v.cuda(), ac.starts([400]).cuda(), scale=1.0, want_lse=True)
        ac.check(out.cpu(), lse.cpu(), prompt_refs(q, k, v, [400], 1.0), dtype, 400, float(v.abs().max()))


# ---------------------------------------------------------------- paged

def paged(rng, news, lens, hq, hk, dim, page, dtype, fill):
    t = sum(news)
    q = normal(rng, (t, hq, dim), dtype, 1.5)
    ks = [normal(rng, (n, hk, dim), dtype) for n in lens]
    vs = [normal(rng, (n, hk, dim), dtype) for n in lens]
    table, total = ac.pages_of(lens, page, 3, rng)
    return (q, ks, vs, table, ac.fill_cache(ks, table, page, total, fill), ac.fill_cache(vs, table, page, total, fill),
            ac.starts(news), torch.tensor(lens, dtype=torch.int32))


def paged_refs(q, ks, vs, news, scale, window=0):
    refs, at = [], 0
    for m, k, v in zip(news, ks, vs):
        refs.append(ac.attend(f64(q[at:at + m]), f64(k), f64(v), scale, window))
        at += m
    return refs


def run_paged(nv, x, **kw):
    q, _, _, table, kc, vc, cu, lens = x
    return nv.paged_attn(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), cu.cuda(), lens.cuda(), want_lse=True, **kw)


# new tokens and cached keys of each request, heads, dim, page
PAGED = [
    ([1], [1], 4, 1, 64, 16), ([1], [1000], 8, 2, 128, 16), ([1], [4097], 4, 1, 128, 64),
    ([1, 1, 1], [5, 300, 129], 7, 1, 128, 16), ([1] * 9, [1, 2, 31, 32, 33, 127, 128, 129, 700], 8, 2, 64, 8),
    ([0, 1, 0, 2], [5, 40, 0, 77], 4, 2, 64, 16), ([3, 1, 4], [50, 600, 4], 8, 2, 96, 24),
    ([8], [500], 4, 1, 80, 1), ([70], [70], 4, 1, 64, 16), ([100], [700], 8, 2, 128, 32),
    ([1, 90, 1, 1, 33], [900, 1100, 3, 64, 33], 8, 2, 128, 16), ([5, 200], [64, 333], 16, 1, 64, 128),
    ([1], [513], 64, 1, 64, 16), ([2, 1], [300, 20], 40, 1, 128, 7), ([300], [2000], 4, 2, 64, 24),
    ([9, 9, 9, 9], [9, 10, 200, 2048], 32, 8, 128, 16),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news,lens,hq,hk,dim,page", PAGED)
def test_paged_attention(nv, news, lens, hq, hk, dim, page, dtype):
    rng = np.random.default_rng([11, sum(news), sum(lens), page])
    x = paged(rng, news, lens, hq, hk, dim, page, dtype, float("nan"))   # unused places hold NaN
    out, lse = run_paged(nv, x)
    ac.check(out.cpu(), lse.cpu(), paged_refs(x[0], x[1], x[2], news, dim ** -0.5), dtype, max(lens), 8.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window", [1, 5, 64, 129, 5000])
def test_paged_window(nv, window, dtype):
    news, lens = [1, 6, 80, 1], [400, 130, 300, 2500]
    rng = np.random.default_rng([12, window])
    x = paged(rng, news, lens, 8, 2, 64, 16, dtype, float("inf"))
    out, lse = run_paged(nv, x, window=window, scale=0.3)
    ac.check(out.cpu(), lse.cpu(), paged_refs(x[0], x[1], x[2], news, 0.3, window), dtype, max(lens), 8.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_paged_rows_that_see_nothing(nv, dtype):
    # more new tokens than keys (the first rows see nothing), no keys at all, and padding tokens
    news, lens = [5, 3, 1, 60], [2, 0, 0, 10]
    rng = np.random.default_rng(13)
    x = list(paged(rng, news, lens, 4, 2, 64, 16, dtype, float("nan")))
    pad = 7
    x[0] = torch.cat([x[0], normal(rng, (pad, 4, 64), dtype)])
    out, lse = run_paged(nv, x)
    t = sum(news)
    ac.check(out[:t].cpu(), lse[:t].cpu(), paged_refs(x[0], x[1], x[2], news, 0.125), dtype, 10, 8.0)
    for rows in (slice(0, 3), slice(5, 9), slice(9, 59), slice(t, t + pad)):
        assert torch.count_nonzero(out[rows]).item() == 0 and torch.all(lse[rows] == -float("inf")).item()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news", [3, 70])
def test_paged_hidden_values_do_not_leak(nv, news, dtype):
    rng = np.random.default_rng([14, news])
    lens = [200]
    for at in (200 - news, 200 - news // 2, 199):
        x = paged(rng, [news], lens, 4, 2, 64, 16, dtype, 0.0)
        q, ks, vs, table, kc, vc, cu, ln = x
        vs[0][at, 0, 9] = float("nan")
        vs[0][at, 1, 3] = float("inf")
        vc = ac.fill_cache(vs, table, 16, vc.shape[0], 0.0)
        out, lse = run_paged(nv, (q, ks, vs, table, kc, vc, cu, ln))
        ac.check(out.cpu(), lse.cpu(), paged_refs(q, ks, vs, [news], 0.125), dtype, 200, 8.0)


def test_paged_equals_prompt_attention(nv):
    # a prompt in one call, and in chunks over the cache: the same numbers up to the two roundings
    dtype, hq, hk, dim, page, n = torch.bfloat16, 8, 2, 128, 16, 333
    rng = np.random.default_rng(15)
    q, k, v = packed(rng, [n], hq, hk, dim, dtype)
    whole, lse = nv.prompt_attn(q.cuda(), k.cuda(), v.cuda(), ac.starts([n]).cuda(), want_lse=True)
    table, total = ac.pages_of([n], page, 0, rng)
    kc, vc = ac.fill_cache([k], table, page, total, 0.0).cuda(), ac.fill_cache([v], table, page, total, 0.0).cuda()
    at = 0
    for m in (100, 1, 31, 1, 200):
        out, part = nv.paged_attn(q[at:at + m].cuda(), kc, vc, table.cuda(), ac.starts([m]).cuda(),
                                  torch.tensor([at + m], dtype=torch.int32).cuda(), want_lse=True)
        refs = [ac.attend(f64(q[at:at + m]), f64(k[:at + m]), f64(v[:at + m]), dim ** -0.5)]
        ac.check(out.cpu(), part.cpu(), refs, dtype, n, float(v.abs().max()))
        ac.check(whole[at:at + m].cpu(), lse[at:at + m].cpu(), refs, dtype, n, float(v.abs().max()))
        at += m


def test_paged_bad_page_ids_read_as_zeros(nv):
    dtype = torch.float16
    rng = np.random.default_rng(16)
    q, ks, vs, table, kc, vc, cu, ln = paged(rng, [1], [100], 4, 2, 64, 16, dtype, 0.0)
    table = table.clone()
    table[0, 2], table[0, 4] = -5, kc.shape[0]
    for p in (2, 4):
        ks[0][16 * p:16 * p + 16] = 0
        vs[0][16 * p:16 * p + 16] = 0
    out, lse = run_paged(nv, (q, ks, vs, table, kc, vc, cu, ln))
    ac.check(out.cpu(), lse.cpu(), paged_refs(q, ks, vs, [1], 0.125), dtype, 100, 8.0)


def test_paged_keys_past_the_table_do_not_exist(nv):
    dtype = torch.float16
    rng = np.random.default_rng(17)
    x = list(paged(rng, [1], [64], 4, 2, 64, 16, dtype, 0.0))
    want, _ = run_paged(nv, x)
    x[7] = torch.tensor([1 << 30], dtype=torch.int32)
    got, _ = run_paged(nv, x)
    assert torch.equal(got, want)


@pytest.mark.parametrize("news", [1, 40])
def test_cache_past_32_bit_offsets(nv, news):
    # pages on both sides of 4 GiB
    dtype, hk, dim, page = torch.float16, 8, 128, 64
    pages = (5 << 30) // (hk * dim * page * 2)
    rng = np.random.default_rng(18)
    q = normal(rng, (news, 16, dim), dtype)
    k, v = normal(rng, (200, hk, dim), dtype), normal(rng, (200, hk, dim), dtype)
    kc = torch.empty((pages, hk, page, dim), dtype=dtype, device="cuda")
    vc = torch.empty((pages, hk, page, dim), dtype=dtype, device="cuda")
    table = torch.tensor([[pages - 1, 3, pages - 2, pages // 2]], dtype=torch.int32)
    slots = torch.tensor([int(table[0, p // page]) * page + p % page for p in range(200)], dtype=torch.int64)
    nv.kv_write(k.cuda(), v.cuda(), slots.cuda(), kc, vc)
    out, lse = nv.paged_attn(q.cuda(), kc, vc, table.cuda(), ac.starts([news]).cuda(),
                             torch.tensor([200], dtype=torch.int32).cuda(), want_lse=True)
    ac.check(out.cpu(), lse.cpu(), [ac.attend(f64(q), f64(k), f64(v), dim ** -0.5)], dtype, 200, 8.0)


# ---------------------------------------------------------------- determinism, streams, graphs, buffers

def test_same_bits_every_time(nv):
    rng = np.random.default_rng(19)
    news, lens = [1, 130, 1, 4], [3000, 900, 17, 1200]
    x = paged(rng, news, lens, 8, 2, 128, 16, torch.bfloat16, 0.0)
    first = run_paged(nv, x)
    for _ in range(3):
        again = run_paged(nv, x)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_other_stream_and_given_buffers(nv):
    rng = np.random.default_rng(20)
    x = paged(rng, [1, 50, 2], [3000, 300, 9], 8, 2, 128, 16, torch.float16, 0.0)
    want, want_lse = run_paged(nv, x)
    q, _, _, table, kc, vc, cu, ln = (t.cuda() if isinstance(t, torch.Tensor) else t for t in x)
    pq, pk, pv = (t.cuda() for t in packed(rng, [300], 4, 2, 64, torch.float16))
    pcu = ac.starts([300]).cuda()
    pwant = nv.prompt_attn(pq, pk, pv, pcu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    size = nv.paged_attn_workspace_size(3, 53, 8, 2, 128)
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    torch.cuda.synchronize()
    got = nv.paged_attn(q, kc, vc, table, cu, ln, out=out, lse=lse, workspace=ws, stream=s)
    fresh = nv.paged_attn(q, kc, vc, table, cu, ln, stream=s)
    pgot = nv.prompt_attn(pq, pk, pv, pcu, stream=s)
    s.synchronize()
    assert got[0] is out and got[1] is lse
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and torch.equal(fresh, want)
    assert torch.equal(pgot, pwant)


def test_graph_replays_follow_the_device_lengths(nv):
    # one captured decode step (maps, write, attention) replayed for several steps: the lengths, the
    # table and the cache change on the device between the replays
    dtype, hq, hk, dim, page, n = torch.bfloat16, 8, 2, 128, 16, 3
    rng = np.random.default_rng(21)
    lens = [15, 200, 31]
    ks = [normal(rng, (m, hk, dim), dtype) for m in lens]
    vs = [normal(rng, (m, hk, dim), dtype) for m in lens]
    table, total = ac.pages_of(lens, page, 0, rng)
    free = torch.arange(total, total + 20, dtype=torch.int32).cuda()
    table = torch.cat([table, torch.full((3, 2), -1, dtype=torch.int32)], 1)
    kc = torch.zeros((total + 20, hk, page, dim), dtype=dtype, device="cuda")
    vc = torch.zeros_like(kc)
    kc[:total] = ac.fill_cache(ks, table, page, total, 0.0).cuda()
    vc[:total] = ac.fill_cache(vs, table, page, total, 0.0).cuda()
    q = torch.zeros((n, hq, dim), dtype=dtype, device="cuda")
    k, v = torch.zeros((n, hk, dim), dtype=dtype, device="cuda"), torch.zeros((n, hk, dim), dtype=dtype, device="cuda")
    ctx, news, dtable = torch.tensor(lens, dtype=torch.int32).cuda(), torch.ones(n, dtype=torch.int32).cuda(), table.cuda()
    maps = {"cu_new": torch.zeros(n + 1, dtype=torch.int32, device="cuda"),
            "kv_lens": torch.zeros(n, dtype=torch.int32, device="cuda"),
            "slot_map": torch.zeros(n, dtype=torch.int64, device="cuda"),
            "positions": torch.zeros(n, dtype=torch.int32, device="cuda"),
            "taken": torch.zeros(1, dtype=torch.int32, device="cuda")}
    out, lse = torch.empty_like(q), torch.empty((n, hq), device="cuda")
    ws = torch.empty(nv.paged_attn_workspace_size(n, n, hq, hk, dim), dtype=torch.uint8, device="cuda")

    def step():
        nv.page_maps(ctx, news, dtable, free, page, n, out=maps)
        nv.kv_write(k, v, maps["slot_map"], kc, vc)
        nv.paged_attn(q, kc, vc, dtable, maps["cu_new"], maps["kv_lens"], out=out, lse=lse, workspace=ws)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = dtable.clone(), kc.clone(), vc.clone()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    for t, c in zip((dtable, kc, vc), keep):
        t.copy_(c)
    with torch.cuda.graph(graph, stream=s):
        step()
    for _ in range(4):
        qn, kn, vn = normal(rng, (n, hq, dim), dtype), normal(rng, (n, hk, dim), dtype), normal(rng, (n, hk, dim), dtype)
        q.copy_(qn), k.copy_(kn), v.copy_(vn)
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        ks = [torch.cat([a, b[None]]) for a, b in zip(ks, kn)]
        vs = [torch.cat([a, b[None]]) for a, b in zip(vs, vn)]
        ac.check(out.cpu(), lse.cpu(), paged_refs(qn, ks, vs, [1] * n, dim ** -0.5), dtype, 210, 8.0)
        ctx.copy_(maps["kv_lens"])
        taken = int(maps["taken"].item())
        free.copy_(torch.cat([free[taken:], free[:taken]]))


@pytest.mark.parametrize("news", [[1, 1], [40, 1]])
def test_nothing_is_written_outside_the_buffers(nv, news):
    dtype, hq, hk, dim = torch.bfloat16, 8, 2, 80
    rng = np.random.default_rng(22)
    x = paged(rng, news, [600, 333], hq, hk, dim, 16, dtype, 0.0)
    t, pad = sum(news), 4096
    buf = torch.full((t * hq * dim * 2 + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
    lbuf = torch.full((t * hq * 4 + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
    size = nv.paged_attn_workspace_size(2, t, hq, hk, dim)
    wbuf = torch.full((size + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
    out = buf[pad:-pad].view(dtype).view(t, hq, dim)
    lse = lbuf[pad:-pad].view(torch.float32).view(t, hq)
    run = {"out": out, "lse": lse, "workspace": wbuf[pad:-pad]}
    q, _, _, table, kc, vc, cu, ln = (a.cuda() if isinstance(a, torch.Tensor) else a for a in x)
    nv.paged_attn(q, kc, vc, table, cu, ln, **run)
    pq, pk, pv = (a.cuda() for a in packed(rng, [t], hq, hk, dim, dtype))
    ac.check(out.cpu(), lse.cpu(), paged_refs(x[0], x[1], x[2], news, dim ** -0.5), dtype, 600, 8.0)
    nv.prompt_attn(pq, pk, pv, ac.starts([t]).cuda(), out=out, lse=lse)
    torch.cuda.synchronize()
    for b in (buf, lbuf, wbuf):
        assert torch.all(b[:pad] == 0x5A).item() and torch.all(b[-pad:] == 0x5A).item()


def test_c_entry_points_refuse_on_a_gpu(nv):
    # the last check before a launch: a workspace that is too small or not aligned
    L = nv.lib()
    need = nv.paged_attn_workspace_size(2, 2, 8, 2, 64)
    t = torch.zeros(need + 512, dtype=torch.uint8, device="cuda")
    p = ctypes.c_void_p(t.data_ptr() // 256 * 256 + 256)
    args = [p, 0, p, p, p, p, p, 2, 2, 8, 2, 64, 16, 1, 1, 512, 64, 0.125, 0, p, None]
    assert L.nvfp4_paged_attn(*args, p, need - 1, None) == nv.NVFP4_EWORKSPACE
    assert L.nvfp4_paged_attn(*args, ctypes.c_void_p(p.value + 16), need, None) == nv.NVFP4_EWORKSPACE
