"""Page and slot maps and the cache writer against plain loops on the host (equal, they compute no
rounded numbers)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return nv


def maps_ref(ctx, new, table, free, page, tokens):
    table = table.copy()
    width = table.shape[1]
    slots, positions = np.full(tokens, -1, np.int64), np.full(tokens, -1, np.int32)
    cu, t, taken = [0], 0, 0
    for i, (c, m) in enumerate(zip(ctx, new)):
        c, m = max(c, 0), max(m, 0)
        held = min(-(-c // page), width)
        need = min(-(-(c + m) // page), width) - held
        for j in range(m):
            pos, here = c + j, t + j
            if here >= tokens:
                continue
            positions[here] = pos
            col = pos // page
            got = -1
            if col < held:
                got = table[i, col]
            elif col < width:
                f = taken + col - held
                got = free[f] if f < len(free) else -1
                if pos % page == 0:
                    table[i, col] = got
            if got >= 0:
                slots[here] = int(got) * page + pos % page
        t += m
        taken += need
        cu.append(t)
    lens = [max(c, 0) + max(m, 0) for c, m in zip(ctx, new)]
    return {"cu_new": np.array(cu), "kv_lens": np.array(lens), "slot_map": slots, "positions": positions,
            "taken": np.array([taken]), "table": table}


def run_maps(nv, ctx, new, table, free, page, tokens):
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32).cuda()   # noqa: E731
    t = i32(table).reshape(table.shape)
    got = nv.page_maps(i32(ctx), i32(new), t, i32(free), page, tokens)
    return {**{k: v.cpu().numpy() for k, v in got.items()}, "table": t.cpu().numpy()}


def compare(got, want):
    for k in want:
        assert np.array_equal(got[k], want[k]), k


def a_table(rng, ctx, page, width, base=0):
    table = np.full((len(ctx), width), -1, np.int32)
    at = base
    for i, c in enumerate(ctx):
        e = min(-(-max(c, 0) // page), width)
        table[i, :e] = np.arange(at, at + e)
        at += e
    return table, at


# cached lengths, new lengths, page, entries of the maps past (or short of) the tokens
MAPS = [
    ([0], [1], 16, 0), ([0], [0], 16, 3), ([15, 16, 17], [1, 1, 1], 16, 0), ([0, 5, 0, 40], [33, 0, 16, 7], 16, 5),
    ([100, -3, 7], [-2, 9, 20], 24, 0), ([3, 9, 2], [50, 60, 70], 1, 0), ([0, 0], [2048, 1], 64, 0),
    ([10], [5000], 8, 11), ([1] * 300, [1] * 300, 16, 0), ([0, 7], [5000, 3000], 16, -2500),
]


@pytest.mark.parametrize("ctx,new,page,more", MAPS)
def test_maps(nv, ctx, new, page, more):
    rng = np.random.default_rng(len(ctx))
    total = sum(max(m, 0) for m in new)
    width = max(1, max(-(-(max(c, 0) + max(m, 0)) // page) for c, m in zip(ctx, new)))
    table, at = a_table(rng, ctx, page, width)
    free = (at + rng.permutation(total // page + len(ctx) + 5)).astype(np.int32)
    compare(run_maps(nv, ctx, new, table, free, page, total + more),
            maps_ref(ctx, new, table, free, page, total + more))


@pytest.mark.parametrize("seqs", [1, 255, 256, 257, 1000, 5000])
def test_maps_many_requests(nv, seqs):
    rng = np.random.default_rng(seqs)
    ctx = rng.integers(0, 200, seqs)
    new = np.where(rng.random(seqs) < 0.3, 0, rng.integers(1, 40, seqs))
    width = 20
    table, at = a_table(rng, ctx, 16, width)
    free = (at + rng.permutation(4 * seqs + 8)).astype(np.int32)
    tokens = int(new.sum())
    compare(run_maps(nv, ctx, new, table, free, 16, tokens), maps_ref(ctx, new, table, free, 16, tokens))


def test_maps_when_pages_or_columns_run_out(nv):
    rng = np.random.default_rng(3)
    ctx, new = [10, 0, 33, 64], [60, 40, 90, 3]
    table, at = a_table(rng, ctx, 16, 5)
    table[2, 1] = -1   # a cached page that is not there: its tokens have no slot
    for count in (0, 1, 5, 40):
        free = (at + rng.permutation(count)).astype(np.int32)
        compare(run_maps(nv, ctx, new, table, free, 16, 193), maps_ref(ctx, new, table, free, 16, 193))
    got = run_maps(nv, ctx, new, table, free[:3], 16, 193)
    assert got["taken"][0] > 3


def test_maps_of_no_requests(nv):
    got = run_maps(nv, [], [], np.zeros((0, 4), np.int32), [1, 2], 16, 5)
    assert got["cu_new"].tolist() == [0] and got["taken"].tolist() == [0]
    assert np.all(got["slot_map"] == -1) and np.all(got["positions"] == -1)


# tokens, heads, dim, page
WRITES = [(1, 1, 8, 16), (3, 2, 64, 16), (256, 8, 128, 16), (100, 3, 80, 24), (17, 5, 7, 4), (33, 4, 96, 1),
          (2, 1, 1, 3), (700, 8, 128, 64)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,heads,dim,page", WRITES)
def test_write(nv, tokens, heads, dim, page, dtype):
    gen = torch.Generator().manual_seed(tokens)
    pages = tokens // page + 3
    k, v = (torch.randn((tokens, heads, dim), generator=gen).to(dtype) for _ in range(2))
    kc, vc = (torch.randn((pages, heads, page, dim), generator=gen).to(dtype) for _ in range(2))
    slots = torch.randperm(pages * page, generator=gen)[:tokens]
    if tokens > 2:
        slots[1], slots[2] = -1, pages * page   # skipped
    want_k, want_v = kc.clone(), vc.clone()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            want_k[s // page, :, s % page], want_v[s // page, :, s % page] = k[t], v[t]
    bits = lambda t: t.cpu().view(torch.int16)   # noqa: E731
    for form in range(3):
        a, b = k.cuda(), v.cuda()
        if form == 1:    # slices of one projection
            a, b = torch.cat([a, b], 1)[:, :heads], torch.cat([a, b], 1)[:, heads:]
        elif form == 2:  # rows at odd addresses
            wide = torch.zeros((tokens, heads, dim + 3), dtype=dtype, device="cuda")
            wide[:, :, 1:dim + 1] = a
            a = wide[:, :, 1:dim + 1]
        dk, dv = kc.cuda(), vc.cuda()
        nv.kv_write(a, b, slots.cuda(), dk, dv)
        assert torch.equal(bits(dk), bits(want_k)) and torch.equal(bits(dv), bits(want_v)), form


def test_write_keeps_every_bit_pattern(nv):
    k = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(512, 1, 128).cuda()
    kc = torch.zeros((32, 1, 16, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    nv.kv_write(k, k, torch.arange(512).cuda(), kc, vc)
    assert torch.equal(kc.view(torch.int16).view(-1), k.view(torch.int16).reshape(-1))
    assert torch.equal(vc.view(torch.int16).view(-1), k.view(torch.int16).reshape(-1))
