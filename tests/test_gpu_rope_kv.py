"""Rotation of q and k with the append to the paged cache, against binary64.

A rotated element may differ from its binary64 value by half a step of the type (eps / 2 of the value, 2^-25
for fp16's smallest), and by what binary32 adds: sine and cosine off by at most 2^-21 (the rest of the
angle is rounded to 2^-25 turns, 2^-22.4 radians; the functions to 2 units), two products and a sum."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return nv


def turned(x, positions, freq, interleaved, mscale):
    """(binary64 values, what binary32 may add) of x [tokens, heads, dim]."""
    x = x.double().numpy()
    r = 2 * len(freq)
    angle = positions.double().numpy()[:, None, None] * freq.double().numpy()
    c, s = np.cos(angle) * mscale, np.sin(angle) * mscale
    ia, ib = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y, room = x.copy(), np.zeros_like(x)
    y[..., ia], y[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ia] * s + x[..., ib] * c
    room[..., ia] = room[..., ib] = (np.abs(x[..., ia]) + np.abs(x[..., ib])) * abs(mscale) * 2.0 ** -20
    return y, room


def near(got, want, room, dtype):
    step = torch.finfo(dtype).eps / 2
    off = np.abs(got.double().numpy() - want)
    assert (off <= step * np.abs(want) * (1 + 2.0 ** -10) + room + (2.0 ** -25 if dtype is torch.float16 else 0)).all()


def run(nv, kind, tokens, hq, hk, d, r, interleaved, page, longest, seed=0, mscale=1.0, fused=True, k_out=True,
        in_place=False, pad=1, gen_slots=None):
    dtype = TYPES[kind]
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn((tokens, hq + 2 * hk, d + pad), generator=g).to(dtype)
    host = wide[..., :d]
    qkv = wide.cuda()[..., :d]
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pages = tokens // page + 3
    positions = torch.randint(0, longest, (tokens,), generator=g).to(torch.int32)
    slots = torch.randperm(pages * page, generator=g)[:tokens].clone()
    if tokens > 4:
        positions[1], slots[1] = -1, -1           # padding
        slots[2] = -1                             # no slot: rotated all the same
        slots[3] = pages * page                   # outside the cache
        positions[4] = -7                         # a slot, but nothing is written
        positions[0] = 0
    freq = (10000.0 ** (-torch.arange(r // 2, dtype=torch.float64) / max(1, r // 2))).float()
    caches = [torch.randn((pages, hk, page, d), generator=g).to(dtype) for _ in range(2)]
    kc, vc = (c.cuda() for c in caches)
    if in_place:
        qo, ko = q, k
        old_q, old_k = host[:, :hq], host[:, hq:hq + hk]
    else:
        old_q, old_k = (torch.randn((tokens, h, d), generator=g).to(dtype) for h in (hq, hk))
        qo, ko = old_q.cuda(), old_k.cuda() if k_out else None
    got = nv.rope_kv_write(q, k, v, positions.cuda(), freq.cuda(), slots.cuda(), kc, vc, interleaved=interleaved,
                           mscale=mscale, q_out=qo, k_out=ko)
    assert got is qo
    torch.cuda.synchronize()
    there = (positions >= 0).numpy()
    for out, x, old in ((qo, host[:, :hq], old_q), (ko, host[:, hq:hq + hk], old_k)):
        if out is None:
            continue
        out = out.cpu()
        want, room = turned(x, positions, freq, interleaved, mscale)
        near(out[there], want[there], room[there], dtype)
        assert torch.equal(out[~there], old[~there])
        assert torch.equal(out[there][..., r:], x[there][..., r:])
    want_k, room_k = turned(host[:, hq:hq + hk], positions, freq, interleaved, mscale)
    kc, vc = kc.cpu(), vc.cpu()
    written = torch.zeros((pages, page), dtype=torch.bool)
    for t in range(tokens):
        s = int(slots[t])
        if there[t] and 0 <= s < pages * page:
            written[s // page, s % page] = True
            near(kc[s // page, :, s % page], want_k[t], room_k[t], dtype)
            assert torch.equal(vc[s // page, :, s % page], host[t, hq + hk:])
            if ko is not None:
                assert torch.equal(kc[s // page, :, s % page], ko[t].cpu())
    for c, old in zip((kc, vc), caches):
        assert torch.equal(c.transpose(1, 2)[~written], old.transpose(1, 2)[~written])


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", [(1, 32, 8, 128, 128), (7, 28, 4, 128, 64), (40, 8, 1, 96, 96), (130, 4, 2, 80, 80),
                                   (33, 2, 2, 80, 48), (9, 3, 1, 10, 6), (5, 1, 1, 2, 2), (12, 2, 1, 264, 256),
                                   (6, 2, 3, 520, 512)])
def test_against_binary64(nv, kind, interleaved, shape):
    tokens, hq, hk, d, r = shape
    pad = 0 if d % 8 == 0 else 1
    run(nv, kind, tokens, hq, hk, d, r, interleaved, 16, 5000, seed=sum(shape), pad=pad)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_not_aligned(nv, interleaved):
    run(nv, "bf16", 21, 4, 2, 64, 64, interleaved, 8, 300, pad=1)            # odd strides
    run(nv, "fp16", 21, 4, 2, 64, 24, interleaved, 8, 300, pad=0)            # runs of 12 elements
    run(nv, "fp16", 21, 4, 2, 68, 32, interleaved, 5, 300, pad=0)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_far_positions(nv, kind):
    run(nv, kind, 64, 2, 1, 64, 64, False, 16, 2 ** 31 - 1, seed=5, pad=0)


def test_in_place_and_without_outputs(nv):
    run(nv, "bf16", 50, 8, 2, 128, 128, False, 16, 9000, in_place=True, pad=0)
    run(nv, "fp16", 50, 8, 2, 64, 32, True, 16, 9000, in_place=True, pad=0)
    run(nv, "bf16", 50, 8, 2, 128, 128, False, 16, 9000, k_out=False, fused=False, pad=0)


def test_many_tokens_and_scale(nv):
    run(nv, "bf16", 5003, 3, 1, 64, 64, False, 24, 70000, mscale=1.25, pad=0)
    run(nv, "fp16", 8200, 2, 1, 16, 16, True, 7, 70000, mscale=-0.5, pad=0)


def test_keys_alone_and_no_tokens(nv):
    k = torch.randn((3, 2, 64)).half()
    v, kc, vc = torch.randn((3, 2, 64)).half(), torch.zeros((2, 2, 4, 64)).half(), torch.zeros((2, 2, 4, 64)).half()
    pos, freq, slots = torch.tensor([5, 6, 7], dtype=torch.int32), torch.ones(32), torch.tensor([0, 3, 6])
    kg, vg = kc.cuda(), vc.cuda()
    assert nv.rope_kv_write(None, k.cuda(), v.cuda(), pos.cuda(), freq.cuda(), slots.cuda(), kg, vg) is None
    want, room = turned(k, pos, freq, False, 1.0)
    for t, s in enumerate(slots.tolist()):
        near(kg.cpu()[s // 4, :, s % 4], want[t], room[t], torch.float16)
        assert torch.equal(vg.cpu()[s // 4, :, s % 4], v[t])
    before = kg.clone()
    q = torch.zeros((0, 4, 64), dtype=torch.float16, device="cuda")
    e = lambda n: torch.zeros((0, n, 64), dtype=torch.float16, device="cuda")   # noqa: E731
    out = nv.rope_kv_write(q, e(2), e(2), pos.cuda()[:0], freq.cuda(), slots.cuda()[:0], kg, vg)
    assert out.shape == (0, 4, 64) and torch.equal(kg, before)
    nothing = torch.zeros((0, 2, 4, 64), dtype=torch.float16, device="cuda")   # a cache without pages: q is rotated
    out = nv.rope_kv_write(k.cuda(), k.cuda(), v.cuda(), pos.cuda(), freq.cuda(), slots.cuda(), nothing, nothing)
    near(out.cpu(), want, room, torch.float16)


def test_values_that_are_not_finite(nv):
    """A pair with a NaN or an infinity spoils itself only."""
    k = torch.ones((2, 1, 16)).half()
    k[0, 0, 3], k[1, 0, 12] = float("nan"), float("inf")
    pos, freq = torch.tensor([1, 2], dtype=torch.int32), torch.full((4,), 0.3)
    z = torch.zeros((1, 1, 2, 16), dtype=torch.float16, device="cuda")
    out = nv.rope_kv_write(k.cuda(), k.cuda(), k.cuda(), pos.cuda(), freq.cuda(), torch.tensor([0, 1]).cuda(), z.clone(),
                           z.clone()).cpu()
    bad = ~torch.isfinite(out)
    assert bad.nonzero().tolist() == [[0, 0, 3], [0, 0, 7], [1, 0, 12]] and out[1, 0, 12] == float("inf")


def test_page_above_two_gib(nv):
    """Offsets in a long cache pass 32 bits: the last slots of 2^21 + 64 pages of 2 KiB."""
    pages = (1 << 21) + 64
    kc = torch.zeros((pages, 1, 8, 128), dtype=torch.float16, device="cuda")
    vc = torch.zeros((1, 1, 8, 128), dtype=torch.float16, device="cuda").expand(1, 1, 8, 128)
    vc = torch.zeros_like(kc)
    k, v = torch.randn((3, 1, 128)).half(), torch.randn((3, 1, 128)).half()
    pos, slots = torch.tensor([3, 4, 5], dtype=torch.int32), torch.tensor([pages * 8 - 1, pages * 8 - 77, 1])
    nv.rope_kv_write(None, k.cuda(), v.cuda(), pos.cuda(), torch.ones(64).cuda(), slots.cuda(), kc, vc)
    want, room = turned(k, pos, torch.ones(64), False, 1.0)
    for t, s in enumerate(slots.tolist()):
        near(kc[s // 8, :, s % 8].cpu(), want[t], room[t], torch.float16)
        assert torch.equal(vc[s // 8, :, s % 8].cpu(), v[t])
    assert int((kc != 0).any(-1).sum()) == 3 and int((vc != 0).any(-1).sum()) == 3


def test_streams_and_replays(nv):
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn((16, 12, 64), generator=g, device="cuda").half()
    pos, slots = torch.arange(16, dtype=torch.int32, device="cuda"), torch.arange(16, device="cuda")
    freq = torch.rand(32, generator=g, device="cuda")
    kc, vc = (torch.zeros((2, 2, 16, 64), dtype=torch.float16, device="cuda") for _ in range(2))
    qo = torch.zeros((16, 8, 64), dtype=torch.float16, device="cuda")

    def call(stream=None):
        return nv.rope_kv_write(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], pos, freq, slots, kc, vc, q_out=qo, stream=stream)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for turn in range(4):
        qkv.normal_(generator=g)
        pos.add_(1000 * turn)
        call()
        want = [t.clone() for t in (qo, kc, vc)]
        for t in (qo, kc, vc):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((qo, kc, vc), want)), turn


def test_broadcast_inputs_and_transposed_outputs(nv):
    """Heads that share one row (stride 0) as inputs; outputs [heads, tokens, dim]; in place of a shared row it is refused."""
    g = torch.Generator().manual_seed(8)
    row = torch.randn((9, 1, 64), generator=g).half()
    q, k = row.cuda().expand(9, 6, 64), row.cuda().expand(9, 2, 64)
    positions, freq = torch.arange(9, dtype=torch.int32), 1000.0 ** -(torch.arange(32) / 32)
    caches = [torch.zeros((2, 2, 8, 64), dtype=torch.float16, device="cuda") for _ in range(2)]
    args = (positions.cuda(), freq.cuda(), torch.arange(9, device="cuda"), *caches)
    out = torch.zeros((6, 9, 64), dtype=torch.float16, device="cuda").transpose(0, 1)
    nv.rope_kv_write(q, k, k, *args, q_out=out)
    want, room = turned(row, positions, freq, False, 1.0)
    for h in range(6):
        near(out[:, h:h + 1].cpu(), want, room, torch.float16)
    near(caches[0].transpose(1, 2).reshape(16, 2, 64)[:9].cpu(), np.repeat(want, 2, 1), np.repeat(room, 2, 1), torch.float16)
    assert torch.equal(caches[1].transpose(1, 2).reshape(16, 2, 64)[:9], k)
    for kw in (dict(q_out=q), dict(q_out=out, k_out=k)):
        with pytest.raises(nv.Nvfp4Error):
            nv.rope_kv_write(q, k, k, *args, **kw)
