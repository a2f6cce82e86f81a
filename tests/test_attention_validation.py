"""The serving attention operators refuse what they cannot run, before any launch: the C entry
points by status, the binding by exception.  No GPU: every call here fails a check (or has nothing
to do) before a device is asked for."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p(4096)          # never dereferenced
ODD = ctypes.c_void_p(4096 + 2)
EIGHT = ctypes.c_void_p(4096 + 8)
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    return nv


def refuses(fn, good, status, **changes):
    args = dict(good, **changes)
    assert fn(*args.values()) == status, changes


MAPS = dict(ctx=P, new=P, seqs=2, table=P, width=4, free=P, num_free=3, page=16, tokens=8, cu=P, lens=P, slots=P,
            positions=P, taken=P, stream=None)
WRITE = dict(k=P, v=P, tokens=4, heads=2, dim=64, ks=128, kh=64, vs=128, vh=64, slots=P, kc=P, vc=P, page=16,
             pages=4, stream=None)
PROMPT = dict(q=P, k=P, v=P, dtype=0, cu=P, seqs=1, tokens=4, hq=4, hk=2, dim=64, qs=256, qh=64, ks=128, kh=64,
              vs=128, vh=64, scale=0.125, window=0, out=P, lse=P, stream=None)
PAGED = dict(q=P, dtype=0, kc=P, vc=P, table=P, cu=P, lens=P, seqs=2, tokens=4, hq=4, hk=2, dim=64, page=16,
             pages=8, width=4, qs=256, qh=64, scale=0.125, window=0, out=P, lse=P, ws=P, ws_bytes=1 << 40, stream=None)


def test_page_maps_status(nv):
    fn = nv.lib().nvfp4_page_maps
    for c in [dict(seqs=-1), dict(width=-1), dict(num_free=-1), dict(page=0), dict(tokens=-1), dict(cu=None),
              dict(taken=None), dict(ctx=None), dict(new=None), dict(lens=None), dict(table=None), dict(free=None),
              dict(slots=None), dict(positions=None), dict(ctx=ODD), dict(table=ODD), dict(cu=ODD),
              dict(slots=ctypes.c_void_p(4096 + 4)), dict(positions=ODD), dict(taken=ODD)]:
        refuses(fn, MAPS, nv.NVFP4_EINVAL, **c)
    refuses(fn, MAPS, nv.NVFP4_EUNSUPPORTED, seqs=(1 << 20) + 1)
    refuses(fn, MAPS, nv.NVFP4_EUNSUPPORTED, tokens=(1 << 31) - 1)


def test_kv_write_status(nv):
    fn = nv.lib().nvfp4_kv_write
    for c in [dict(tokens=-1), dict(heads=0), dict(dim=0), dict(page=0), dict(pages=-1), dict(ks=-8), dict(vh=-64),
              dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None),
              dict(k=ctypes.c_void_p(4097)), dict(vc=ctypes.c_void_p(4097)), dict(slots=ctypes.c_void_p(4100))]:
        refuses(fn, WRITE, nv.NVFP4_EINVAL, **c)
    for c in [dict(heads=65537), dict(dim=65537), dict(tokens=1 << 50), dict(pages=1 << 47), dict(tokens=1 << 62),
              dict(pages=1 << 62)]:
        refuses(fn, WRITE, nv.NVFP4_EUNSUPPORTED, **c)
    refuses(fn, WRITE, nv.NVFP4_OK, tokens=0, k=None)
    refuses(fn, WRITE, nv.NVFP4_OK, pages=0, kc=None, vc=None)


ATTENTION = [dict(dtype=2), dict(dtype=-1), dict(seqs=-1), dict(tokens=-1), dict(hq=0), dict(hk=0), dict(hq=3),
             dict(dim=0), dict(dim=4), dict(dim=60), dict(dim=136), dict(window=-1), dict(scale=0.0),
             dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e-38),
             dict(scale=1e38), dict(qs=-8), dict(qh=-8), dict(qs=260), dict(qh=4), dict(q=None), dict(out=None),
             dict(q=EIGHT), dict(out=EIGHT), dict(lse=ODD), dict(cu=None), dict(cu=ODD)]


def test_prompt_attn_status(nv):
    fn = nv.lib().nvfp4_prompt_attn
    for c in ATTENTION + [dict(k=None), dict(v=None), dict(k=EIGHT), dict(v=EIGHT), dict(ks=-8), dict(kh=4),
                          dict(vs=130), dict(vh=-64)]:
        refuses(fn, PROMPT, nv.NVFP4_EINVAL, **c)
    refuses(fn, PROMPT, nv.NVFP4_EUNSUPPORTED, seqs=(1 << 20) + 1)
    refuses(fn, PROMPT, nv.NVFP4_EUNSUPPORTED, tokens=1 << 30)             # two rows a token
    refuses(fn, PROMPT, nv.NVFP4_EUNSUPPORTED, tokens=1 << 62)
    refuses(fn, PROMPT, nv.NVFP4_EUNSUPPORTED, tokens=1 << 29, hq=65536, hk=65536)   # above 2^31 workgroups
    refuses(fn, PROMPT, nv.NVFP4_OK, tokens=0, q=None, k=None, v=None, out=None, cu=None)


def test_paged_attn_status(nv):
    fn = nv.lib().nvfp4_paged_attn
    for c in ATTENTION + [dict(page=0), dict(pages=-1), dict(width=-1), dict(lens=None), dict(lens=ODD),
                          dict(table=None), dict(table=ODD), dict(kc=None), dict(vc=None), dict(kc=EIGHT),
                          dict(vc=EIGHT)]:
        refuses(fn, PAGED, nv.NVFP4_EINVAL, **c)
    for c in [dict(seqs=(1 << 20) + 1), dict(tokens=1 << 30), dict(width=1 << 27), dict(pages=(1 << 31) + 1)]:
        refuses(fn, PAGED, nv.NVFP4_EUNSUPPORTED, **c)
    need = nv.paged_attn_workspace_size(2, 4, 4, 2, 64)
    assert need > 0
    for c in [dict(ws=None), dict(ws_bytes=need - 1), dict(ws=ctypes.c_void_p(4096 + 128))]:
        refuses(fn, PAGED, nv.NVFP4_EWORKSPACE, **c)
    refuses(fn, PAGED, nv.NVFP4_OK, tokens=0, q=None, out=None, cu=None, ws=None)


def test_paged_workspace_size(nv):
    size = nv.lib().nvfp4_paged_attn_workspace_size
    for args in [(-1, 4, 4, 2, 64), (2, 0, 4, 2, 64), (2, -4, 4, 2, 64), (2, 4, 0, 2, 64), (2, 4, 4, 0, 64),
                 (2, 4, 3, 2, 64), (2, 4, 4, 2, 4), (2, 4, 4, 2, 136)]:
        assert size(*args) == 0, args
    # a bound for every call: it does not grow with the tokens or the keys
    assert size(1, 1, 32, 8, 128) <= size(4, 100, 32, 8, 128) == size(4, 100000, 32, 8, 128) < 160 << 20


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def test_page_maps_operands(nv):
    ok = dict(ctx_lens=i32(2), new_lens=i32(2), block_table=i32(2, 4), free_pages=i32(3), page_size=16, tokens=8)
    out = dict(cu_new=i32(3), kv_lens=i32(2), slot_map=torch.zeros(8, dtype=torch.int64), positions=i32(8),
               taken=i32(1))
    for key, bad, exc in [("ctx_lens", i32(2, 1), ValueError), ("ctx_lens", torch.zeros(2), TypeError),
                          ("ctx_lens", None, ValueError), ("new_lens", i32(3), ValueError),
                          ("new_lens", i32(4)[::2], ValueError), ("block_table", i32(3, 4), ValueError),
                          ("block_table", i32(4), ValueError), ("block_table", i32(4, 2).t(), ValueError),
                          ("free_pages", i32(1, 3), ValueError),
                          ("free_pages", torch.zeros(3, dtype=torch.int64), TypeError), ("tokens", -1, ValueError)]:
        with pytest.raises(exc, match=key):
            nv.page_maps(**dict(ok, **{key: bad}))
    for key, bad, exc in [("cu_new", i32(2), ValueError), ("kv_lens", i32(3), ValueError),
                          ("slot_map", i32(8), TypeError), ("positions", i32(7), ValueError),
                          ("taken", None, TypeError)]:
        with pytest.raises(exc, match=key):
            nv.page_maps(**ok, out=dict(out, **{key: bad}))
    with pytest.raises(ValueError, match="GPU"):
        nv.page_maps(**ok, out=out)


def test_kv_write_operands(nv):
    kv = torch.zeros((4, 2, 64), dtype=BF16)
    cache = torch.zeros((3, 2, 16, 64), dtype=BF16)
    ok = dict(k=kv, v=kv, slot_map=torch.zeros(4, dtype=torch.int64), k_cache=cache, v_cache=cache)
    for key, bad, exc in [("k", kv[0], ValueError), ("k", kv.transpose(1, 2), ValueError),
                          ("v", kv[:3], ValueError), ("v", kv.half(), TypeError), ("k_cache", cache[0], ValueError),
                          ("k_cache", cache.half(), TypeError), ("v_cache", cache[:2], ValueError),
                          ("k_cache", torch.zeros((3, 16, 2, 64), dtype=BF16).transpose(1, 2), ValueError),
                          ("slot_map", i32(4), TypeError),
                          ("slot_map", torch.zeros(5, dtype=torch.int64), ValueError)]:
        with pytest.raises(exc, match=key):
            nv.kv_write(**dict(ok, **{key: bad}))
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        nv.kv_write(kv.float(), kv.float(), ok["slot_map"], cache.float(), cache.float())
    with pytest.raises(ValueError, match="heads"):
        nv.kv_write(kv, kv, ok["slot_map"], torch.zeros((3, 1, 16, 64), dtype=BF16), cache[:, :1].contiguous())
    with pytest.raises(ValueError, match="GPU"):
        nv.kv_write(**ok)


def test_prompt_attn_operands(nv):
    q, kv = torch.zeros((4, 4, 64), dtype=BF16), torch.zeros((4, 2, 64), dtype=BF16)
    ok = dict(q=q, k=kv, v=kv, cu_seqlens=i32(2))
    for key, bad, exc in [("q", q[0], ValueError), ("q", q.transpose(1, 2), ValueError), ("k", kv[:2], ValueError),
                          ("k", kv.half(), TypeError), ("v", kv[:, :1], ValueError),
                          ("cu_seqlens", i32(0), ValueError), ("cu_seqlens", i32(2, 2), ValueError),
                          ("cu_seqlens", torch.zeros(2), TypeError), ("cu_seqlens", None, ValueError)]:
        with pytest.raises(exc, match=key):
            nv.prompt_attn(**dict(ok, **{key: bad}))
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        nv.prompt_attn(q.float(), kv.float(), kv.float(), i32(2))
    for key, bad, exc in [("out", q.half(), TypeError), ("out", q[:3], ValueError),
                          ("lse", torch.zeros((4, 2)), ValueError), ("lse", torch.zeros((4, 4), dtype=BF16), TypeError)]:
        with pytest.raises(exc, match=key):
            nv.prompt_attn(**ok, **{key: bad})
    with pytest.raises(ValueError, match="GPU"):
        nv.prompt_attn(**ok)


def test_paged_attn_operands(nv):
    q, cache = torch.zeros((4, 4, 64), dtype=BF16), torch.zeros((3, 2, 16, 64), dtype=BF16)
    ok = dict(q=q, k_cache=cache, v_cache=cache, block_table=i32(2, 4), cu_new=i32(3), kv_lens=i32(2))
    for key, bad, exc in [("q", q[0], ValueError), ("k_cache", cache[0], ValueError),
                          ("k_cache", cache.half(), TypeError), ("v_cache", cache[:1], ValueError),
                          ("block_table", i32(8), ValueError), ("block_table", i32(4, 2).t(), ValueError),
                          ("block_table", torch.zeros((2, 4)), TypeError), ("cu_new", i32(2), ValueError),
                          ("kv_lens", i32(3), ValueError), ("kv_lens", torch.zeros(2, dtype=torch.int64), TypeError)]:
        with pytest.raises(exc, match=key):
            nv.paged_attn(**dict(ok, **{key: bad}))
    with pytest.raises(ValueError, match="head_dim"):
        nv.paged_attn(**dict(ok, q=torch.zeros((4, 4, 32), dtype=BF16)))
    for key, bad, exc in [("out", q[:, :2], ValueError), ("lse", torch.zeros((3, 4)), ValueError)]:
        with pytest.raises(exc, match=key):
            nv.paged_attn(**ok, **{key: bad})
    with pytest.raises(ValueError, match="GPU"):
        nv.paged_attn(**ok)


def test_division_by_multiplication():
    # the kernels' page and group numbers: floor(j / d) as a multiply-high, and the places where it
    # could be off by one are around the multiples of d
    for d in list(range(2, 300)) + [1000, 4095, 4096, 4097, 65537, (1 << 20) + 7, (1 << 30) - 1, 1 << 30, (1 << 31) - 1]:
        shift = (d - 1).bit_length() - 1
        magic = ((1 << (32 + shift)) + d - 1) // d
        assert magic < 1 << 32
        top = ((1 << 31) - 1) // d
        for n in {1, 2, 3, 7, top // 3, top // 2, top - 1, top}:
            for j in (n * d - 1, n * d, n * d + 1, n * d + d - 1):
                if 0 <= j < 1 << 31:
                    assert (j * magic) >> (32 + shift) == j // d, (j, d)
