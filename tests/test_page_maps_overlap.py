"""Every workgroup of the page maps reads all the lengths while others already write: what is written may
overlap nothing that is passed, but for the lengths updated in place.  Refusals need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

SIZES = dict(ctx=8, new=8, table=32, free=12, cu=12, lens=8, slots=64, positions=32, taken=4)   # bytes
WRITTEN = ("table", "cu", "lens", "slots", "positions", "taken")
ORDER = ("ctx", "new", "seqs", "table", "width", "free", "num_free", "page", "tokens", "cu", "lens", "slots", "positions",
         "taken", "stream")


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    return nv


def addresses():
    return {name: 4096 + 256 * i for i, name in enumerate(SIZES)}   # never dereferenced


# addresses that nothing may ever read: a call that is not refused must not find a device to launch on
@pytest.mark.skipif(torch.cuda.is_available(), reason="refusals only, without a GPU")
@pytest.mark.parametrize("one", WRITTEN)
@pytest.mark.parametrize("two", SIZES)
def test_overlaps_are_refused(nv, one, two):
    if one == two:
        return
    # the last bytes of one buffer are the first of the other, and the other way round
    for first, second in ((one, two), (two, one)):
        step = 8 if second == "slots" else 4
        at = addresses()
        at[second] = at[first] + (SIZES[first] - 1) // step * step
        args = dict({n: ctypes.c_void_p(a) for n, a in at.items()}, seqs=2, width=4, num_free=3, page=16, tokens=8,
                    stream=None)
        assert nv.lib().nvfp4_page_maps(*(args[n] for n in ORDER)) == nv.NVFP4_EINVAL, (first, second)


@pytest.mark.skipif(torch.cuda.is_available(), reason="refusals only, without a GPU")
def test_lengths_in_place_admit_nothing_else(nv):
    at = addresses()
    at["lens"] = at["ctx"]
    for other in ("cu", "taken", "positions", "table"):
        args = dict({n: ctypes.c_void_p(a) for n, a in dict(at, **{other: at["ctx"]}).items()}, seqs=2, width=4, num_free=3,
                    page=16, tokens=8, stream=None)
        assert nv.lib().nvfp4_page_maps(*(args[n] for n in ORDER)) == nv.NVFP4_EINVAL, other


def operands(device="cpu"):
    def i32(*s):
        return torch.zeros(s, dtype=torch.int32, device=device)
    ok = dict(ctx_lens=i32(2), new_lens=i32(2), block_table=i32(2, 4), free_pages=i32(3), page_size=16, tokens=8)
    out = dict(cu_new=i32(3), kv_lens=i32(2), slot_map=torch.zeros(8, dtype=torch.int64, device=device),
               positions=i32(8), taken=i32(1))
    return ok, out


def aliased(ok, out):
    """Calls whose buffers overlap."""
    base = torch.cat([ok["new_lens"], ok["ctx_lens"]])
    return [dict(ok, out=dict(out, kv_lens=ok["new_lens"])), dict(ok, out=dict(out, cu_new=out["positions"][:3])),
            dict(ok, out=dict(out, positions=ok["block_table"].view(-1))),
            dict(ok, ctx_lens=base[:2], out=dict(out, kv_lens=base[1:3])),
            dict(ok, free_pages=ok["block_table"].view(-1)[:3]), dict(ok, free_pages=ok["block_table"].view(-1)[:3], out=out)]


def test_overlaps_are_named(nv):
    ok, out = operands()
    for call in aliased(ok, out):
        with pytest.raises(ValueError, match="overlap"):
            nv.page_maps(**call)
    with pytest.raises(ValueError, match="GPU"):   # lengths in place are accepted
        nv.page_maps(**ok, out=dict(out, kv_lens=ok["ctx_lens"]))


@pytest.mark.gpu
def test_overlaps_are_named_on_a_gpu(nv):
    ok, out = operands("cuda")
    for call in aliased(ok, out):
        with pytest.raises(ValueError, match="overlap"):
            nv.page_maps(**call)


@pytest.mark.gpu
@pytest.mark.parametrize("seqs,longest", [(1, 1), (300, 1), (300, 9), (2000, 200), (7, 60000)])
def test_lengths_updated_in_place(nv, seqs, longest):
    # one workgroup (up to 1024 tokens) and up to several hundred
    rng = np.random.default_rng([51, seqs])
    ctx = torch.from_numpy(rng.integers(-2, 500, seqs).astype(np.int32))
    new = torch.from_numpy(rng.integers(0, longest + 1, seqs).astype(np.int32))
    tokens, page = int(new.sum()), 16
    width = int(-(-(ctx.clamp(min=0) + new).max() // page))
    table = torch.full((seqs, width), -1, dtype=torch.int32)
    for i in range(seqs):
        held = -(-max(int(ctx[i]), 0) // page)
        table[i, :held] = torch.arange(held) + 40 * i
    free = torch.arange(40 * seqs, 40 * seqs + tokens // page + seqs + 1, dtype=torch.int32)
    a, b = table.cuda(), table.cuda()
    want = nv.page_maps(ctx.cuda(), new.cuda(), a, free.cuda(), page, tokens)
    assert torch.equal(want["kv_lens"].cpu(), ctx.clamp(min=0) + new)
    lens = ctx.cuda()
    got = nv.page_maps(lens, new.cuda(), b, free.cuda(), page, tokens,
                       out={k: lens if k == "kv_lens" else torch.full_like(v, 77) for k, v in want.items()})
    assert torch.equal(a, b) and all(torch.equal(got[k], want[k]) for k in want)
