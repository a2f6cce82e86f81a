"""What the FP8 operators, the rotation with the append and the MoE layer of a decode step refuse, before any launch: the C entry points by
status, the binding by exception.  No GPU: every call here fails a check (or has nothing to do) before a
device is asked for."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p(4096)          # never dereferenced
ODD = ctypes.c_void_p(4096 + 1)
TWO = ctypes.c_void_p(4096 + 2)
FOUR = ctypes.c_void_p(4096 + 4)
EIGHT = ctypes.c_void_p(4096 + 8)
BF16, F16, F32, I32, FP8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def nv():
    import nvfp4_block_scaled_quantize_amd as nv
    return nv


def refuses(fn, good, status, **changes):
    args = dict(good, **changes)
    assert fn(*args.values()) == status, changes


ROPE = dict(q=P, k=P, v=P, dtype=0, tokens=4, hq=4, hk=2, dim=64, qs=256, qh=64, ks=128, kh=64, vs=128, vh=64, pos=P,
            freq=P, rotary=64, paired=0, mscale=1.0, slots=P, qo=P, qos=256, qoh=64, ko=P, kos=128, koh=64, kc=P, vc=P,
            page=16, pages=4, stream=None)
QUANT = dict(x=P, dtype=0, rows=4, k=256, act=0, block=1, codes=P, scale=P, stream=None)
GEMM = dict(a=P, sa=P, w=P, sw=P, y=P, dtype=0, B=4, N=64, K=256, stream=None)

MOE = dict(x=P, dtype=1, router=P, bias=P, w1=P, w1_sf=P, w1_g=P, w2=P, w2_sf=P, w2_g=P, tiled=0, out=P, ids=None, w=None,
           tokens=4, experts=16, top_k=4, hidden=256, inter=128, act=2, groups=4, kept=2, norm=1, scaling=1.0, ws=P,
           ws_bytes=1 << 40, stream=None)


def test_moe_decode_status(nv):
    fn = nv.lib().nvfp4_moe_decode
    for c in [dict(dtype=2), dict(act=0), dict(act=3), dict(tokens=-1), dict(experts=0), dict(experts=257), dict(top_k=0),
              dict(top_k=17), dict(top_k=9), dict(hidden=0), dict(hidden=96), dict(inter=0), dict(inter=96), dict(groups=0),
              dict(groups=3), dict(kept=0), dict(kept=5), dict(hidden=192, tiled=1), dict(inter=192, tiled=1), dict(x=None),
              dict(router=None), dict(bias=None), dict(w1=None), dict(w1_sf=None), dict(w1_g=None), dict(w2=None),
              dict(w2_sf=None), dict(w2_g=None), dict(out=None), dict(x=EIGHT), dict(router=EIGHT), dict(w1=EIGHT),
              dict(w2=EIGHT), dict(out=FOUR), dict(w1_sf=TWO), dict(w2_sf=TWO), dict(bias=TWO), dict(w1_g=TWO),
              dict(w2_g=TWO), dict(ids=TWO), dict(w=TWO)]:
        refuses(fn, MOE, nv.NVFP4_EINVAL, **c)
    for c in [dict(tokens=33), dict(hidden=65536 + 64), dict(inter=65536 + 64)]:
        refuses(fn, MOE, nv.NVFP4_EUNSUPPORTED, **c)
    need = nv.moe_decode_workspace_size(4, 16, 4, 256, 128)
    assert need > 0
    for c in [dict(ws=None), dict(ws_bytes=need - 1), dict(ws=ctypes.c_void_p(4096 + 128))]:
        refuses(fn, MOE, nv.NVFP4_EWORKSPACE, **c)
    refuses(fn, MOE, nv.NVFP4_OK, tokens=0, x=None, out=None, ws=None)
    size = nv.lib().nvfp4_moe_decode_workspace_size
    for args in [(0, 16, 4, 256, 128), (33, 16, 4, 256, 128), (-1, 16, 4, 256, 128), (4, 0, 4, 256, 128),
                 (4, 16, 17, 256, 128), (4, 16, 4, 100, 128), (4, 16, 4, 256, 0), (4, 16, 4, 1 << 20, 128)]:
        assert size(*args) == 0, args


def test_rope_kv_write_status(nv):
    fn = nv.lib().nvfp4_rope_kv_write
    for c in [dict(dtype=2), dict(dtype=-1), dict(tokens=-1), dict(hq=-1), dict(hk=0), dict(dim=0), dict(dim=1),
              dict(page=0), dict(pages=-1), dict(rotary=0), dict(rotary=63), dict(rotary=66), dict(rotary=-2),
              dict(mscale=float("nan")), dict(mscale=float("inf")), dict(mscale=1e38), dict(qs=-1), dict(qh=-1), dict(ks=-1),
              dict(kh=-1), dict(vs=-1), dict(vh=-1), dict(qos=-1), dict(qoh=-1), dict(kos=-1), dict(koh=-1), dict(q=None),
              dict(k=None), dict(v=None), dict(pos=None), dict(freq=None), dict(slots=None), dict(qo=None), dict(kc=None),
              dict(vc=None), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(qo=ODD), dict(ko=ODD), dict(kc=ODD), dict(vc=ODD),
              dict(pos=TWO), dict(freq=TWO), dict(slots=FOUR)]:
        refuses(fn, ROPE, nv.NVFP4_EINVAL, **c)
    for c in [dict(dim=514, rotary=514), dict(hq=65537), dict(hk=65537), dict(dim=1 << 22), dict(tokens=1 << 24),
              dict(tokens=1 << 62), dict(pages=1 << 47)]:
        refuses(fn, ROPE, nv.NVFP4_EUNSUPPORTED, **c)
    refuses(fn, ROPE, nv.NVFP4_OK, tokens=0, q=None, k=None, v=None, pos=None, freq=None, slots=None)


def test_fp8_quantize_status(nv):
    fn = nv.lib().nvfp4_fp8_quantize
    for c in [dict(dtype=2), dict(rows=-1), dict(k=0), dict(k=-16), dict(k=24), dict(act=3), dict(act=-1), dict(block=0),
              dict(block=64), dict(x=None), dict(codes=None), dict(scale=None), dict(x=ODD), dict(scale=TWO)]:
        refuses(fn, QUANT, nv.NVFP4_EINVAL, **c)
    for c in [dict(rows=1 << 30), dict(rows=1 << 62), dict(k=1 << 31), dict(rows=1 << 31, block=128), dict(k=1 << 40)]:
        refuses(fn, QUANT, nv.NVFP4_EUNSUPPORTED, **c)
    refuses(fn, QUANT, nv.NVFP4_OK, rows=0, x=None, codes=None, scale=None)


def test_fp8_gemm_status(nv):
    fn = nv.lib().nvfp4_fp8_gemm
    for c in [dict(dtype=2), dict(B=-1), dict(N=0), dict(K=0), dict(K=24), dict(a=None), dict(sa=None), dict(w=None),
              dict(sw=None), dict(y=None), dict(a=EIGHT), dict(w=EIGHT), dict(sa=TWO), dict(sw=TWO), dict(y=ODD)]:
        refuses(fn, GEMM, nv.NVFP4_EINVAL, **c)
    for c in [dict(K=1 << 24), dict(B=1 << 31), dict(N=1 << 31), dict(B=1 << 20, N=1 << 20), dict(B=1 << 62)]:
        refuses(fn, GEMM, nv.NVFP4_EUNSUPPORTED, **c)
    refuses(fn, GEMM, nv.NVFP4_OK, B=0, a=None, y=None)


def z(*s, dtype=F16):
    return torch.zeros(s, dtype=dtype)


def test_rope_kv_write_operands(nv):
    ok = dict(q=z(4, 6, 64), k=z(4, 2, 64), v=z(4, 2, 64), positions=z(4, dtype=I32), inv_freq=z(32, dtype=F32),
              slot_map=z(4, dtype=torch.int64), k_cache=z(3, 2, 16, 64), v_cache=z(3, 2, 16, 64))
    for key, bad, exc in [("q", z(3, 6, 64), ValueError), ("q", z(4, 6, 32), ValueError), ("q", z(4, 384), ValueError),
                          ("q", z(4, 6, 64, dtype=BF16), TypeError), ("q", z(4, 6, 128)[..., ::2], ValueError),
                          ("k", z(4, 2, 64, dtype=F32), TypeError), ("k", z(4, 2, 128)[..., ::2], ValueError),
                          ("v", z(4, 3, 64), ValueError), ("v", z(4, 2, 64, dtype=BF16), TypeError),
                          ("positions", z(3, dtype=I32), ValueError), ("positions", z(4, dtype=torch.int64), TypeError),
                          ("positions", z(8, dtype=I32)[::2], ValueError), ("inv_freq", z(32), TypeError),
                          ("inv_freq", z(4, 8, dtype=F32), ValueError), ("inv_freq", None, ValueError),
                          ("slot_map", z(4, dtype=I32), TypeError), ("slot_map", z(5, dtype=torch.int64), ValueError),
                          ("k_cache", z(3, 1, 16, 64), ValueError), ("k_cache", z(3, 2, 16, 64, dtype=BF16), TypeError),
                          ("v_cache", z(2, 2, 16, 64), ValueError), ("q_out", z(4, 5, 64), ValueError),
                          ("q_out", z(4, 6, 64, dtype=BF16), TypeError), ("k_out", z(4, 2, 128)[..., ::2], ValueError),
                          ("k_out", z(5, 2, 64), ValueError)]:
        with pytest.raises(exc) as e:
            nv.rope_kv_write(**dict(ok, **{key: bad}))
        assert "GPU" not in str(e.value), key
    base = z(4 * 6 * 64 * 2)
    q = base.as_strided((4, 6, 64), (768, 64, 1))
    with pytest.raises(ValueError, match="strides"):
        nv.rope_kv_write(**dict(ok, q=q, q_out=base.as_strided((4, 6, 64), (384, 64, 1))))
    with pytest.raises(ValueError, match="q_out"):
        nv.rope_kv_write(**dict(ok, q=None, q_out=z(4, 6, 64)))
    with pytest.raises(ValueError, match="GPU"):
        nv.rope_kv_write(**ok)


def test_fp8_quantize_operands(nv):
    out = dict(codes=torch.zeros((4, 256)).to(FP8), scale=z(4, 2, dtype=F32))
    for kw, exc, what in [(dict(x=z(4, 2, 128)), ValueError, "x"), (dict(x=None), ValueError, "x"),
                          (dict(x=z(4, 256, dtype=F32)), TypeError, "input"), (dict(x=z(256, 4).t()), ValueError, "x"),
                          (dict(x=z(4, 256), block_rows=64), ValueError, "block_rows"),
                          (dict(x=z(4, 257), act="swiglu"), ValueError, "swiglu|GPU"),
                          (dict(x=z(4, 256), out=dict(out, codes=z(4, 256, dtype=torch.uint8))), TypeError, "codes"),
                          (dict(x=z(4, 256), out=dict(out, codes=torch.zeros((4, 128)).to(FP8))), ValueError, "codes"),
                          (dict(x=z(4, 256), out=dict(out, scale=z(4, 3, dtype=F32))), ValueError, "scale"),
                          (dict(x=z(4, 256), out=dict(codes=out["codes"])), TypeError, "scale"),
                          (dict(x=z(200, 256), block_rows=128, out=dict(codes=torch.zeros((200, 256)).to(FP8),
                                                                        scale=z(200, 2, dtype=F32))), ValueError, "scale"),
                          (dict(x=z(4, 256), out=out), ValueError, "GPU"), (dict(x=z(4, 256)), ValueError, "GPU")]:
        with pytest.raises(exc, match=what):
            nv.fp8_quantize(**kw)
    with pytest.raises(KeyError):
        nv.fp8_quantize(z(4, 256), act="gelu")


def test_fp8_gemm_operands(nv):
    e = lambda *s: torch.zeros(s).to(FP8)   # noqa: E731
    ok = dict(a=e(4, 272), a_scale=z(4, 3, dtype=F32), w=e(130, 272), w_scale=z(2, 3, dtype=F32))
    for key, bad, exc in [("a", e(4, 272, 1), ValueError), ("a", z(4, 272), TypeError), ("a", None, ValueError),
                          ("a_scale", z(4, 2, dtype=F32), ValueError), ("a_scale", z(4, 3), TypeError),
                          ("w", e(130, 256), ValueError), ("w", e(272, 130).t(), ValueError),
                          ("w_scale", z(1, 3, dtype=F32), ValueError), ("w_scale", z(3, 2, dtype=F32).t(), ValueError),
                          ("out", z(4, 130, dtype=F32), TypeError), ("out", z(4, 131), ValueError),
                          ("out", z(130, 4).t(), ValueError)]:
        with pytest.raises(exc):
            nv.fp8_gemm(**dict(ok, **{key: bad}))
    with pytest.raises(ValueError, match="GPU"):
        nv.fp8_gemm(**ok)


def test_moe_decode_operands(nv):
    u8 = torch.uint8
    ok = dict(x=z(4, 256), router=z(16, 256), bias=z(16, dtype=F32), w1=z(16, 128, 128, dtype=u8),
              w1_sf=z(16, 128, 16, dtype=u8), w1_g=z(16, dtype=F32), w2=z(16, 256, 64, dtype=u8),
              w2_sf=z(16, 256, 8, dtype=u8), w2_g=z(16, dtype=F32), top_k=4)
    for key, bad, exc in [("x", z(4, 256, 1), ValueError), ("x", z(4, 256, dtype=F32), TypeError), ("x", z(256, 4).t(), ValueError),
                          ("x", z(4, 128), ValueError), ("router", z(16, 256, dtype=BF16), TypeError),
                          ("router", z(15, 256), ValueError), ("bias", z(16), TypeError), ("bias", z(15, dtype=F32), ValueError),
                          ("w1", z(16, 256, 128, dtype=u8), ValueError), ("w1", z(16, 128, 128, dtype=torch.int8), TypeError),
                          ("w1_sf", z(16, 128, 8, dtype=u8), ValueError), ("w1_g", z(1, dtype=F32), ValueError),
                          ("w2", z(16, 256, dtype=u8), ValueError), ("w2", z(16, 64, 256, dtype=u8).transpose(1, 2), ValueError),
                          ("w2_sf", z(16, 128, 8, dtype=u8), ValueError), ("w2_g", z(16), TypeError),
                          ("out", z(4, 256, dtype=BF16), TypeError), ("out", z(4, 512)[:, ::2], ValueError),
                          ("act", "swiglu", ValueError)]:
        with pytest.raises(exc) as e:
            nv.moe_decode(**dict(ok, **{key: bad}))
        assert "GPU" not in str(e.value), key
    with pytest.raises(ValueError, match="GPU"):
        nv.moe_decode(**ok)


def test_rope_kv_write_rows_of_an_output_lie_apart(nv):
    fn = nv.lib().nvfp4_rope_kv_write
    for c in [dict(qoh=0), dict(qoh=63), dict(qos=0), dict(qos=255), dict(qoh=64, qos=64), dict(koh=0), dict(kos=127),
              dict(koh=65, kos=128), dict(qoh=1 << 62, qos=63), dict(qoh=255, qos=64), dict(tokens=1, qoh=63),
              dict(hq=1, qos=63)]:
        refuses(fn, ROPE, nv.NVFP4_EINVAL, **c)
    # apart: these get as far as the device (none here), or run
    q = torch.zeros((3, 1, 64), dtype=F16).expand(3, 4, 64)
    z = torch.zeros
    with pytest.raises((nv.Nvfp4Error, ValueError)):
        nv.rope_kv_write(q, z((3, 2, 64), dtype=F16), z((3, 2, 64), dtype=F16), z(3, dtype=I32), z(32), z(3, dtype=torch.int64),
                         z((2, 2, 16, 64), dtype=F16), z((2, 2, 16, 64), dtype=F16), q_out=q)
