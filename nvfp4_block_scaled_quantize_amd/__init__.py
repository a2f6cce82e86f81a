"""Python binding of libnvfp4_mi355x.so (the C ABI in include/nvfp4_mi355x.h).

Argument marshalling only: every step of the NVFP4 path runs in the HIP
kernels of the shared library.  torch supplies device memory and the current
HIP stream.  There is no CPU fallback: if the library is missing the import
fails, and every call checks the library's status code.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4_mi355x.so")

NVFP4_OK, NVFP4_EINVAL, NVFP4_EUNSUPPORTED, NVFP4_EWORKSPACE, NVFP4_EHIP, NVFP4_ESCRATCH = range(6)
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024   # NVFP4_NOALLOC_SCRATCH_BYTES
NVFP4_BF16, NVFP4_FP16 = 0, 1
ACT = {"none": 0, "swiglu": 1, "relu2": 2}
_TYPE_CODE = {torch.bfloat16: NVFP4_BF16, torch.float16: NVFP4_FP16}

EXPORTS = [
    "nvfp4_status_string", "nvfp4_quantize", "nvfp4_quantize_workspace_size", "nvfp4_act_quant",
    "nvfp4_gemm", "nvfp4_gemm_workspace_size", "nvfp4_moe_w4a16", "nvfp4_moe_w4a16_workspace_size",
    "nvfp4_register_weight", "nvfp4_unregister_weight", "nvfp4_gemm_external",
    "nvfp4_pretile_weight", "nvfp4_gemm_pretiled", "nvfp4_mx_quantize", "nvfp4_mx_tile",
    "nvfp4_mx_gemm", "nvfp4_moe_w4a16_noalloc", "nvfp4_moe_w4a16_pretiled",
    "nvfp4_page_maps", "nvfp4_kv_write", "nvfp4_prompt_attn", "nvfp4_paged_attn",
    "nvfp4_paged_attn_workspace_size", "nvfp4_rope_kv_write", "nvfp4_fp8_quantize", "nvfp4_fp8_gemm",
    "nvfp4_moe_decode", "nvfp4_moe_decode_workspace_size",
]
MX_ROWS, MX_TILED = 0, 1


class Nvfp4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (what, _lib.nvfp4_status_string(status).decode(), status))


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError("libnvfp4_mi355x.so is not built; run nvfp4_block_scaled_quantize_amd/build.py "
                          "(hipcc, gfx950) first -- there is no fallback implementation")
    L = ctypes.CDLL(LIB_PATH)
    p, i32, i64, sz, f32 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                            ctypes.c_float)
    L.nvfp4_status_string.argtypes = [i32]; L.nvfp4_status_string.restype = ctypes.c_char_p
    L.nvfp4_quantize.argtypes = [p, i32, i64, i64, i64, p, p, p, p, p, sz, p]
    L.nvfp4_quantize.restype = i32
    L.nvfp4_quantize_workspace_size.argtypes = [i64, i64, i64]
    L.nvfp4_quantize_workspace_size.restype = sz
    L.nvfp4_act_quant.argtypes = [p, i32, i64, i64, i32, p, p, p, p, p]
    L.nvfp4_act_quant.restype = i32
    L.nvfp4_gemm.argtypes = [p, p, p, p, p, p, i64, i64, i64, p, sz, p]
    L.nvfp4_gemm.restype = i32
    L.nvfp4_gemm_workspace_size.argtypes = [i64, i64, i64]
    L.nvfp4_gemm_workspace_size.restype = sz
    L.nvfp4_moe_w4a16.argtypes = [p, p, p, p, p, p, p, p, p, p, p, p,
                                  i32, i32, i32, i32, i32, i32, i32, i32, f32, p, sz, p]
    L.nvfp4_moe_w4a16.restype = i32
    L.nvfp4_moe_w4a16_pretiled.argtypes = [p, p, p, p, p, p, p, p, p, p, p, p,
                                           i32, i32, i32, i32, i32, i32, i32, i32, f32, p, sz, p]
    L.nvfp4_moe_w4a16_pretiled.restype = i32
    L.nvfp4_moe_w4a16_noalloc.argtypes = [p, p, p, p, p, p, p, p, p, p, p, p,
                                          i32, i32, i32, i32, i32, i32, i32, i32, f32, p]
    L.nvfp4_moe_w4a16_noalloc.restype = i32
    L.nvfp4_moe_w4a16_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    L.nvfp4_moe_w4a16_workspace_size.restype = sz
    L.nvfp4_register_weight.argtypes = [i32, i32, p, p, i32, i32, i32]
    L.nvfp4_register_weight.restype = i32
    L.nvfp4_unregister_weight.argtypes = [i32, i32]
    L.nvfp4_unregister_weight.restype = i32
    L.nvfp4_gemm_external.argtypes = [p, p, i32, p, p, i64, i64, i64, p, sz, p]
    L.nvfp4_gemm_external.restype = i32
    L.nvfp4_pretile_weight.argtypes = [p, p, i64, i64, p, p, p]
    L.nvfp4_pretile_weight.restype = i32
    L.nvfp4_gemm_pretiled.argtypes = [p, p, p, p, p, p, i64, i64, i64, p, sz, p]
    L.nvfp4_gemm_pretiled.restype = i32
    L.nvfp4_mx_quantize.argtypes = [p, i32, i64, i64, i32, i64, i32, p, p, p, p, sz, p]
    L.nvfp4_mx_quantize.restype = i32
    L.nvfp4_mx_tile.argtypes = [p, p, i64, i64, p, p, p]
    L.nvfp4_mx_tile.restype = i32
    L.nvfp4_mx_gemm.argtypes = [p, p, p, i64, p, p, p, p, i64, i64, i64, p]
    L.nvfp4_mx_gemm.restype = i32
    L.nvfp4_page_maps.argtypes = [p, p, i32, p, i32, p, i32, i32, i64, p, p, p, p, p, p]
    L.nvfp4_page_maps.restype = i32
    L.nvfp4_kv_write.argtypes = [p, p, i64, i32, i32, i64, i64, i64, i64, p, p, p, i32, i64, p]
    L.nvfp4_kv_write.restype = i32
    L.nvfp4_prompt_attn.argtypes = [p, p, p, i32, p, i32, i64, i32, i32, i32, i64, i64, i64, i64, i64, i64,
                                    f32, i32, p, p, p]
    L.nvfp4_prompt_attn.restype = i32
    L.nvfp4_paged_attn.argtypes = [p, i32, p, p, p, p, p, i32, i64, i32, i32, i32, i32, i64, i32, i64, i64,
                                   f32, i32, p, p, p, sz, p]
    L.nvfp4_paged_attn.restype = i32
    L.nvfp4_paged_attn_workspace_size.argtypes = [i32, i64, i32, i32, i32]
    L.nvfp4_paged_attn_workspace_size.restype = sz
    L.nvfp4_rope_kv_write.argtypes = [p, p, p, i32, i64, i32, i32, i32, i64, i64, i64, i64, i64, i64, p, p, i32, i32,
                                      f32, p, p, i64, i64, p, i64, i64, p, p, i32, i64, p]
    L.nvfp4_rope_kv_write.restype = i32
    L.nvfp4_fp8_quantize.argtypes = [p, i32, i64, i64, i32, i32, p, p, p]
    L.nvfp4_fp8_quantize.restype = i32
    L.nvfp4_fp8_gemm.argtypes = [p, p, p, p, p, i32, i64, i64, i64, p]
    L.nvfp4_fp8_gemm.restype = i32
    L.nvfp4_moe_decode.argtypes = [p, i32, p, p, p, p, p, p, p, p, i32, p, p, p, i32, i32, i32, i32, i32, i32, i32, i32,
                                   i32, f32, p, sz, p]
    L.nvfp4_moe_decode.restype = i32
    L.nvfp4_moe_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    L.nvfp4_moe_decode_workspace_size.restype = sz
    return L


_lib = _load()


def lib() -> ctypes.CDLL:
    return _lib


def _stream(stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    # the handle itself: building a Stream object takes longer than a small kernel
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check_dev(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous and on the GPU")


def _need(t, name: str, dtype, shape=None, min_numel=None):
    """Checks what the C ABI cannot: the dtype and the shape (or, for flat
    buffers, the element count) of an operand or a caller-supplied output.  A
    wrong one would be an out-of-bounds device access, so it is an error here."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError("%s must hold at least %d elements, got %d" % (name, min_numel, t.numel()))


def _need_2d(x, name: str):
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("%s must be a 2-D tensor" % name)


def _dtype_code(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return NVFP4_BF16
    if x.dtype == torch.float16:
        return NVFP4_FP16
    raise TypeError("input must be bfloat16 or float16")


def _need_32_bits(**numbers):
    """The C entry points take these as 32-bit integers, and ctypes would cut them without a word."""
    for name, v in numbers.items():
        if not -(1 << 31) <= v < 1 << 31:
            raise ValueError("%s must fit 32 bits, got %d" % (name, v))


def _act_code(act) -> int:
    a = ACT[act] if isinstance(act, str) else int(act)
    if a >> 31:
        _need_32_bits(act=a)
    return a


def _workspace(nbytes: int, device, workspace: torch.Tensor | None):
    if nbytes == 0:
        return None, 0
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor")
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small: need %d bytes" % nbytes)
        return workspace, workspace.numel() * workspace.element_size()
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def _quant_out(o: dict, rows: int, k: int, ngroups: int):
    """Checks a caller-supplied output dict of quantize() / act_quant()."""
    _need(o.get("codes"), "out['codes']", torch.uint8, (rows, k // 2))
    _need(o.get("sf"), "out['sf']", torch.uint8, (rows, k // 16))
    _need(o.get("g_dec"), "out['g_dec']", torch.float32, min_numel=ngroups)
    if o.get("scale") is not None:
        _need(o["scale"], "out['scale']", torch.float32, (rows, k // 16))


def quantize_workspace_size(rows: int, k: int, group_rows: int) -> int:
    """Bytes of caller workspace that quantize() / mx_quantize() need for one
    global per `group_rows` rows (0 for per-token globals)."""
    return int(_lib.nvfp4_quantize_workspace_size(rows, k, group_rows))


def quantize(x: torch.Tensor, group_rows: int = 1, want_scale: bool = True, out: dict | None = None,
             workspace: torch.Tensor | None = None, stream=None) -> dict:
    """NVFP4-quantize x [rows, k] with one global scale per `group_rows` rows."""
    _need_2d(x, "x")
    _dtype_code(x)
    rows, k = x.shape
    if out is not None:
        _quant_out(out, rows, k, rows // max(group_rows, 1))
    _check_dev(x)
    dev = x.device
    o = out or {
        "codes": torch.empty((rows, k // 2), dtype=torch.uint8, device=dev),
        "sf": torch.empty((rows, k // 16), dtype=torch.uint8, device=dev),
        "g_dec": torch.empty((rows // max(group_rows, 1),), dtype=torch.float32, device=dev),
        "scale": torch.empty((rows, k // 16), dtype=torch.float32, device=dev) if want_scale else None,
    }
    ws, wsb = _workspace(_lib.nvfp4_quantize_workspace_size(rows, k, group_rows), dev, workspace)
    st = _lib.nvfp4_quantize(_ptr(x), _dtype_code(x), rows, k, group_rows, _ptr(o["codes"]), _ptr(o["sf"]),
                             _ptr(o["g_dec"]), _ptr(o.get("scale")), _ptr(ws), wsb, _stream(stream))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_quantize")
    return o


def act_quant(x: torch.Tensor, act: str = "none", want_scale: bool = True, out: dict | None = None,
              stream=None) -> dict:
    """Fused activation (none / swiglu / relu2) + per-token NVFP4 quantization."""
    _need_2d(x, "x")
    _dtype_code(x)
    rows, k_in = x.shape
    a = _act_code(act)
    k_out = k_in // 2 if a == ACT["swiglu"] else k_in
    if out is not None:
        _quant_out(out, rows, k_out, rows)
    _check_dev(x)
    dev = x.device
    o = out or {
        "codes": torch.empty((rows, k_out // 2), dtype=torch.uint8, device=dev),
        "sf": torch.empty((rows, k_out // 16), dtype=torch.uint8, device=dev),
        "g_dec": torch.empty((rows,), dtype=torch.float32, device=dev),
        "scale": torch.empty((rows, k_out // 16), dtype=torch.float32, device=dev) if want_scale else None,
    }
    st = _lib.nvfp4_act_quant(_ptr(x), _dtype_code(x), rows, k_out, a, _ptr(o["codes"]), _ptr(o["sf"]),
                              _ptr(o["g_dec"]), _ptr(o.get("scale")), _stream(stream))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_act_quant")
    return o


def gemm_workspace_size(B: int, N: int, K: int) -> int:
    return int(_lib.nvfp4_gemm_workspace_size(B, N, K))


def gemm(a_codes: torch.Tensor, a_scale: torch.Tensor, w_codes: torch.Tensor, w_sf: torch.Tensor,
         w_g: torch.Tensor, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """y[B, N] fp16 = deq(a) . deq(w)^T."""
    _need_2d(a_codes, "a_codes")
    _need_2d(w_codes, "w_codes")
    B, K = a_codes.shape[0], a_codes.shape[1] * 2
    N = w_codes.shape[0]
    _need(a_codes, "a_codes", torch.uint8)
    _need(a_scale, "a_scale", torch.float32, (B, K // 16))
    _need(w_codes, "w_codes", torch.uint8, (N, K // 2))
    _need(w_sf, "w_sf", torch.uint8, (N, K // 16))
    _need(w_g, "w_g", torch.float32, min_numel=1)
    if out is not None:
        _need(out, "out", torch.float16, (B, N))
    _check_dev(a_codes, a_scale, w_codes, w_sf, w_g, out)
    y = out if out is not None else torch.empty((B, N), dtype=torch.float16, device=a_codes.device)
    ws, wsb = _workspace(gemm_workspace_size(B, N, K), a_codes.device, workspace)
    st = _lib.nvfp4_gemm(_ptr(a_codes), _ptr(a_scale), _ptr(w_codes), _ptr(w_sf), _ptr(w_g), _ptr(y),
                         B, N, K, _ptr(ws), wsb, _stream(stream))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_gemm")
    return y


def pretile_weight(w_codes: torch.Tensor, w_sf: torch.Tensor, stream=None) -> dict:
    """The pre-tiled layout of [N, K/2] codes and [N, K/16] E4M3 bytes (flat
    uint8 tensors of N*K/2 and N*K/16 bytes)."""
    _need_2d(w_codes, "w_codes")
    N, K = w_codes.shape[0], w_codes.shape[1] * 2
    _need(w_codes, "w_codes", torch.uint8)
    _need(w_sf, "w_sf", torch.uint8, (N, K // 16))
    _check_dev(w_codes, w_sf)
    wt = torch.empty(N * K // 2, dtype=torch.uint8, device=w_codes.device)
    st = torch.empty(N * K // 16, dtype=torch.uint8, device=w_codes.device)
    rc = _lib.nvfp4_pretile_weight(_ptr(w_codes), _ptr(w_sf), N, K, _ptr(wt), _ptr(st), _stream(stream))
    if rc != NVFP4_OK:
        raise Nvfp4Error(rc, "nvfp4_pretile_weight")
    return {"codes": wt, "sf": st, "N": N, "K": K}


def gemm_pretiled(a_codes: torch.Tensor, a_scale: torch.Tensor, wt: dict, w_g: torch.Tensor,
                  out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """gemm() with weights from pretile_weight()."""
    _need_2d(a_codes, "a_codes")
    B, K = a_codes.shape[0], a_codes.shape[1] * 2
    N = wt["N"]
    if K != wt["K"]:
        raise ValueError("activation K %d differs from the pre-tiled weight's K %d" % (K, wt["K"]))
    _need(a_codes, "a_codes", torch.uint8)
    _need(a_scale, "a_scale", torch.float32, (B, K // 16))
    _need(wt["codes"], "wt['codes']", torch.uint8, min_numel=N * K // 2)
    _need(wt["sf"], "wt['sf']", torch.uint8, min_numel=N * K // 16)
    _need(w_g, "w_g", torch.float32, min_numel=1)
    if out is not None:
        _need(out, "out", torch.float16, (B, N))
    _check_dev(a_codes, a_scale, w_g, wt["codes"], wt["sf"], out)
    y = out if out is not None else torch.empty((B, N), dtype=torch.float16, device=a_codes.device)
    ws, wsb = _workspace(gemm_workspace_size(B, N, K), a_codes.device, workspace)
    rc = _lib.nvfp4_gemm_pretiled(_ptr(a_codes), _ptr(a_scale), _ptr(wt["codes"]), _ptr(wt["sf"]), _ptr(w_g),
                                  _ptr(y), B, N, K, _ptr(ws), wsb, _stream(stream))
    if rc != NVFP4_OK:
        raise Nvfp4Error(rc, "nvfp4_gemm_pretiled")
    return y


def register_weight(resource_id: int, w_codes: torch.Tensor, w_sf: torch.Tensor) -> None:
    """Registers an external weight ([N, K/2] codes, [N, K/16] E4M3 bytes) for
    (the tensors' device, resource_id).  The tensors must outlive the
    registration: unregister before freeing them."""
    _need_2d(w_codes, "w_codes")
    N, K = w_codes.shape[0], w_codes.shape[1] * 2
    _need(w_codes, "w_codes", torch.uint8)
    _need(w_sf, "w_sf", torch.uint8, (N, K // 16))
    _check_dev(w_codes, w_sf)
    st = _lib.nvfp4_register_weight(w_codes.device.index or 0, resource_id, _ptr(w_codes), _ptr(w_sf),
                                    N, K, K // 16)
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_register_weight")


def unregister_weight(resource_id: int, device: int = 0) -> None:
    st = _lib.nvfp4_unregister_weight(device, resource_id)
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_unregister_weight")


def gemm_external(a_codes: torch.Tensor, a_scale: torch.Tensor, resource_id: int, N: int,
                  w_g: torch.Tensor, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gemm() with the weight registered under resource_id on the current device."""
    _need_2d(a_codes, "a_codes")
    B, K = a_codes.shape[0], a_codes.shape[1] * 2
    _need(a_codes, "a_codes", torch.uint8)
    _need(a_scale, "a_scale", torch.float32, (B, K // 16))
    _need(w_g, "w_g", torch.float32, min_numel=1)
    if out is not None:
        _need(out, "out", torch.float16, (B, N))
    _check_dev(a_codes, a_scale, w_g, out)
    y = out if out is not None else torch.empty((B, N), dtype=torch.float16, device=a_codes.device)
    ws, wsb = _workspace(gemm_workspace_size(B, N, K), a_codes.device, workspace)
    st = _lib.nvfp4_gemm_external(_ptr(a_codes), _ptr(a_scale), resource_id, _ptr(w_g), _ptr(y),
                                  B, N, K, _ptr(ws), wsb, _stream(stream))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_gemm_external")
    return y


def moe_workspace_size(tokens, experts, top_k, hidden, inter) -> int:
    return int(_lib.nvfp4_moe_w4a16_workspace_size(tokens, experts, top_k, hidden, inter))


def moe_w4a16(logits, bias, x, w1, w1_sf, w1_g, w2, w2_sf, w2_g, top_k, n_group, topk_group,
              norm_topk_prob=True, routed_scaling=1.0, out=None, want_routing=False,
              workspace=None, stream=None):
    """Routed W4A16 MoE layer; returns out (and (ids, weights) if want_routing)."""
    return _moe(_lib.nvfp4_moe_w4a16, "nvfp4_moe_w4a16", logits, bias, x, w1, w1_sf, w1_g, w2, w2_sf,
                w2_g, top_k, n_group, topk_group, norm_topk_prob, routed_scaling, out, want_routing,
                workspace, stream)


def moe_pretile_weights(w: torch.Tensor, w_sf: torch.Tensor, stream=None) -> tuple:
    """The pre-tiled layout of stacked expert weights [E, N, K/2] codes and
    [E, N, K/16] E4M3 bytes (nvfp4_pretile_weight of the [E*N, K] matrix),
    returned with the same shapes."""
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w must be a 3-D tensor [experts, rows, K/2]")
    E, N, K2 = w.shape
    _need(w, "w", torch.uint8)
    _need(w_sf, "w_sf", torch.uint8, (E, N, K2 // 8))
    t = pretile_weight(w.reshape(E * N, K2), w_sf.reshape(E * N, K2 // 8), stream=stream)
    return t["codes"].view(E, N, K2), t["sf"].view(E, N, K2 // 8)


def moe_w4a16_pretiled(logits, bias, x, w1, w1_sf, w1_g, w2, w2_sf, w2_g, top_k, n_group, topk_group,
                       norm_topk_prob=True, routed_scaling=1.0, out=None, want_routing=False,
                       workspace=None, stream=None):
    """moe_w4a16() with w1/w1_sf and w2/w2_sf from moe_pretile_weights()
    (same shapes and results)."""
    return _moe(_lib.nvfp4_moe_w4a16_pretiled, "nvfp4_moe_w4a16_pretiled", logits, bias, x, w1, w1_sf,
                w1_g, w2, w2_sf, w2_g, top_k, n_group, topk_group, norm_topk_prob, routed_scaling, out,
                want_routing, workspace, stream)


def _moe(fn, name, logits, bias, x, w1, w1_sf, w1_g, w2, w2_sf, w2_g, top_k, n_group, topk_group,
         norm_topk_prob, routed_scaling, out, want_routing, workspace, stream):
    _need_2d(logits, "logits")
    _need_2d(x, "x")
    T, E = logits.shape
    hidden = x.shape[1]
    if not isinstance(w1, torch.Tensor) or w1.dim() != 3:
        raise ValueError("w1 must be a 3-D tensor [experts, inter, hidden/2]")
    inter = w1.shape[1]
    _need(logits, "logits", torch.float32)
    _need(bias, "bias", torch.float32, (E,))
    _need(x, "x", torch.float16, (T, hidden))
    _need(w1, "w1", torch.uint8, (E, inter, hidden // 2))
    _need(w1_sf, "w1_sf", torch.uint8, (E, inter, hidden // 16))
    _need(w1_g, "w1_g", torch.float32, min_numel=E)
    _need(w2, "w2", torch.uint8, (E, hidden, inter // 2))
    _need(w2_sf, "w2_sf", torch.uint8, (E, hidden, inter // 16))
    _need(w2_g, "w2_g", torch.float32, min_numel=E)
    if out is not None:
        _need(out, "out", torch.float16, (T, hidden))
    _check_dev(logits, bias, x, w1, w1_sf, w1_g, w2, w2_sf, w2_g, out)
    o = out if out is not None else torch.empty((T, hidden), dtype=torch.float16, device=x.device)
    ids = torch.empty((T, top_k), dtype=torch.int32, device=x.device) if want_routing else None
    wts = torch.empty((T, top_k), dtype=torch.float32, device=x.device) if want_routing else None
    ws, wsb = _workspace(moe_workspace_size(T, E, top_k, hidden, inter), x.device, workspace)
    st = fn(_ptr(logits), _ptr(bias), _ptr(x), _ptr(w1), _ptr(w1_sf), _ptr(w1_g),
            _ptr(w2), _ptr(w2_sf), _ptr(w2_g), _ptr(o), _ptr(ids), _ptr(wts),
            T, E, top_k, hidden, inter, n_group, topk_group, int(bool(norm_topk_prob)),
            float(routed_scaling), _ptr(ws), wsb, _stream(stream))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, name)
    return (o, ids, wts) if want_routing else o


def moe_w4a16_noalloc(logits, bias, x, w1, w1_sf, w1_g, w2, w2_sf, w2_g, top_k, n_group, topk_group,
                      norm_topk_prob=True, routed_scaling=1.0, out=None, ids_out=None, w_out=None, stream=None):
    """moe_w4a16() on the library's fixed device scratch: no workspace, nothing
    allocated by the library (pass `out` to allocate nothing here either).
    Calls that overlap in time on one GPU race."""
    _need_2d(logits, "logits")
    _need_2d(x, "x")
    T, E = logits.shape
    hidden = x.shape[1]
    if not isinstance(w1, torch.Tensor) or w1.dim() != 3:
        raise ValueError("w1 must be a 3-D tensor [experts, inter, hidden/2]")
    inter = w1.shape[1]
    _need(logits, "logits", torch.float32)
    _need(bias, "bias", torch.float32, (E,))
    _need(x, "x", torch.float16, (T, hidden))
    _need(w1, "w1", torch.uint8, (E, inter, hidden // 2))
    _need(w1_sf, "w1_sf", torch.uint8, (E, inter, hidden // 16))
    _need(w1_g, "w1_g", torch.float32, min_numel=E)
    _need(w2, "w2", torch.uint8, (E, hidden, inter // 2))
    _need(w2_sf, "w2_sf", torch.uint8, (E, hidden, inter // 16))
    _need(w2_g, "w2_g", torch.float32, min_numel=E)
    for t, name, dt in ((out, "out", torch.float16), (ids_out, "ids_out", torch.int32), (w_out, "w_out", torch.float32)):
        if t is not None:
            _need(t, name, dt, (T, hidden) if name == "out" else (T, top_k))
    _check_dev(logits, bias, x, w1, w1_sf, w1_g, w2, w2_sf, w2_g, out, ids_out, w_out)
    o = out if out is not None else torch.empty((T, hidden), dtype=torch.float16, device=x.device)
    st = _lib.nvfp4_moe_w4a16_noalloc(_ptr(logits), _ptr(bias), _ptr(x), _ptr(w1), _ptr(w1_sf), _ptr(w1_g),
                                      _ptr(w2), _ptr(w2_sf), _ptr(w2_g), _ptr(o), _ptr(ids_out), _ptr(w_out),
                                      T, E, top_k, hidden, inter, n_group, topk_group, int(bool(norm_topk_prob)),
                                      float(routed_scaling), _stream(stream))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_moe_w4a16_noalloc")
    return o


# ---------------------------------------------------------------- MXFP4 variant

def mx_tiled_sizes(rows: int, k: int) -> tuple[int, int]:
    """Bytes of the MX tile layout of a [rows, k] operand: (codes, scale bytes)."""
    r32 = (rows + 31) // 32 * 32
    return r32 * k // 2, r32 * k // 32


def mx_quantize(x: torch.Tensor, act: str = "none", group_rows: int = 1, tiled: bool = False,
                out: dict | None = None, workspace: torch.Tensor | None = None, stream=None) -> dict:
    """MXFP4 quantization (E8M0 scale per 32 elements) of x [rows, k_in], with the
    optional activation in front.  Returns dict(codes, sf, g_dec, rows, K, tiled):
    [rows, k/2] and [rows, k/32] uint8 in the row layout, flat uint8 tensors in
    the MX tile layout."""
    _need_2d(x, "x")
    _dtype_code(x)
    rows, k_in = x.shape
    a = _act_code(act)
    k = k_in // 2 if a == ACT["swiglu"] else k_in
    if out is not None:
        if tiled:
            nc, ns = mx_tiled_sizes(rows, k)
            _need(out.get("codes"), "out['codes']", torch.uint8, min_numel=nc)
            _need(out.get("sf"), "out['sf']", torch.uint8, min_numel=ns)
        else:
            _need(out.get("codes"), "out['codes']", torch.uint8, (rows, k // 2))
            _need(out.get("sf"), "out['sf']", torch.uint8, (rows, k // 32))
        _need(out.get("g_dec"), "out['g_dec']", torch.float32, min_numel=rows // max(group_rows, 1))
    _check_dev(x)
    dev = x.device
    if out is None:
        if tiled:
            nc, ns = mx_tiled_sizes(rows, k)
            codes = torch.empty(nc, dtype=torch.uint8, device=dev)
            sf = torch.empty(ns, dtype=torch.uint8, device=dev)
        else:
            codes = torch.empty((rows, k // 2), dtype=torch.uint8, device=dev)
            sf = torch.empty((rows, k // 32), dtype=torch.uint8, device=dev)
        out = {"codes": codes, "sf": sf,
               "g_dec": torch.empty((rows // max(group_rows, 1),), dtype=torch.float32, device=dev)}
    out.update(rows=rows, K=k, tiled=bool(tiled))
    ws, wsb = _workspace(_lib.nvfp4_quantize_workspace_size(rows, k, group_rows), dev, workspace)
    st = _lib.nvfp4_mx_quantize(_ptr(x), _dtype_code(x), rows, k, a, group_rows,
                                MX_TILED if tiled else MX_ROWS, _ptr(out["codes"]), _ptr(out["sf"]),
                                _ptr(out["g_dec"]), _ptr(ws), wsb, _stream(stream))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_mx_quantize")
    return out


def mx_tile(codes: torch.Tensor, sf: torch.Tensor, stream=None) -> dict:
    """The MX tile layout of [rows, k/2] codes and [rows, k/32] E8M0 bytes."""
    _need_2d(codes, "codes")
    rows, k = codes.shape[0], codes.shape[1] * 2
    _need(codes, "codes", torch.uint8)
    _need(sf, "sf", torch.uint8, (rows, k // 32))
    _check_dev(codes, sf)
    nc, ns = mx_tiled_sizes(rows, k)
    ct = torch.empty(nc, dtype=torch.uint8, device=codes.device)
    stt = torch.empty(ns, dtype=torch.uint8, device=codes.device)
    rc = _lib.nvfp4_mx_tile(_ptr(codes), _ptr(sf), rows, k, _ptr(ct), _ptr(stt), _stream(stream))
    if rc != NVFP4_OK:
        raise Nvfp4Error(rc, "nvfp4_mx_tile")
    return {"codes": ct, "sf": stt, "rows": rows, "K": k, "tiled": True}


def mx_gemm(a: dict, a_g: torch.Tensor, w: dict, w_g: torch.Tensor, a_group_rows: int = 1,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[B, N] fp16 = deq(a) . deq(w)^T for MXFP4 operands in the MX tile layout
    (dicts from mx_quantize(tiled=True) or mx_tile)."""
    if not (a.get("tiled") and w.get("tiled")):
        raise ValueError("mx_gemm takes operands in the MX tile layout")
    B, N, K = a["rows"], w["rows"], a["K"]
    if w["K"] != K:
        raise ValueError("operand K differs")
    for op, r in ((a, B), (w, N)):
        nc, ns = mx_tiled_sizes(r, K)
        if op["codes"].dtype != torch.uint8 or op["sf"].dtype != torch.uint8 or \
                op["codes"].numel() < nc or op["sf"].numel() < ns:
            raise ValueError("tile buffers smaller than the MX tile layout of %d x %d" % (r, K))
    _need(a_g, "a_g", torch.float32, min_numel=B // max(a_group_rows, 1))
    _need(w_g, "w_g", torch.float32, min_numel=1)
    if out is not None:
        _need(out, "out", torch.float16, (B, N))
    _check_dev(a["codes"], a["sf"], a_g, w["codes"], w["sf"], w_g, out)
    y = out if out is not None else torch.empty((B, N), dtype=torch.float16, device=a["codes"].device)
    rc = _lib.nvfp4_mx_gemm(_ptr(a["codes"]), _ptr(a["sf"]), _ptr(a_g), a_group_rows, _ptr(w["codes"]),
                            _ptr(w["sf"]), _ptr(w_g), _ptr(y), B, N, K, _stream(stream))
    if rc != NVFP4_OK:
        raise Nvfp4Error(rc, "nvfp4_mx_gemm")
    return y


# ---------------------------------------------------------------- calls of a few microseconds
#
# A decode step's kernels take a few microseconds, about as long as checking their operands one by
# one in Python.  Each call therefore first asks one plain question -- are the operands what they are
# in an ordinary call -- and only where the answer is no runs the checks that name what is wrong.

def _need_gpu(first: torch.Tensor, *ts):
    dev = first.device
    if dev.type != "cuda" or dev.index != torch.cuda.current_device():
        raise ValueError("tensors must be on the current GPU")
    for t in ts:
        if t is not None and t.device != dev:
            raise ValueError("tensors must be on one GPU")


def _dense(t: torch.Tensor, name: str, dtype, shape):
    _need(t, name, dtype, shape)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _gpu_of(t) -> int:
    """Index of the tensor's GPU if that is the current one, else -1."""
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    return dev if dev >= 0 and dev == torch._C._cuda_getDevice() else -1


def _is(t, dtype, shape, dev) -> bool:
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


def _need_heads(t, name: str):
    """[tokens, heads, head_dim] with a dense last dimension; other strides are free."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError("%s must be a 3-D tensor [tokens, heads, head_dim]" % name)
    if t.stride(2) != 1 and t.shape[2] > 1 and t.numel() > 0:
        raise ValueError("%s must have a dense last dimension" % name)


def _steps(t):
    """Token and head stride in elements; a dimension of size 1 has none."""
    a, b, _ = t.stride()
    return (a if t.shape[0] > 1 else 0), (b if t.shape[1] > 1 else 0)


def _fresh(stream, make):
    """New buffers of a call: allocated on the stream that the call runs on, so that their
    memory is not reused before the call's work on that stream is done."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        return make()


def _handle(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _overlap(a, b) -> bool:
    """Whether two dense tensors share memory."""
    x, y, n, m = a.data_ptr(), b.data_ptr(), a.numel() * a.element_size(), b.numel() * b.element_size()
    return n > 0 and m > 0 and x < y + m and y < x + n


# ---------------------------------------------------------------- FP8, a scale per 128

_FP8 = torch.float8_e4m3fn


def _check_fp8_quantize(x, k, block_rows, out):
    _need_2d(x, "x")
    _dtype_code(x)
    rows = x.shape[0]
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128, got %s" % (block_rows,))
    if out is not None:
        _dense(out.get("codes"), "out['codes']", _FP8, (rows, k))
        _dense(out.get("scale"), "out['scale']", torch.float32, (-(-rows // block_rows), -(-k // 128)))
    _need_gpu(x, *(() if out is None else (out["codes"], out["scale"])))


def fp8_quantize(x: torch.Tensor, block_rows: int = 1, act: str = "none", out: dict | None = None,
                 stream=None) -> dict:
    """E4M3 quantization of x [rows, k] (bfloat16 or float16; [rows, 2 k] for act="swiglu") with one float32
    scale per 128 values of a row (block_rows=1: activations) or per 128 x 128 values (block_rows=128:
    weights), with the optional activation in front.  Returns dict(codes [rows, k] float8_e4m3fn, scale
    [ceil(rows / block_rows), ceil(k / 128)] float32)."""
    a = _act_code(act)
    dev = _gpu_of(x)
    try:
        rows, k_in = x.shape
        k = k_in // 2 if a == 1 else k_in
        plain = (dev >= 0 and x.dtype in _TYPE_CODE and x.is_contiguous() and (block_rows == 1 or block_rows == 128) and
                 (out is None or (_is(out["codes"], _FP8, (rows, k), dev) and
                                  _is(out["scale"], torch.float32, (-(-rows // block_rows), -(-k // 128)), dev))))
    except (AttributeError, KeyError, TypeError, ValueError):
        plain = False
    if not plain:
        _need_2d(x, "x")
        k_in = x.shape[1]
        k = k_in // 2 if a == 1 else k_in
        _check_fp8_quantize(x, k, block_rows, out)
    if a == 1 and k_in % 2:
        raise ValueError("x must hold a gate and an up half for swiglu, got %d columns" % k_in)
    if out is None:
        out = _fresh(stream, lambda: {
            "codes": torch.empty((rows, k), dtype=_FP8, device=x.device),
            "scale": torch.empty((-(-rows // block_rows), -(-k // 128)), dtype=torch.float32, device=x.device)})
    st = _lib.nvfp4_fp8_quantize(x.data_ptr(), _TYPE_CODE[x.dtype], rows, k, a, block_rows, out["codes"].data_ptr(),
                                 out["scale"].data_ptr(), _handle(stream, dev))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_fp8_quantize")
    return out


def _check_fp8_gemm(a, a_scale, w, w_scale, out):
    _need_2d(a, "a")
    _need_2d(w, "w")
    (B, K), N = a.shape, w.shape[0]
    _dense(a, "a", _FP8, (B, K))
    _dense(w, "w", _FP8, (N, K))
    _dense(a_scale, "a_scale", torch.float32, (B, -(-K // 128)))
    _dense(w_scale, "w_scale", torch.float32, (-(-N // 128), -(-K // 128)))
    if out is not None:
        _need_2d(out, "out")
        _dtype_code(out)
        _dense(out, "out", out.dtype, (B, N))
    _need_gpu(a, a_scale, w, w_scale, out)


def fp8_gemm(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
             out_dtype: torch.dtype = torch.float16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[B, N] = sum_k a[b, k] a_scale[b, k / 128] w[n, k] w_scale[n / 128, k / 128] for float8_e4m3fn a [B, K]
    and w [N, K] with float32 scales (fp8_quantize with block_rows 1 and 128, or a checkpoint's).
    float16 or bfloat16 out (out_dtype, or the type of `out`).  The sums inside a block of 128 are those of the E4M3 matrix
    instructions (about 2^-16 of the block's size, at most 7 * 2^-13), the others binary32."""
    dev = _gpu_of(a)
    f32 = torch.float32
    try:
        (B, K), (N, K2) = a.shape, w.shape
        nkb = -(-K // 128)
        plain = (dev >= 0 and K == K2 and _is(a, _FP8, (B, K), dev) and _is(w, _FP8, (N, K), dev) and
                 _is(a_scale, f32, (B, nkb), dev) and _is(w_scale, f32, (-(-N // 128), nkb), dev) and
                 (out is None or (out.dtype in _TYPE_CODE and _is(out, out.dtype, (B, N), dev))))
    except (AttributeError, TypeError, ValueError):
        plain = False
    if not plain:
        _check_fp8_gemm(a, a_scale, w, w_scale, out)
    if out is None:
        if out_dtype not in _TYPE_CODE:
            raise TypeError("out_dtype must be bfloat16 or float16")
        out = _fresh(stream, lambda: torch.empty((B, N), dtype=out_dtype, device=a.device))
    st = _lib.nvfp4_fp8_gemm(a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), out.data_ptr(),
                             _TYPE_CODE[out.dtype], B, N, K, _handle(stream, dev))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_fp8_gemm")
    return out


# ---------------------------------------------------------------- MoE layer of a decode step

@functools.lru_cache(maxsize=1024)
def moe_decode_workspace_size(tokens: int, experts: int, top_k: int, hidden: int, inter: int) -> int:
    _need_32_bits(tokens=tokens, experts=experts, top_k=top_k, hidden=hidden, inter=inter)
    return int(_lib.nvfp4_moe_decode_workspace_size(tokens, experts, top_k, hidden, inter))


def _check_moe_decode(x, router, bias, w1, w1_sf, w1_g, w2, w2_sf, w2_g, gated, out, workspace):
    _need_2d(x, "x")
    _dtype_code(x)
    _need_2d(router, "router")
    (T, hidden), E = x.shape, router.shape[0]
    _dense(x, "x", x.dtype, (T, hidden))
    _dense(router, "router", x.dtype, (E, hidden))
    _dense(bias, "bias", torch.float32, (E,))
    if not isinstance(w2, torch.Tensor) or w2.dim() != 3:
        raise ValueError("w2 must be a 3-D tensor [experts, hidden, inter/2]")
    inter = 2 * w2.shape[2]
    rows = 2 * inter if gated else inter
    _dense(w1, "w1", torch.uint8, (E, rows, hidden // 2))
    _dense(w1_sf, "w1_sf", torch.uint8, (E, rows, hidden // 16))
    _dense(w1_g, "w1_g", torch.float32, (E,))
    _dense(w2, "w2", torch.uint8, (E, hidden, inter // 2))
    _dense(w2_sf, "w2_sf", torch.uint8, (E, hidden, inter // 16))
    _dense(w2_g, "w2_g", torch.float32, (E,))
    if out is not None:
        _dense(out, "out", x.dtype, (T, hidden))
    _need_gpu(x, router, bias, w1, w1_sf, w1_g, w2, w2_sf, w2_g, out, workspace)


def _plain_moe_decode(x, router, bias, w1, w1_sf, w1_g, w2, w2_sf, w2_g, gated, out, workspace, dev) -> bool:
    try:
        dt, u8, f32 = x.dtype, torch.uint8, torch.float32
        (T, hidden), (E, _) = x.shape, router.shape
        inter = 2 * w2.shape[2]
        rows = 2 * inter if gated else inter
        return (dt in _TYPE_CODE and _is(x, dt, (T, hidden), dev) and _is(router, dt, (E, hidden), dev) and
                _is(bias, f32, (E,), dev) and _is(w1, u8, (E, rows, hidden // 2), dev) and
                _is(w1_sf, u8, (E, rows, hidden // 16), dev) and _is(w1_g, f32, (E,), dev) and
                _is(w2, u8, (E, hidden, inter // 2), dev) and _is(w2_sf, u8, (E, hidden, inter // 16), dev) and
                _is(w2_g, f32, (E,), dev) and (out is None or _is(out, dt, (T, hidden), dev)) and
                (workspace is None or workspace.get_device() == dev))
    except (AttributeError, IndexError, TypeError, ValueError):
        return False


def moe_decode(x: torch.Tensor, router: torch.Tensor, bias: torch.Tensor, w1: torch.Tensor, w1_sf: torch.Tensor,
               w1_g: torch.Tensor, w2: torch.Tensor, w2_sf: torch.Tensor, w2_g: torch.Tensor, top_k: int,
               n_group: int = 1, topk_group: int = 1, norm_topk_prob: bool = True, routed_scaling: float = 1.0,
               act: str = "relu2", tiled: bool = False, out: torch.Tensor | None = None, want_routing: bool = False,
               workspace: torch.Tensor | None = None, stream=None):
    """A whole MoE layer for up to 32 tokens: x [tokens, hidden] and router [experts, hidden] (float16 or
    bfloat16), the expert weights of moe_w4a16() (or, with `tiled`, of moe_pretile_weights()); for act="swiglu" w1
    holds [experts, 2 inter, ...] gate and up rows.  `out` may be x.  Returns out [tokens, hidden] of x's type, or (out, ids,
    weights) with want_routing."""
    a = _act_code(act)
    gated = a == ACT["swiglu"]
    dev = _gpu_of(x)
    if dev < 0 or not _plain_moe_decode(x, router, bias, w1, w1_sf, w1_g, w2, w2_sf, w2_g, gated, out, workspace, dev):
        _check_moe_decode(x, router, bias, w1, w1_sf, w1_g, w2, w2_sf, w2_g, gated, out, workspace)
    (T, hidden), E, inter = x.shape, router.shape[0], 2 * w2.shape[2]
    if (T | hidden | E | inter | top_k | n_group | topk_group) >> 31:
        _need_32_bits(tokens=T, hidden=hidden, experts=E, inter=inter, top_k=top_k, n_group=n_group, topk_group=topk_group)
    if out is None:
        out = _fresh(stream, lambda: torch.empty((T, hidden), dtype=x.dtype, device=x.device))
    ids = wts = None
    if want_routing:
        ids, wts = _fresh(stream, lambda: (torch.empty((T, top_k), dtype=torch.int32, device=x.device),
                                           torch.empty((T, top_k), dtype=torch.float32, device=x.device)))
    ws, wsb = _fresh(stream, lambda: _workspace(moe_decode_workspace_size(T, E, top_k, hidden, inter), x.device, workspace))
    st = _lib.nvfp4_moe_decode(x.data_ptr(), _TYPE_CODE[x.dtype], router.data_ptr(), bias.data_ptr(), w1.data_ptr(),
                               w1_sf.data_ptr(), w1_g.data_ptr(), w2.data_ptr(), w2_sf.data_ptr(), w2_g.data_ptr(),
                               1 if tiled else 0, out.data_ptr(), None if ids is None else ids.data_ptr(),
                               None if wts is None else wts.data_ptr(), T, E, top_k, hidden, inter, a, n_group,
                               topk_group, 1 if norm_topk_prob else 0, routed_scaling,
                               None if ws is None else ws.data_ptr(), wsb, _handle(stream, dev))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_moe_decode")
    return (out, ids, wts) if want_routing else out


# ---------------------------------------------------------------- serving attention

def _check_page_maps(ctx_lens, new_lens, block_table, free_pages, tokens, out):
    if not isinstance(ctx_lens, torch.Tensor) or ctx_lens.dim() != 1:
        raise ValueError("ctx_lens must be a 1-D tensor")
    n = ctx_lens.shape[0]
    _dense(ctx_lens, "ctx_lens", torch.int32, (n,))
    _dense(new_lens, "new_lens", torch.int32, (n,))
    _need_2d(block_table, "block_table")
    _dense(block_table, "block_table", torch.int32, (n, block_table.shape[1]))
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise ValueError("free_pages must be a 1-D tensor")
    _dense(free_pages, "free_pages", torch.int32, free_pages.shape)
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    if out is not None:
        for key, dt, shape in (("cu_new", torch.int32, (n + 1,)), ("kv_lens", torch.int32, (n,)),
                               ("slot_map", torch.int64, (tokens,)), ("positions", torch.int32, (tokens,)),
                               ("taken", torch.int32, (1,))):
            _dense(out.get(key), "out['%s']" % key, dt, shape)
    written = [("block_table", block_table)]
    if out is not None:
        written += [("out['%s']" % key, out[key]) for key in ("cu_new", "kv_lens", "slot_map", "positions", "taken")]
    everything = written + [("ctx_lens", ctx_lens), ("new_lens", new_lens), ("free_pages", free_pages)]
    for i, (name, t) in enumerate(written):
        for other, u in everything[i + 1:]:
            in_place = name == "out['kv_lens']" and other == "ctx_lens" and t.data_ptr() == u.data_ptr()
            if _overlap(t, u) and not in_place:
                raise ValueError("%s must not overlap %s" % (name, other))
    _need_gpu(ctx_lens, new_lens, block_table, free_pages, *(t for _, t in written))


def _plain_page_maps(ctx_lens, new_lens, block_table, free_pages, tokens, out, dev) -> bool:
    try:
        n, i32 = ctx_lens.shape[0], torch.int32
        return (tokens >= 0 and _is(ctx_lens, i32, (n,), dev) and _is(new_lens, i32, (n,), dev) and
                _is(block_table, i32, (n, block_table.shape[1]), dev) and
                _is(free_pages, i32, (free_pages.shape[0],), dev) and
                (out is None or
                 (_is(out["cu_new"], i32, (n + 1,), dev) and _is(out["kv_lens"], i32, (n,), dev) and
                  _is(out["slot_map"], torch.int64, (tokens,), dev) and _is(out["positions"], i32, (tokens,), dev) and
                  _is(out["taken"], i32, (1,), dev))))
    except (AttributeError, IndexError, KeyError, TypeError):
        return False


def page_maps(ctx_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
              free_pages: torch.Tensor, page_size: int, tokens: int, out: dict | None = None,
              stream=None) -> dict:
    """One step's bookkeeping on the GPU: extends block_table [seqs, max_pages] in place with pages
    from free_pages for new_lens[i] tokens after the ctx_lens[i] cached ones, and returns
    dict(cu_new [seqs + 1], kv_lens [seqs], slot_map [tokens] int64, positions [tokens],
    taken [1]).  `tokens` is the size of the maps (entries past the last token are -1); `taken`
    above len(free_pages) means that pages ran out.  out["kv_lens"] may be ctx_lens itself, which then
    holds the new lengths; other buffers must not overlap."""
    if page_size >> 31:
        _need_32_bits(page_size=page_size)
    tokens, dev = int(tokens), _gpu_of(ctx_lens)
    if dev < 0 or not _plain_page_maps(ctx_lens, new_lens, block_table, free_pages, tokens, out, dev):
        _check_page_maps(ctx_lens, new_lens, block_table, free_pages, tokens, out)
    (n, width), (num_free,) = block_table.shape, free_pages.shape
    if (n | width | num_free) >> 31:
        _need_32_bits(seqs=n, max_pages=width, num_free=num_free)
    if out is None:
        where = ctx_lens.device
        out = _fresh(stream, lambda: {
            "cu_new": torch.empty(n + 1, dtype=torch.int32, device=where),
            "kv_lens": torch.empty(n, dtype=torch.int32, device=where),
            "slot_map": torch.empty(tokens, dtype=torch.int64, device=where),
            "positions": torch.empty(tokens, dtype=torch.int32, device=where),
            "taken": torch.empty(1, dtype=torch.int32, device=where)})
    st = _lib.nvfp4_page_maps(ctx_lens.data_ptr(), new_lens.data_ptr(), n, block_table.data_ptr(),
                              width, free_pages.data_ptr(), num_free, page_size, tokens,
                              out["cu_new"].data_ptr(), out["kv_lens"].data_ptr(), out["slot_map"].data_ptr(),
                              out["positions"].data_ptr(), out["taken"].data_ptr(), _handle(stream, dev))
    if st != NVFP4_OK:
        if st == NVFP4_EINVAL:   # buffers that overlap: only the library looks for them in a plain call
            _check_page_maps(ctx_lens, new_lens, block_table, free_pages, tokens, out)
        raise Nvfp4Error(st, "nvfp4_page_maps")
    return out


def _check_caches(k_cache, v_cache, dtype):
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a 4-D tensor [pages, kv_heads, page_size, head_dim]")
    _dense(k_cache, "k_cache", dtype, k_cache.shape)
    _dense(v_cache, "v_cache", dtype, k_cache.shape)


def _check_kv_operands(k, v, slot_map, k_cache, v_cache):
    _need_heads(k, "k")
    _need_heads(v, "v")
    _dtype_code(k)
    T, H, D = k.shape
    _need(v, "v", k.dtype, (T, H, D))
    _check_caches(k_cache, v_cache, k.dtype)
    if (k_cache.shape[1], k_cache.shape[3]) != (H, D):
        raise ValueError("the cache holds %d heads of %d, k has %d of %d" % (k_cache.shape[1], k_cache.shape[3], H, D))
    _dense(slot_map, "slot_map", torch.int64, (T,))


def _check_kv_write(k, v, slot_map, k_cache, v_cache):
    _check_kv_operands(k, v, slot_map, k_cache, v_cache)
    _need_gpu(k, v, slot_map, k_cache, v_cache)


def _plain_kv_write(k, v, slot_map, k_cache, v_cache, dev) -> bool:
    try:
        dt, shape, cache = k.dtype, k.shape, k_cache.shape
        T, H, D = shape
        _, heads, _, dim = cache
        return (dt in _TYPE_CODE and T > 0 and heads == H and dim == D and v.dtype is dt and v.shape == shape and
                k.stride(2) == 1 and v.stride(2) == 1 and k.get_device() == dev and v.get_device() == dev and
                _is(slot_map, torch.int64, (T,), dev) and _is(k_cache, dt, cache, dev) and _is(v_cache, dt, cache, dev))
    except (AttributeError, IndexError, TypeError, ValueError):
        return False


def kv_write(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor, k_cache: torch.Tensor,
             v_cache: torch.Tensor, stream=None) -> None:
    """Writes k, v [tokens, kv_heads, head_dim] to their slots of the caches
    [pages, kv_heads, page_size, head_dim]; slots outside the cache (-1) are skipped."""
    dev = _gpu_of(k)
    if dev < 0 or not _plain_kv_write(k, v, slot_map, k_cache, v_cache, dev):
        _check_kv_write(k, v, slot_map, k_cache, v_cache)
    T = k.shape[0]
    pages, H, page_size, D = k_cache.shape
    if (H | page_size | D) >> 31:
        _need_32_bits(kv_heads=H, page_size=page_size, head_dim=D)
    (kt, kh), (vt, vh) = _steps(k), _steps(v)
    st = _lib.nvfp4_kv_write(k.data_ptr(), v.data_ptr(), T, H, D, kt, kh, vt, vh, slot_map.data_ptr(),
                             k_cache.data_ptr(), v_cache.data_ptr(), page_size, pages,
                             _handle(stream, dev))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_kv_write")


def _check_rope(q, k, v, positions, inv_freq, slot_map, k_cache, v_cache, q_out, k_out):
    _check_kv_operands(k, v, slot_map, k_cache, v_cache)
    T, _, D = k.shape
    if q is not None:
        _need_heads(q, "q")
        _need(q, "q", k.dtype, (T, q.shape[1], D))
    _dense(positions, "positions", torch.int32, (T,))
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a 1-D tensor of half the rotary dimension")
    _dense(inv_freq, "inv_freq", torch.float32, inv_freq.shape)
    for t, like, name in ((q_out, q, "q_out"), (k_out, k, "k_out")):
        if t is None:
            continue
        if like is None:
            raise ValueError("%s needs its input" % name)
        _need_heads(t, name)
        _need(t, name, k.dtype, like.shape)
        if t.data_ptr() == like.data_ptr() and _steps(t) != _steps(like) and t.numel() > 0:
            raise ValueError("%s in the place of its input must have its strides" % name)
    _need_gpu(k, v, slot_map, k_cache, v_cache, q, positions, inv_freq, q_out, k_out)


def rope_kv_write(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                  inv_freq: torch.Tensor, slot_map: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  interleaved: bool = False, mscale: float = 1.0, q_out: torch.Tensor | None = None,
                  k_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Rotates q [tokens, q_heads, head_dim] and k [tokens, kv_heads, head_dim] by positions [tokens]
    int32 and inv_freq [rotary_dim / 2] float32, and writes k and v to their slots of the caches
    [pages, kv_heads, page_size, head_dim], in one launch.  Pairs are (i, i + rotary_dim / 2), or
    (2 i, 2 i + 1) with `interleaved`; cosine and sine are multiplied by mscale.  Returns q_out (new unless
    given; may be q itself); k_out (may be k itself) receives the rotated keys too.  Nothing is written for
    tokens of a negative position (in a new q_out their rows are undefined); slots outside the cache are
    skipped.  q may be None."""
    dev, i32, ints = _gpu_of(k), torch.int32, torch.int64
    try:
        shape, dt, cache = k.shape, k.dtype, k_cache.shape
        T, Hk, D = shape
        pages, heads, page_size, dim = cache
        kt, kh, k1 = k.stride()
        vt, vh, v1 = v.stride()
        half = inv_freq.shape[0]
        plain = (dev >= 0 and T > 0 and dt in _TYPE_CODE and heads == Hk and dim == D and k1 == v1 == 1 and
                 v.dtype is dt and v.shape == shape and v.get_device() == dev and
                 _is(k_cache, dt, cache, dev) and _is(v_cache, dt, cache, dev) and
                 _is(slot_map, ints, (T,), dev) and _is(positions, i32, (T,), dev) and
                 _is(inv_freq, torch.float32, (half,), dev))
        Hq = qt = qh = qot = qoh = kot = koh = 0
        if plain and q is not None:
            _, Hq, _ = of_q = q.shape
            qt, qh, q1 = q.stride()
            plain = q.dtype is dt and of_q == (T, Hq, D) and q1 == 1 and q.get_device() == dev
            if plain and q_out is not None:
                qot, qoh, q1 = q_out.stride()
                plain = (q_out.dtype is dt and q_out.shape == of_q and q1 == 1 and q_out.get_device() == dev and
                         (q_out.data_ptr() != q.data_ptr() or (qot == qt and qoh == qh)))
        elif q_out is not None:
            plain = False
        if plain and k_out is not None:
            kot, koh, k1 = k_out.stride()
            plain = (k_out.dtype is dt and k_out.shape == shape and k1 == 1 and k_out.get_device() == dev and
                     (k_out.data_ptr() != k.data_ptr() or (kot == kt and koh == kh)))
    except (AttributeError, IndexError, TypeError, ValueError):
        plain = False
    if not plain:
        _check_rope(q, k, v, positions, inv_freq, slot_map, k_cache, v_cache, q_out, k_out)
        T, Hk, D = k.shape
        pages, _, page_size, _ = k_cache.shape
        half, Hq = inv_freq.shape[0], 0 if q is None else q.shape[1]
        (qt, qh), (kt, kh), (vt, vh) = (0, 0) if q is None else _steps(q), _steps(k), _steps(v)
        (qot, qoh), (kot, koh) = ((0, 0) if t is None else _steps(t) for t in (q_out, k_out))
    if (Hq | Hk | page_size | D | 2 * half) >> 31:
        _need_32_bits(q_heads=Hq, kv_heads=Hk, page_size=page_size, head_dim=D, rotary_dim=2 * half)
    if q is not None and q_out is None:
        q_out = _fresh(stream, lambda: torch.empty((T, Hq, D), dtype=q.dtype, device=q.device))
        qot, qoh = Hq * D, D
    st = _lib.nvfp4_rope_kv_write(None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(), _TYPE_CODE[k.dtype],
                                  T, Hq, Hk, D, qt, qh, kt, kh, vt, vh, positions.data_ptr(), inv_freq.data_ptr(),
                                  2 * half, 1 if interleaved else 0, mscale, slot_map.data_ptr(),
                                  None if q_out is None else q_out.data_ptr(), qot, qoh,
                                  None if k_out is None else k_out.data_ptr(), kot, koh,
                                  k_cache.data_ptr(), v_cache.data_ptr(), page_size, pages, _handle(stream, dev))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_rope_kv_write")
    return q_out


def _check_attn_out(q, out, lse):
    T, H, D = q.shape
    if out is not None:
        _dense(out, "out", q.dtype, (T, H, D))
    if lse is not None:
        _dense(lse, "lse", torch.float32, (T, H))


def _check_prompt_attn(q, k, v, cu_seqlens, out, lse):
    _need_heads(q, "q")
    _need_heads(k, "k")
    _need_heads(v, "v")
    _dtype_code(q)
    T, _, D = q.shape
    _need(k, "k", q.dtype, (T, k.shape[1], D))
    _need(v, "v", q.dtype, k.shape)
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be a 1-D tensor of seqs + 1 entries")
    _dense(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape)
    _check_attn_out(q, out, lse)
    _need_gpu(q, k, v, cu_seqlens, out, lse)


def _plain_prompt_attn(q, k, v, cu_seqlens, out, lse, dev) -> bool:
    try:
        dt, shape = q.dtype, q.shape
        T, H, D = shape
        return (dt in _TYPE_CODE and T > 0 and k.dtype is dt and v.dtype is dt and
                k.shape == (T, k.shape[1], D) and v.shape == k.shape and
                q.stride(2) == 1 and k.stride(2) == 1 and v.stride(2) == 1 and
                q.get_device() == dev and k.get_device() == dev and v.get_device() == dev and
                cu_seqlens.shape[0] > 0 and _is(cu_seqlens, torch.int32, (cu_seqlens.shape[0],), dev) and
                (out is None or _is(out, dt, shape, dev)) and (lse is None or _is(lse, torch.float32, (T, H), dev)))
    except (AttributeError, IndexError, TypeError, ValueError):
        return False


def prompt_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                scale: float | None = None, window: int = 0, want_lse: bool = False,
                out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """Causal attention of whole packed prompts: q [tokens, q_heads, head_dim], k and v
    [tokens, kv_heads, head_dim] (any token and head strides that are multiples of 8), cu_seqlens
    [seqs + 1] int32.  Returns out, or (out, lse) with want_lse or a given lse buffer.  scale
    defaults to head_dim ** -0.5; window > 0 limits a row to the last `window` keys."""
    if window >> 31:
        _need_32_bits(window=window)
    dev = _gpu_of(q)
    if dev < 0 or not _plain_prompt_attn(q, k, v, cu_seqlens, out, lse, dev):
        _check_prompt_attn(q, k, v, cu_seqlens, out, lse)
    T, Hq, D = q.shape
    Hk, starts = k.shape[1], cu_seqlens.shape[0]
    if (Hq | Hk | starts) >> 31:
        _need_32_bits(q_heads=Hq, kv_heads=Hk, seqs=starts)
    if out is None:
        out = _fresh(stream, lambda: torch.empty((T, Hq, D), dtype=q.dtype, device=q.device))
    if lse is None and want_lse:
        lse = _fresh(stream, lambda: torch.empty((T, Hq), dtype=torch.float32, device=q.device))
    (qt, qh), (kt, kh), (vt, vh) = _steps(q), _steps(k), _steps(v)
    st = _lib.nvfp4_prompt_attn(q.data_ptr(), k.data_ptr(), v.data_ptr(), _TYPE_CODE[q.dtype], cu_seqlens.data_ptr(),
                                starts - 1, T, Hq, Hk, D, qt, qh, kt, kh, vt, vh,
                                (D or 1) ** -0.5 if scale is None else scale, window, out.data_ptr(),
                                None if lse is None else lse.data_ptr(), _handle(stream, dev))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_prompt_attn")
    return out if lse is None else (out, lse)


@functools.lru_cache(maxsize=1024)
def paged_attn_workspace_size(seqs: int, tokens: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(_lib.nvfp4_paged_attn_workspace_size(seqs, tokens, q_heads, kv_heads, head_dim))


def _check_paged_attn(q, k_cache, v_cache, block_table, cu_new, kv_lens, out, lse, workspace):
    _need_heads(q, "q")
    _dtype_code(q)
    _check_caches(k_cache, v_cache, q.dtype)
    if k_cache.shape[3] != q.shape[2]:
        raise ValueError("q has head_dim %d, the cache %d" % (q.shape[2], k_cache.shape[3]))
    _need_2d(block_table, "block_table")
    n = block_table.shape[0]
    _dense(block_table, "block_table", torch.int32, block_table.shape)
    _dense(cu_new, "cu_new", torch.int32, (n + 1,))
    _dense(kv_lens, "kv_lens", torch.int32, (n,))
    _check_attn_out(q, out, lse)
    _need_gpu(q, k_cache, v_cache, block_table, cu_new, kv_lens, out, lse, workspace)


def _plain_paged_attn(q, k_cache, v_cache, block_table, cu_new, kv_lens, out, lse, workspace, dev) -> bool:
    try:
        dt, shape, cache, i32 = q.dtype, q.shape, k_cache.shape, torch.int32
        T, H, D = shape
        n, width = block_table.shape
        _, _, _, dim = cache
        return (dt in _TYPE_CODE and T > 0 and dim == D and q.stride(2) == 1 and q.get_device() == dev and
                _is(k_cache, dt, cache, dev) and _is(v_cache, dt, cache, dev) and
                _is(block_table, i32, (n, width), dev) and _is(cu_new, i32, (n + 1,), dev) and
                _is(kv_lens, i32, (n,), dev) and (out is None or _is(out, dt, shape, dev)) and
                (lse is None or _is(lse, torch.float32, (T, H), dev)) and
                (workspace is None or workspace.get_device() == dev))
    except (AttributeError, IndexError, TypeError, ValueError):
        return False


def paged_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
               cu_new: torch.Tensor, kv_lens: torch.Tensor, scale: float | None = None, window: int = 0,
               want_lse: bool = False, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None):
    """Causal attention of new tokens over the paged cache, which already holds them: q [tokens,
    q_heads, head_dim] packed by cu_new [seqs + 1], caches [pages, kv_heads, page_size, head_dim],
    block_table [seqs, max_pages], kv_lens [seqs] (all int32).  Decode steps, chunks of prompts and
    mixtures.  Returns out, or (out, lse) with want_lse or a given lse buffer."""
    if window >> 31:
        _need_32_bits(window=window)
    dev = _gpu_of(q)
    if dev < 0 or not _plain_paged_attn(q, k_cache, v_cache, block_table, cu_new, kv_lens, out, lse, workspace, dev):
        _check_paged_attn(q, k_cache, v_cache, block_table, cu_new, kv_lens, out, lse, workspace)
    T, Hq, D = q.shape
    pages, Hk, page_size, _ = k_cache.shape
    n, width = block_table.shape
    if (Hq | Hk | page_size | n | width) >> 31:
        _need_32_bits(q_heads=Hq, kv_heads=Hk, page_size=page_size, seqs=n, max_pages=width)
    if out is None:
        out = _fresh(stream, lambda: torch.empty((T, Hq, D), dtype=q.dtype, device=q.device))
    if lse is None and want_lse:
        lse = _fresh(stream, lambda: torch.empty((T, Hq), dtype=torch.float32, device=q.device))
    ws, wsb = _fresh(stream, lambda: _workspace(paged_attn_workspace_size(n, T, Hq, Hk, D), q.device, workspace))
    qt, qh = _steps(q)
    st = _lib.nvfp4_paged_attn(q.data_ptr(), _TYPE_CODE[q.dtype], k_cache.data_ptr(), v_cache.data_ptr(),
                               block_table.data_ptr(), cu_new.data_ptr(), kv_lens.data_ptr(), n, T, Hq, Hk, D,
                               page_size, pages, width, qt, qh, (D or 1) ** -0.5 if scale is None else scale, window,
                               out.data_ptr(), None if lse is None else lse.data_ptr(),
                               None if ws is None else ws.data_ptr(), wsb, _handle(stream, dev))
    if st != NVFP4_OK:
        raise Nvfp4Error(st, "nvfp4_paged_attn")
    return out if lse is None else (out, lse)
