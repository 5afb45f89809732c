"""Python binding of libmoefp8.so, the sm_100a fused W8A8 block-scaled MoE
library (C ABI in include/moefp8.h).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  PyTorch supplies device memory and streams.  The
binding raises if the compiled library is missing; there is no fallback.

Functions keep the C names:
  moe_route_permute, moe_fp8_fused, moe_fp8_fused_debug,
  fp8_groupwise_moe_gemm, swiglu_mxfp8_quant, moe_select_tile_m,
  moe_workspace_size, moe_route_workspace_size, moe_get_device_status,
  moe_set_wait_timeout_ns, moe_set_expert_fusion, moe_status_string.
Tensor arguments may be torch tensors (their data_ptr is passed) or raw
integer device addresses.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "MoEError", "lib", "lib_path", "EXPORTS",
    "moe_route_permute", "moe_fp8_fused", "moe_fp8_fused_debug", "fp8_groupwise_moe_gemm",
    "swiglu_mxfp8_quant", "moe_select_tile_m", "moe_workspace_size", "moe_route_workspace_size",
    "moe_get_device_status", "moe_set_wait_timeout_ns", "moe_status_string",
    "moe_set_stage_events", "moe_route_permute_noalloc", "mxfp8_moe_gemm",
    "mxfp8_tile_scales", "moe_mxfp8_fused", "moe_mxfp8_fused_debug", "moe_router_topk",
    "nvfp4_moe_gemm", "nvfp4_tile_scales", "moe_nvfp4_fused", "moe_nvfp4_fused_debug",
    "nvfp4_quantize", "moe_tactic_tune_gemm", "moe_tactic_lookup", "moe_tactic_store",
    "moe_tactic_clear", "moe_ep_workspace_size", "moe_ep_plan", "moe_ep_pack",
    "moe_fp8_expert_rows_workspace_size", "moe_fp8_expert_rows", "moe_combine", "moe_router_route",
    "moe_set_expert_fusion", "moe_fp8_fused_plan",
    "moe_router_score_topk", "moe_router_score_route", "moe_rmsnorm_quant", "int8_quantize",
    "int8_moe_gemm",
    "MOE_FUSION_AUTO", "MOE_FUSION_ON", "MOE_FUSION_OFF",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoefp8.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_CUDA = 3
MOE_ERR_NO_TILE_CONFIG = 4
MOE_ERR_DEVICE_TIMEOUT = 5
MOE_ERR_BAD_EXPERT_ID = 6

MOE_FUSION_AUTO = 0
MOE_FUSION_ON = 1
MOE_FUSION_OFF = 2

# Every symbol declared in include/moefp8.h.
EXPORTS = (
    "moe_status_string", "moe_route_workspace_size", "moe_route_permute", "moe_workspace_size",
    "moe_fp8_fused", "moe_fp8_fused_debug", "fp8_groupwise_moe_gemm", "moe_select_tile_m",
    "swiglu_mxfp8_quant", "moe_get_device_status", "moe_set_wait_timeout_ns",
    "moe_set_stage_events", "moe_route_permute_noalloc", "mxfp8_moe_gemm", "mxfp8_tile_scales",
    "moe_mxfp8_fused", "moe_mxfp8_fused_debug", "moe_router_topk", "nvfp4_moe_gemm",
    "nvfp4_tile_scales", "moe_nvfp4_fused", "moe_nvfp4_fused_debug", "nvfp4_quantize",
    "moe_tactic_tune_gemm", "moe_tactic_lookup", "moe_tactic_store", "moe_tactic_clear",
    "moe_ep_workspace_size", "moe_ep_plan", "moe_ep_pack", "moe_fp8_expert_rows_workspace_size",
    "moe_fp8_expert_rows", "moe_combine", "moe_router_route", "moe_set_expert_fusion",
    "moe_fp8_fused_plan",
    "moe_router_score_topk", "moe_router_score_route", "moe_rmsnorm_quant", "int8_quantize",
    "int8_moe_gemm",
)

_lib = None


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = int(status)
        super().__init__(f"{where}: {moe_status_string(status)} ({status})")


def lib_path() -> str:
    return LIB_PATH


def lib():
    """Loads libmoefp8.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -m fp8_block_scaled_route_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, Z, U64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint64
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_status_string.argtypes = [I]
    L.moe_route_workspace_size.restype = Z
    L.moe_route_workspace_size.argtypes = [I, I, I]
    L.moe_route_permute.restype = I
    L.moe_route_permute.argtypes = [P, I, I, I, P, P, P, P, Z, P]
    L.moe_workspace_size.restype = Z
    L.moe_workspace_size.argtypes = [I] * 5
    L.moe_fp8_fused.restype = I
    L.moe_fp8_fused.argtypes = [P] * 8 + [I] * 5 + [P, Z, P]
    L.moe_fp8_fused_debug.restype = I
    L.moe_fp8_fused_debug.argtypes = [P] * 8 + [I] * 5 + [P, Z, P] + [P] * 4
    L.fp8_groupwise_moe_gemm.restype = I
    L.fp8_groupwise_moe_gemm.argtypes = [P] * 6 + [I] * 11 + [P]
    L.moe_select_tile_m.restype = I
    L.moe_select_tile_m.argtypes = [I] * 6 + [ctypes.POINTER(I), ctypes.POINTER(I)]
    L.swiglu_mxfp8_quant.restype = I
    L.swiglu_mxfp8_quant.argtypes = [P, P, P, I, I, P]
    L.mxfp8_moe_gemm.restype = I
    L.mxfp8_moe_gemm.argtypes = [P] * 6 + [I] * 6 + [P]
    L.moe_router_topk.restype = I
    L.moe_router_topk.argtypes = [P, I, I, I, P, P, P]
    L.mxfp8_tile_scales.restype = I
    L.mxfp8_tile_scales.argtypes = [P, P, I, I, P]
    L.nvfp4_moe_gemm.restype = I
    L.nvfp4_moe_gemm.argtypes = [P] * 7 + [I] * 6 + [P]
    L.nvfp4_tile_scales.restype = I
    L.nvfp4_tile_scales.argtypes = [P, P, I, I, P]
    F = ctypes.c_float
    L.moe_tactic_tune_gemm.restype = I
    L.moe_tactic_tune_gemm.argtypes = [P] * 6 + [I] * 7 + [P, ctypes.POINTER(I)]
    L.moe_tactic_lookup.restype = I
    L.moe_tactic_lookup.argtypes = [I] * 5 + [ctypes.POINTER(I)]
    L.moe_tactic_store.restype = I
    L.moe_tactic_store.argtypes = [I] * 6
    L.moe_tactic_clear.restype = None
    L.moe_tactic_clear.argtypes = []
    L.nvfp4_quantize.restype = I
    L.nvfp4_quantize.argtypes = [P, F, P, P, I, I, P]
    L.moe_nvfp4_fused.restype = I
    L.moe_nvfp4_fused.argtypes = [P] * 9 + [F, F, P] + [I] * 5 + [P, ctypes.c_size_t, P]
    L.moe_nvfp4_fused_debug.restype = I
    L.moe_nvfp4_fused_debug.argtypes = ([P] * 9 + [F, F, P] + [I] * 5 +
                                        [P, ctypes.c_size_t, P] + [P] * 4)
    L.moe_mxfp8_fused.restype = I
    L.moe_mxfp8_fused.argtypes = [P] * 8 + [I] * 5 + [P, ctypes.c_size_t, P]
    L.moe_mxfp8_fused_debug.restype = I
    L.moe_mxfp8_fused_debug.argtypes = [P] * 8 + [I] * 5 + [P, ctypes.c_size_t, P] + [P] * 4
    L.moe_get_device_status.restype = I
    L.moe_get_device_status.argtypes = [P, P]
    L.moe_set_wait_timeout_ns.restype = None
    L.moe_set_wait_timeout_ns.argtypes = [U64]
    L.moe_set_expert_fusion.restype = I
    L.moe_set_expert_fusion.argtypes = [I]
    L.moe_fp8_fused_plan.restype = I
    L.moe_fp8_fused_plan.argtypes = [I] * 5 + [P] * 3
    L.moe_route_permute_noalloc.restype = I
    L.moe_route_permute_noalloc.argtypes = [P, I, I, I, P, P, P, P]
    L.moe_set_stage_events.restype = I
    L.moe_set_stage_events.argtypes = [ctypes.POINTER(P), I]
    L.moe_ep_workspace_size.restype = Z
    L.moe_ep_workspace_size.argtypes = [I, I, I]
    L.moe_ep_plan.restype = I
    L.moe_ep_plan.argtypes = [P, I, I, I, I, P, P, P, P, Z, P]
    L.moe_ep_pack.restype = I
    L.moe_ep_pack.argtypes = [P, P, P] + [I] * 6 + [P, P, P, P]
    L.moe_fp8_expert_rows_workspace_size.restype = Z
    L.moe_fp8_expert_rows_workspace_size.argtypes = [I] * 4
    L.moe_fp8_expert_rows.restype = I
    L.moe_fp8_expert_rows.argtypes = [P, P, P, I, P, P, P, P, P, I, I, I, P, Z, P]
    L.moe_combine.restype = I
    L.moe_combine.argtypes = [P, P, P, I, I, I, P, P]
    L.moe_router_route.restype = I
    L.moe_router_route.argtypes = [P, I, I, I, P, P, P, P, P, P, Z, P]
    D = ctypes.c_double
    score = [P, I, P] + [I] * 8 + [F, P, P]
    L.moe_router_score_topk.restype = I
    L.moe_router_score_topk.argtypes = score + [P]
    L.moe_router_score_route.restype = I
    L.moe_router_score_route.argtypes = score + [P, P, P, P, Z, P]
    L.moe_rmsnorm_quant.restype = I
    L.moe_rmsnorm_quant.argtypes = [P, P, P, I, D, I, I, P, P, I, P, P, I, P]
    L.int8_quantize.restype = I
    L.int8_quantize.argtypes = [P, I, I, I, I, P, P, P, P]
    L.int8_moe_gemm.restype = I
    L.int8_moe_gemm.argtypes = [P] * 6 + [I] * 6 + [P]
    _lib = L
    return L


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status: int, where: str, check: bool) -> int:
    if check and status != MOE_OK:
        raise MoEError(status, where)
    return status


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def moe_set_wait_timeout_ns(ns: int) -> None:
    lib().moe_set_wait_timeout_ns(int(ns))


def moe_set_expert_fusion(mode: int) -> None:
    """MOE_FUSION_AUTO, MOE_FUSION_ON or MOE_FUSION_OFF (process-wide)."""
    _check(lib().moe_set_expert_fusion(int(mode)), "moe_set_expert_fusion", True)


def moe_fp8_fused_plan(T: int, H: int, I: int, E: int, k: int) -> dict:
    """Launch plan of moe_fp8_fused on the current device:
    {"tile_m1", "tile_m2", "fused"}."""
    a, b, c = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().moe_fp8_fused_plan(T, H, I, E, k, ctypes.byref(a), ctypes.byref(b),
                                    ctypes.byref(c)), "moe_fp8_fused_plan", True)
    return {"tile_m1": a.value, "tile_m2": b.value, "fused": bool(c.value)}


def moe_workspace_size(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(lib().moe_workspace_size(T, H, I, E, k))


def moe_route_workspace_size(T: int, k: int, E: int) -> int:
    return int(lib().moe_route_workspace_size(T, k, E))


def moe_select_tile_m(total_rows: int, n: int, k: int, E: int, num_sms: int, is_gated: bool):
    tm, tn = ctypes.c_int(0), ctypes.c_int(0)
    st = lib().moe_select_tile_m(total_rows, n, k, E, num_sms, int(bool(is_gated)),
                                 ctypes.byref(tm), ctypes.byref(tn))
    _check(st, "moe_select_tile_m", True)
    return tm.value, tn.value


def moe_route_permute(topk_ids, E: int, m_indptr, perm, inv_perm, ws, ws_bytes=None, *,
                      T=None, k=None, stream=None, check=True) -> int:
    if T is None or k is None:
        T, k = topk_ids.shape
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    st = lib().moe_route_permute(_ptr(topk_ids), T, k, E, _ptr(m_indptr), _ptr(perm),
                                 _ptr(inv_perm), _ptr(ws), ws_bytes, _stream(stream))
    return _check(st, "moe_route_permute", check)


def moe_router_route(logits, k: int, topk_ids, topk_w, m_indptr, perm, inv_perm, ws, ws_bytes=None,
                     *, dims=None, stream=None, check=True) -> int:
    """moe_router_topk + moe_route_permute in one call (one launch for up to
    8192 pairs); dims = (T, E) when raw addresses are passed."""
    T, E = dims if dims is not None else logits.shape
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    st = lib().moe_router_route(_ptr(logits), T, E, k, _ptr(topk_ids), _ptr(topk_w),
                                _ptr(m_indptr), _ptr(perm), _ptr(inv_perm), _ptr(ws), ws_bytes,
                                _stream(stream))
    return _check(st, "moe_router_route", check)


def moe_route_permute_noalloc(topk_ids, E: int, m_indptr, perm, inv_perm, *, T=None, k=None,
                              stream=None, check=True) -> int:
    """moe_route_permute without a workspace: the scratch is a device array
    inside the library, shared by every call (T*k <= 65536)."""
    if T is None or k is None:
        T, k = topk_ids.shape
    st = lib().moe_route_permute_noalloc(_ptr(topk_ids), T, k, E, _ptr(m_indptr), _ptr(perm),
                                         _ptr(inv_perm), _stream(stream))
    return _check(st, "moe_route_permute_noalloc", check)


def _fused_dims(x, topk_ids, w13):
    T, H = x.shape
    k = topk_ids.shape[1]
    E, I2, _ = w13.shape
    return T, H, I2 // 2, E, k


def moe_fp8_fused(x, topk_ids, topk_w, w13, w13_scale, w2, w2_scale, out, ws, ws_bytes=None, *,
                  dims=None, stream=None, check=True) -> int:
    """dims = (T, H, I, E, k) when raw addresses are passed."""
    T, H, I, E, k = dims if dims is not None else _fused_dims(x, topk_ids, w13)
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    st = lib().moe_fp8_fused(_ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(w13), _ptr(w13_scale),
                             _ptr(w2), _ptr(w2_scale), _ptr(out), T, H, I, E, k, _ptr(ws),
                             ws_bytes, _stream(stream))
    return _check(st, "moe_fp8_fused", check)


def moe_fp8_fused_debug(x, topk_ids, topk_w, w13, w13_scale, w2, w2_scale, out, ws,
                        m_indptr=None, perm=None, h_fp8=None, h_scale=None, ws_bytes=None, *,
                        dims=None, stream=None, check=True) -> int:
    T, H, I, E, k = dims if dims is not None else _fused_dims(x, topk_ids, w13)
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    st = lib().moe_fp8_fused_debug(_ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(w13),
                                   _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), _ptr(out), T, H, I,
                                   E, k, _ptr(ws), ws_bytes, _stream(stream), _ptr(m_indptr),
                                   _ptr(perm), _ptr(h_fp8), _ptr(h_scale))
    return _check(st, "moe_fp8_fused_debug", check)


def fp8_groupwise_moe_gemm(a, b, a_scale, b_scale, m_indptr, out, scale_major_mode="K",
                           scale_granularity=(1, 128, 128), is_gated=False, tile_m=-1, tile_n=-1,
                           *, dims=None, stream=None, check=True) -> int:
    """scale_major_mode "K": a_scale [R, K/128]; "MN": [K/128, R].
    dims = (R, N, K, E) when raw addresses are passed."""
    if dims is None:
        R, K = a.shape
        E, N, _ = b.shape
    else:
        R, N, K, E = dims
    mode = {"K": 0, "MN": 1}.get(scale_major_mode, scale_major_mode)
    sg_m, sg_n, sg_k = scale_granularity
    st = lib().fp8_groupwise_moe_gemm(_ptr(a), _ptr(b), _ptr(a_scale), _ptr(b_scale),
                                      _ptr(m_indptr), _ptr(out), R, N, K, E, mode, sg_m, sg_n,
                                      sg_k, int(bool(is_gated)), tile_m, tile_n, _stream(stream))
    return _check(st, "fp8_groupwise_moe_gemm", check)


def mxfp8_moe_gemm(a, b, a_sf, b_sf, m_indptr, out, is_gated=False, a_sf_major="K", *,
                   dims=None, stream=None, check=True) -> int:
    """a [R,K] fp8, b [E,N,K] fp8, a_sf [R,K/32] uint8 E8M0 row-major, b_sf the
    weight scales tiled by mxfp8_tile_scales, out bf16 [R, N/2 if gated else N].  dims = (R, N, K, E) when raw addresses
    are passed."""
    if dims is None:
        R, K = a.shape
        E, N, _ = b.shape
    else:
        R, N, K, E = dims
    mode = {"K": 0, "MN": 1}.get(a_sf_major, a_sf_major)
    st = lib().mxfp8_moe_gemm(_ptr(a), _ptr(b), _ptr(a_sf), _ptr(b_sf), _ptr(m_indptr), _ptr(out),
                              R, N, K, E, mode, int(bool(is_gated)), _stream(stream))
    return _check(st, "mxfp8_moe_gemm", check)


def moe_router_topk(logits, topk_ids, topk_w, *, dims=None, stream=None, check=True) -> int:
    """logits fp32 [T, E] -> topk_ids int32 [T, k], topk_w fp32 [T, k].
    dims = (T, E, k) when raw addresses are passed."""
    if dims is None:
        T, E = logits.shape
        k = topk_ids.shape[1]
    else:
        T, E, k = dims
    st = lib().moe_router_topk(_ptr(logits), T, E, k, _ptr(topk_ids), _ptr(topk_w), _stream(stream))
    return _check(st, "moe_router_topk", check)


def moe_mxfp8_fused(x, topk_ids, topk_w, w13, w13_sf, w2, w2_sf, out, ws, ws_bytes=None, *,
                    dims=None, stream=None, check=True) -> int:
    """w13_sf / w2_sf: weight scales tiled by mxfp8_tile_scales.  dims = (T, H, I, E, k)
    when raw addresses are passed."""
    T, H, I, E, k = dims if dims is not None else _fused_dims(x, topk_ids, w13)
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    st = lib().moe_mxfp8_fused(_ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(w13), _ptr(w13_sf),
                               _ptr(w2), _ptr(w2_sf), _ptr(out), T, H, I, E, k, _ptr(ws), ws_bytes,
                               _stream(stream))
    return _check(st, "moe_mxfp8_fused", check)


def moe_mxfp8_fused_debug(x, topk_ids, topk_w, w13, w13_sf, w2, w2_sf, out, ws, m_indptr=None,
                          perm=None, h_fp8=None, h_sf=None, ws_bytes=None, *, dims=None,
                          stream=None, check=True) -> int:
    T, H, I, E, k = dims if dims is not None else _fused_dims(x, topk_ids, w13)
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    st = lib().moe_mxfp8_fused_debug(_ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(w13),
                                     _ptr(w13_sf), _ptr(w2), _ptr(w2_sf), _ptr(out), T, H, I, E,
                                     k, _ptr(ws), ws_bytes, _stream(stream), _ptr(m_indptr),
                                     _ptr(perm), _ptr(h_fp8), _ptr(h_sf))
    return _check(st, "moe_mxfp8_fused_debug", check)


def mxfp8_tile_scales(sf_rowmajor, sf_tiled, *, dims=None, stream=None, check=True) -> int:
    """sf_rowmajor uint8 [rows, K/32] -> sf_tiled uint8 (rows * K/32 bytes, tiled).
    dims = (rows, K) when raw addresses are passed."""
    if dims is None:
        rows = sf_rowmajor.shape[0] if sf_rowmajor.dim() == 2 else sf_rowmajor.shape[0] * sf_rowmajor.shape[1]
        K = sf_rowmajor.shape[-1] * 32
    else:
        rows, K = dims
    st = lib().mxfp8_tile_scales(_ptr(sf_rowmajor), _ptr(sf_tiled), rows, K, _stream(stream))
    return _check(st, "mxfp8_tile_scales", check)


def nvfp4_moe_gemm(a, b, a_sf, b_sf, alpha, m_indptr, out, is_gated=False, a_sf_major="K", *,
                   dims=None, stream=None, check=True) -> int:
    """a uint8 [R, K/2] packed E2M1, b uint8 [E, N, K/2], a_sf uint8 E4M3
    [R, K/16] ("K") or [K/64, R, 4] ("MN"), b_sf the weight scales tiled by
    nvfp4_tile_scales, alpha fp32 [E], out bf16 [R, N/2 if gated else N].
    dims = (R, N, K, E) when raw addresses are passed."""
    if dims is None:
        R = a.shape[0]
        K = a.shape[1] * 2
        E, N = b.shape[0], b.shape[1]
    else:
        R, N, K, E = dims
    mode = {"K": 0, "MN": 1}.get(a_sf_major, a_sf_major)
    st = lib().nvfp4_moe_gemm(_ptr(a), _ptr(b), _ptr(a_sf), _ptr(b_sf), _ptr(alpha), _ptr(m_indptr),
                              _ptr(out), R, N, K, E, mode, int(bool(is_gated)), _stream(stream))
    return _check(st, "nvfp4_moe_gemm", check)


def moe_tactic_tune_gemm(a, b, a_scale, b_scale, m_indptr, out, scale_major="K",
                         is_gated=False, iters=5, *, dims=None, stream=None) -> int:
    """Times fp8_groupwise_moe_gemm at every tile_m valid for K on these
    buffers (out is overwritten), stores the fastest in the tactic table and
    returns it.  dims = (R, N, K, E) when raw addresses are passed."""
    if dims is None:
        R, K = a.shape
        E, N, _ = b.shape
    else:
        R, N, K, E = dims
    mode = {"K": 0, "MN": 1}.get(scale_major, scale_major)
    tm = ctypes.c_int(0)
    st = lib().moe_tactic_tune_gemm(_ptr(a), _ptr(b), _ptr(a_scale), _ptr(b_scale), _ptr(m_indptr),
                                    _ptr(out), R, N, K, E, mode, int(bool(is_gated)), int(iters),
                                    _stream(stream), ctypes.byref(tm))
    _check(st, "moe_tactic_tune_gemm", True)
    return tm.value


def moe_tactic_lookup(R, N, K, E, is_gated=False):
    """Stored tile_m of the shape class, or None (host only)."""
    tm = ctypes.c_int(0)
    st = lib().moe_tactic_lookup(R, N, K, E, int(bool(is_gated)), ctypes.byref(tm))
    if st == MOE_ERR_NO_TILE_CONFIG:
        return None
    _check(st, "moe_tactic_lookup", True)
    return tm.value


def moe_tactic_store(R, N, K, E, is_gated, tile_m, *, check=True) -> int:
    """Sets the shape class's tile_m (host only)."""
    return _check(lib().moe_tactic_store(R, N, K, E, int(bool(is_gated)), tile_m),
                  "moe_tactic_store", check)


def moe_tactic_clear() -> None:
    lib().moe_tactic_clear()


def nvfp4_quantize(x, gscale, q, sf, *, dims=None, stream=None, check=True) -> int:
    """x bf16 [M, K] -> q uint8 [M, K/2] packed E2M1, sf uint8 [M, K/16] E4M3.
    dims = (M, K) when raw addresses are passed."""
    M, K = dims if dims is not None else x.shape
    st = lib().nvfp4_quantize(_ptr(x), float(gscale), _ptr(q), _ptr(sf), M, K, _stream(stream))
    return _check(st, "nvfp4_quantize", check)


def _nv_fused_dims(x, topk_ids, w13):
    T, H = x.shape
    return T, H, w13.shape[1] // 2, w13.shape[0], topk_ids.shape[1]


def moe_nvfp4_fused(x, topk_ids, topk_w, w13, w13_sf, w13_alpha, w2, w2_sf, w2_alpha, a1_gscale,
                    a2_gscale, out, ws, ws_bytes=None, *, dims=None, stream=None,
                    check=True) -> int:
    """w13 / w2 packed E2M1 [E, 2I, H/2] / [E, H, I/2]; w13_sf / w2_sf tiled by
    nvfp4_tile_scales; *_alpha fp32 [E]; a1_gscale / a2_gscale floats.
    dims = (T, H, I, E, k) when raw addresses are passed."""
    T, H, I, E, k = dims if dims is not None else _nv_fused_dims(x, topk_ids, w13)
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    st = lib().moe_nvfp4_fused(_ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(w13), _ptr(w13_sf),
                               _ptr(w13_alpha), _ptr(w2), _ptr(w2_sf), _ptr(w2_alpha),
                               float(a1_gscale), float(a2_gscale), _ptr(out), T, H, I, E, k,
                               _ptr(ws), ws_bytes, _stream(stream))
    return _check(st, "moe_nvfp4_fused", check)


def moe_nvfp4_fused_debug(x, topk_ids, topk_w, w13, w13_sf, w13_alpha, w2, w2_sf, w2_alpha,
                          a1_gscale, a2_gscale, out, ws, m_indptr=None, perm=None, h_fp4=None,
                          h_sf=None, ws_bytes=None, *, dims=None, stream=None, check=True) -> int:
    T, H, I, E, k = dims if dims is not None else _nv_fused_dims(x, topk_ids, w13)
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    st = lib().moe_nvfp4_fused_debug(_ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(w13),
                                     _ptr(w13_sf), _ptr(w13_alpha), _ptr(w2), _ptr(w2_sf),
                                     _ptr(w2_alpha), float(a1_gscale), float(a2_gscale),
                                     _ptr(out), T, H, I, E, k, _ptr(ws), ws_bytes,
                                     _stream(stream), _ptr(m_indptr), _ptr(perm), _ptr(h_fp4),
                                     _ptr(h_sf))
    return _check(st, "moe_nvfp4_fused_debug", check)


def nvfp4_tile_scales(sf_rowmajor, sf_tiled, *, dims=None, stream=None, check=True) -> int:
    """sf_rowmajor uint8 [rows, K/16] E4M3 -> sf_tiled uint8 (rows * K/16 bytes, tiled).
    dims = (rows, K) when raw addresses are passed."""
    if dims is None:
        rows = sf_rowmajor.numel() // sf_rowmajor.shape[-1]
        K = sf_rowmajor.shape[-1] * 16
    else:
        rows, K = dims
    st = lib().nvfp4_tile_scales(_ptr(sf_rowmajor), _ptr(sf_tiled), rows, K, _stream(stream))
    return _check(st, "nvfp4_tile_scales", check)


def swiglu_mxfp8_quant(inp, out, scale, *, dims=None, stream=None, check=True) -> int:
    if dims is None:
        M, K2 = inp.shape
        K = K2 // 2
    else:
        M, K = dims
    st = lib().swiglu_mxfp8_quant(_ptr(inp), _ptr(out), _ptr(scale), M, K, _stream(stream))
    return _check(st, "swiglu_mxfp8_quant", check)


def moe_set_stage_events(events) -> int:
    """events: six torch.cuda.Event (timing enabled, already created on the
    device; None entries are not recorded) or None to switch stage timing off."""
    if events is None:
        return _check(lib().moe_set_stage_events(None, 0), "moe_set_stage_events", True)
    handles = (ctypes.c_void_p * len(events))(
        *[ctypes.c_void_p(e.cuda_event if e is not None else None) for e in events])
    return _check(lib().moe_set_stage_events(handles, len(events)), "moe_set_stage_events", True)


def moe_get_device_status(ws=None, *, stream=None) -> int:
    return int(lib().moe_get_device_status(_ptr(ws), _stream(stream)))


# ---------------------------------------------------------------- scored router, norm, int8
# These calls are a few microseconds of GPU work at decoding sizes, so their
# marshalling is kept short: tensors are checked by identity, and only a call
# that fails the short check goes through the one that says what is wrong.
_SCORING = {"softmax": 0, "sigmoid": 1}
_Q_FORMAT = {"none": 0, "fp8": 1, "mxfp8": 2, "int8": 3}
_MAJOR = {"K": 0, "MN": 1}
_DTYPE = {"float32": 0, "bfloat16": 1}


class _Torch:
    """What the checks need of torch, looked up once (on the first call that
    passes tensors)."""

    def __init__(self):
        import torch
        self.f32, self.bf16, self.i32 = torch.float32, torch.bfloat16, torch.int32
        self.i8, self.u8 = torch.int8, torch.uint8
        self.float = (torch.float32, torch.bfloat16)
        self.e4m3 = (torch.float8_e4m3fn, torch.uint8)
        self.e8m0 = (torch.uint8, torch.float8_e8m0fnu)
        self.code = {self.f32: 0, self.bf16: 1}
        self.current_device = torch.cuda.current_device
        self.on_device = torch.cuda.device
        # the current stream's handle without building a Stream object (3 us);
        # the public way where this torch lacks it
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda dev: torch.cuda.current_stream(dev).cuda_stream)


_tc = None


def _torch():
    global _tc
    if _tc is None:
        _tc = _Torch()
    return _tc


def _is(t, dtype, shape, dev):
    """A contiguous tensor of this dtype, shape and device."""
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev


def _tensors(where, dev, *specs):
    """Checks tensors against (name, tensor, dtype or dtypes, shape or None):
    raises ValueError for one that the C entry would misread.  None passes."""
    for name, t, dtype, shape in specs:
        if t is None:
            continue
        ok = t.dtype in dtype if dtype.__class__ is tuple else t.dtype is dtype
        if not ok:
            raise ValueError(f"{where}: {name} is {t.dtype}, expected {dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} is not contiguous")
        if t.get_device() != dev:
            raise ValueError(f"{where}: {name} is on {t.device}, expected CUDA device {dev}")


def _addr(t):
    return t if t is None or t.__class__ is int else t.data_ptr()


def _call(where, fn, args, dev, stream, check):
    """fn(*args, stream) with device `dev` current (None: whichever is)."""
    if dev is None:
        st = fn(*args, _stream(stream))
    elif dev < 0:
        raise ValueError(f"{where}: tensors are not on a CUDA device")
    elif dev == _tc.current_device():
        st = fn(*args, _tc.raw_stream(dev) if stream is None else _stream(stream))
    else:
        with _tc.on_device(dev):
            st = fn(*args, _tc.raw_stream(dev) if stream is None else _stream(stream))
    if check and st != MOE_OK:
        raise MoEError(st, where)
    return st


def _score_check(where, tc, logits, topk_ids, topk_w, bias, T, E, k, dev):
    if not (logits.dtype in tc.float and logits.is_contiguous() and _is(topk_ids, tc.i32, (T, k), dev)
            and _is(topk_w, tc.f32, (T, k), dev) and (bias is None or _is(bias, tc.f32, (E,), dev))):
        _tensors(where, dev, ("logits", logits, tc.float, None), ("topk_ids", topk_ids, tc.i32, (T, k)),
                 ("topk_w", topk_w, tc.f32, (T, k)), ("bias", bias, tc.f32, (E,)))


def moe_router_score_topk(logits, topk_ids, topk_w, *, bias=None, scoring="softmax", n_group=1,
                          topk_group=1, group_top=1, renorm=True, scale=1.0, dims=None,
                          logits_dtype="float32", stream=None, check=True) -> int:
    """logits fp32 or bf16 [T, E], bias fp32 [E] or None -> topk_ids int32
    [T, k], topk_w fp32 [T, k].  scoring "softmax" or "sigmoid".
    dims = (T, E, k) and logits_dtype when raw addresses are passed."""
    where = "moe_router_score_topk"
    if dims is None:
        tc = _tc or _torch()
        T, E = logits.shape
        k = topk_ids.shape[1]
        dev = logits.get_device()
        _score_check(where, tc, logits, topk_ids, topk_w, bias, T, E, k, dev)
        dtype = tc.code[logits.dtype]
    else:
        T, E, k = dims
        dev, dtype = None, _DTYPE.get(logits_dtype, logits_dtype)
    a = (_addr(logits), dtype, _addr(bias), T, E, k, _SCORING.get(scoring, scoring), n_group, topk_group,
         group_top, 1 if renorm else 0, scale, _addr(topk_ids), _addr(topk_w))
    return _call(where, (_lib or lib()).moe_router_score_topk, a, dev, stream, check)


def moe_router_score_route(logits, topk_ids, topk_w, m_indptr, perm, inv_perm, ws, ws_bytes=None, *,
                           bias=None, scoring="softmax", n_group=1, topk_group=1, group_top=1,
                           renorm=True, scale=1.0, dims=None, logits_dtype="float32", stream=None,
                           check=True) -> int:
    """moe_router_score_topk + moe_route_permute in one call.
    dims = (T, E, k) and logits_dtype when raw addresses are passed."""
    where = "moe_router_score_route"
    if dims is None:
        tc = _tc or _torch()
        T, E = logits.shape
        k = topk_ids.shape[1]
        dev = logits.get_device()
        _score_check(where, tc, logits, topk_ids, topk_w, bias, T, E, k, dev)
        if not (_is(m_indptr, tc.i32, (E + 1,), dev) and _is(perm, tc.i32, (T * k,), dev)
                and (inv_perm is None or _is(inv_perm, tc.i32, (T * k,), dev))
                and ws.dtype is tc.u8 and ws.is_contiguous() and ws.get_device() == dev):
            _tensors(where, dev, ("m_indptr", m_indptr, tc.i32, (E + 1,)), ("perm", perm, tc.i32, (T * k,)),
                     ("inv_perm", inv_perm, tc.i32, (T * k,)), ("ws", ws, tc.u8, None))
        dtype = tc.code[logits.dtype]
    else:
        T, E, k = dims
        dev, dtype = None, _DTYPE.get(logits_dtype, logits_dtype)
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    a = (_addr(logits), dtype, _addr(bias), T, E, k, _SCORING.get(scoring, scoring), n_group, topk_group,
         group_top, 1 if renorm else 0, scale, _addr(topk_ids), _addr(topk_w), _addr(m_indptr), _addr(perm),
         _addr(inv_perm), _addr(ws), ws_bytes)
    return _call(where, (_lib or lib()).moe_router_score_route, a, dev, stream, check)


def moe_rmsnorm_quant(x, weight, eps, *, residual=None, residual_out=None, y=None, q_format="none",
                      q=None, q_scale=None, scale_major="K", dims=None, weight_dtype="float32",
                      stream=None, check=True) -> int:
    """x bf16 [T, H], weight fp32 or bf16 [H], residual / residual_out / y bf16
    [T, H] or None.  q_format "none", "fp8" (q [T, H] 8-bit, q_scale fp32
    [T, H/128] or, with scale_major "MN", [H/128, T]), "mxfp8" (q_scale uint8
    [T, H/32] or [H/128, T, 4]) or "int8" (q int8 [T, H], q_scale fp32 [T]).
    dims = (T, H) and weight_dtype when raw addresses are passed."""
    where = "moe_rmsnorm_quant"
    fmt, mn = _Q_FORMAT.get(q_format, q_format), _MAJOR.get(scale_major, scale_major)
    if dims is None:
        tc = _tc or _torch()
        shape = x.shape
        T, H = shape
        dev = x.get_device()
        bf16 = tc.bf16
        if not (x.dtype is bf16 and x.is_contiguous()
                and (residual is None or _is(residual, bf16, shape, dev))
                and weight.dtype in tc.float and _is(weight, weight.dtype, (H,), dev)
                and (residual_out is None or _is(residual_out, bf16, shape, dev))
                and (y is None or _is(y, bf16, shape, dev))):
            _tensors(where, dev, ("x", x, bf16, None), ("residual", residual, bf16, shape),
                     ("weight", weight, tc.float, (H,)), ("residual_out", residual_out, bf16, shape),
                     ("y", y, bf16, shape))
        if fmt == 1:
            _tensors(where, dev, ("q", q, tc.e4m3, shape),
                     ("q_scale", q_scale, tc.f32, (H // 128, T) if mn == 1 else (T, H // 128)))
        elif fmt == 2:
            _tensors(where, dev, ("q", q, tc.e4m3, shape),
                     ("q_scale", q_scale, tc.e8m0, (H // 128, T, 4) if mn == 1 else (T, H // 32)))
        elif fmt == 3:
            _tensors(where, dev, ("q", q, tc.i8, shape), ("q_scale", q_scale, tc.f32, (T,)))
        wd = tc.code[weight.dtype]
    else:
        T, H = dims
        dev, wd = None, _DTYPE.get(weight_dtype, weight_dtype)
    a = (_addr(x), _addr(residual), _addr(weight), wd, eps, T, H, _addr(residual_out), _addr(y), fmt,
         _addr(q), _addr(q_scale), mn)
    return _call(where, (_lib or lib()).moe_rmsnorm_quant, a, dev, stream, check)


def int8_quantize(x, q, q_scale, *, inv_perm=None, k=1, dims=None, stream=None, check=True) -> int:
    """x bf16 [T, K] -> q int8 [R, K], q_scale fp32 [R]; row t goes to the rows
    inv_perm[t*k : (t+1)*k] (row t without inv_perm).  dims = (T, K, R) when
    raw addresses are passed."""
    where = "int8_quantize"
    if dims is None:
        tc = _tc or _torch()
        T, K = x.shape
        R = q.shape[0]
        dev = x.get_device()
        if not (x.dtype is tc.bf16 and x.is_contiguous() and _is(q, tc.i8, (R, K), dev)
                and _is(q_scale, tc.f32, (R,), dev)
                and (inv_perm is None or _is(inv_perm, tc.i32, (T * k,), dev))):
            _tensors(where, dev, ("x", x, tc.bf16, None), ("q", q, tc.i8, (R, K)),
                     ("q_scale", q_scale, tc.f32, (R,)), ("inv_perm", inv_perm, tc.i32, (T * k,)))
    else:
        T, K, R = dims
        dev = None
    a = (_addr(x), T, K, k, R, _addr(inv_perm), _addr(q), _addr(q_scale))
    return _call(where, (_lib or lib()).int8_quantize, a, dev, stream, check)


def int8_moe_gemm(a, b, a_scale, b_scale, out, *, m_indptr=None, is_gated=False, dims=None,
                  out_dtype="bfloat16", stream=None, check=True) -> int:
    """a int8 [R, K], b int8 [E, N, K] (or [N, K]: one expert), a_scale fp32
    [R], b_scale fp32 [E, N] (or [N]), m_indptr int32 [E+1] or None (one
    expert, all rows), out bf16 or fp32 [R, N/2 if gated else N].
    dims = (R, N, K, E) and out_dtype when raw addresses are passed."""
    where = "int8_moe_gemm"
    if dims is None:
        tc = _tc or _torch()
        R, K = a.shape
        bs = b.shape
        if len(bs) != 2 and len(bs) != 3:
            raise ValueError(f"{where}: b has shape {tuple(bs)}, expected [E, N, K] or [N, K]")
        E, N = (bs[0], bs[1]) if len(bs) == 3 else (1, bs[0])
        dev = a.get_device()
        n_out = N // 2 if is_gated else N
        s_shape = (N,) if E == 1 and b_scale.dim() == 1 else (E, N)
        if not (a.dtype is tc.i8 and a.is_contiguous() and bs[-1] == K and _is(b, tc.i8, bs, dev)
                and _is(a_scale, tc.f32, (R,), dev) and _is(b_scale, tc.f32, s_shape, dev)
                and (m_indptr is None or _is(m_indptr, tc.i32, (E + 1,), dev))
                and out.dtype in tc.float and _is(out, out.dtype, (R, n_out), dev)):
            _tensors(where, dev, ("a", a, tc.i8, None),
                     ("b", b, tc.i8, (E, N, K) if len(bs) == 3 else (N, K)),
                     ("a_scale", a_scale, tc.f32, (R,)), ("b_scale", b_scale, tc.f32, s_shape),
                     ("m_indptr", m_indptr, tc.i32, (E + 1,)), ("out", out, tc.float, (R, n_out)))
        od = tc.code[out.dtype]
    else:
        R, N, K, E = dims
        dev, od = None, _DTYPE.get(out_dtype, out_dtype)
    args = (_addr(a), _addr(b), _addr(a_scale), _addr(b_scale), _addr(m_indptr), _addr(out), od, R, N, K,
            E, 1 if is_gated else 0)
    return _call(where, (_lib or lib()).int8_moe_gemm, args, dev, stream, check)


# ---------------------------------------------------------------- expert parallelism
def moe_ep_workspace_size(T: int, k: int, G: int) -> int:
    return int(lib().moe_ep_workspace_size(T, k, G))


def moe_ep_plan(topk_ids, E: int, G: int, send_indptr, send_pair, slot_of_pair, ws, ws_bytes=None,
                *, T=None, k=None, stream=None, check=True) -> int:
    if T is None or k is None:
        T, k = topk_ids.shape
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    st = lib().moe_ep_plan(_ptr(topk_ids), T, k, E, G, _ptr(send_indptr), _ptr(send_pair),
                           _ptr(slot_of_pair), _ptr(ws), ws_bytes, _stream(stream))
    return _check(st, "moe_ep_plan", check)


def moe_ep_pack(x, topk_ids, slot_of_pair, E: int, G: int, S: int, xq_send, xs_send, eid_send, *,
                dims=None, stream=None, check=True) -> int:
    """dims = (T, H, k) when raw addresses are passed."""
    if dims is None:
        T, H = x.shape
        k = topk_ids.shape[1]
    else:
        T, H, k = dims
    st = lib().moe_ep_pack(_ptr(x), _ptr(topk_ids), _ptr(slot_of_pair), T, H, k, E, G, S,
                           _ptr(xq_send), _ptr(xs_send), _ptr(eid_send), _stream(stream))
    return _check(st, "moe_ep_pack", check)


def moe_fp8_expert_rows_workspace_size(n: int, H: int, I: int, E: int) -> int:
    return int(lib().moe_fp8_expert_rows_workspace_size(n, H, I, E))


def moe_fp8_expert_rows(xq, xs, eid, w13, w13_scale, w2, w2_scale, y, ws, ws_bytes=None, *,
                        dims=None, stream=None, check=True) -> int:
    """dims = (n, H, I, E) when raw addresses are passed."""
    if dims is None:
        n, H = xq.shape
        E, I2, _ = w13.shape
        I = I2 // 2
    else:
        n, H, I, E = dims
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    st = lib().moe_fp8_expert_rows(_ptr(xq), _ptr(xs), _ptr(eid), n, _ptr(w13), _ptr(w13_scale),
                                   _ptr(w2), _ptr(w2_scale), _ptr(y), H, I, E, _ptr(ws), ws_bytes,
                                   _stream(stream))
    return _check(st, "moe_fp8_expert_rows", check)


def moe_combine(y, row_of_pair, topk_w, out, *, dims=None, stream=None, check=True) -> int:
    """dims = (T, k, H) when raw addresses are passed."""
    if dims is None:
        T, k = topk_w.shape
        H = out.shape[1]
    else:
        T, k, H = dims
    st = lib().moe_combine(_ptr(y), _ptr(row_of_pair), _ptr(topk_w), T, k, H, _ptr(out),
                           _stream(stream))
    return _check(st, "moe_combine", check)
