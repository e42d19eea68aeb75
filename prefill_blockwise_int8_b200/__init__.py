"""Tile-routed FP16/INT8 causal prefill attention on B200 (sm_100a).

Thin Python binding of the C ABI in ``include/tilemix.h`` (``libtilemix.so``,
built in-tree by ``python -m prefill_blockwise_int8_b200.build``).  This
module only marshals arguments: it takes torch tensors that already live on
the GPU, passes their device pointers and the current CUDA stream, and
raises ``TilemixError`` when a call returns a non-OK status.  Every step of
the computation runs in the library's CUDA kernels; there is no CPU or
PyTorch fallback, and importing this package fails loudly when the library
is missing.

Entry points (same names as the C ABI):
  tilemix_quantize_blockwise(x, cu_seqlens, max_seqlen, block=128)
      -> (x8, scale)
  tilemix_quantize_blockwise_qk(q, k, cu_seqlens, max_seqlen) (one launch)
      -> (q8, q_scale, k8, k_scale)
  tilemix_pack_mask(route, cu_seqlens, max_seqlen, block_m, block_n, group)
      -> mask
  tilemix_attn_prefill(q, k, v, cu_seqlens, max_seqlen, ...) -> out
  tilemix_rope_frequencies(rot_dim, base, ...) -> (freqs, attn_factor)
  tilemix_rope(q, k, positions, freqs, ...) -> (q_out, k_out)
  tilemix_paged_append(k, v, page_table, cu_seqlens, kv_lens, k_pages,
      v_pages, ...) -> rotated q or None
  tilemix_attn_paged(q, k_pages, v_pages, page_table, cu_seqlens, kv_lens,
      max_q_len, max_kv_len, ...) -> out
"""
from __future__ import annotations

import ctypes as C
import functools
import struct as _struct
from pathlib import Path

__all__ = [
    "TilemixError", "lib", "library_path", "EXPORTED_SYMBOLS",
    "tilemix_quantize_blockwise", "tilemix_quantize_blockwise_qk",
    "tilemix_pack_mask", "tilemix_attn_prefill",
    "tilemix_route_template", "tilemix_route_adaptive",
    "tilemix_route_adaptive_workspace_bytes", "tilemix_route_adaptive_noalloc",
    "ROUTE_ADAPTIVE_STATIC_BYTES", "tilemix_status_string",
    "tilemix_last_error", "tilemix_version", "KV_FP16", "KV_INT8", "FLAG_FP16_ONLY",
    "FLAG_QUANT_ON_CHIP", "FLAG_TEST_EXPIRE_WAIT", "FLAG_PV_F16_ACC", "STATUS",
    "LAYOUTS", "tilemix_rope_frequencies", "tilemix_rope",
    "tilemix_paged_append", "tilemix_attn_paged",
    "tilemix_attn_paged_workspace_bytes", "ROPE_LAYOUTS", "ROPE_SCALINGS",
]

_LIB_PATH = Path(__file__).resolve().parent / "libtilemix.so"

KV_FP16, KV_INT8 = 0, 1
FLAG_FP16_ONLY = 1
FLAG_QUANT_ON_CHIP = 2
FLAG_TEST_EXPIRE_WAIT = 4  # test only: makes a bounded device wait expire
FLAG_PV_F16_ACC = 8  # study only: O accumulated in fp16 (no tolerance)
STATUS = {0: "TILEMIX_OK", 1: "TILEMIX_ERR_INVALID_ARG",
          2: "TILEMIX_ERR_UNSUPPORTED", 3: "TILEMIX_ERR_CUDA",
          4: "TILEMIX_ERR_TIMEOUT", 5: "TILEMIX_ERR_BAD_SEQLENS",
          6: "TILEMIX_ERR_NO_DEVICE", 7: "TILEMIX_ERR_BAD_PAGES"}

# Routing-template layouts (TILEMIX_LAYOUT_*).
LAYOUTS = {"all_fp16": 0, "all_int8": 1, "band": 2, "global": 3,
           "row_random": 4, "aligned": 5, "bigbird": 6, "sptrans": 7}

# Rotary pair layouts (TILEMIX_ROPE_*) and frequency scalings
# (TILEMIX_ROPE_SCALE_*).
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "wavelength": 3, "yarn": 4}

# Every function include/tilemix.h declares.
EXPORTED_SYMBOLS = (
    "tilemix_quantize_blockwise", "tilemix_quantize_blockwise_qk",
    "tilemix_pack_mask", "tilemix_attn_prefill",
    "tilemix_route_template", "tilemix_route_adaptive_workspace_bytes",
    "tilemix_route_adaptive", "tilemix_route_adaptive_noalloc",
    "tilemix_rope_frequencies", "tilemix_rope", "tilemix_paged_append",
    "tilemix_attn_paged_workspace_bytes", "tilemix_attn_paged",
    "tilemix_status_string", "tilemix_last_error", "tilemix_version",
)

# TILEMIX_ROUTE_ADAPTIVE_STATIC_BYTES: the static scratch of
# tilemix_route_adaptive_noalloc on each device.
ROUTE_ADAPTIVE_STATIC_BYTES = 32 << 20


class TilemixError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {detail}")
        self.status = status


class AttnParams(C.Structure):
    """Mirror of tilemix_attn_params (include/tilemix.h)."""
    _fields_ = [
        ("struct_size", C.c_uint32), ("kv_format", C.c_int),
        ("flags", C.c_uint32),
        ("q", C.c_void_p), ("q8", C.c_void_p), ("q_scale", C.c_void_p),
        ("k", C.c_void_p), ("k8", C.c_void_p), ("k_scale", C.c_void_p),
        ("v", C.c_void_p), ("v8", C.c_void_p), ("v_scale", C.c_void_p),
        ("cu_seqlens", C.c_void_p), ("batch", C.c_int),
        ("max_seqlen", C.c_int), ("total_tokens", C.c_int),
        ("hq", C.c_int), ("hkv", C.c_int), ("head_dim", C.c_int),
        ("head_map", C.c_void_p),
        ("mask", C.c_void_p), ("block_m", C.c_int), ("block_n", C.c_int),
        ("group", C.c_int),
        ("quant_block_q", C.c_int), ("quant_block_k", C.c_int),
        ("softmax_scale", C.c_float), ("causal", C.c_int),
        ("out", C.c_void_p), ("lse", C.c_void_p), ("qk_dump", C.c_void_p),
        ("status", C.c_void_p),
    ]


class RopeParams(C.Structure):
    """Mirror of tilemix_rope_params (include/tilemix.h)."""
    _fields_ = [
        ("struct_size", C.c_uint32), ("dtype", C.c_int), ("layout", C.c_int),
        ("inverse", C.c_int),
        ("q", C.c_void_p), ("k", C.c_void_p), ("q_out", C.c_void_p),
        ("k_out", C.c_void_p),
        ("q_stride_t", C.c_int64), ("q_stride_h", C.c_int64),
        ("k_stride_t", C.c_int64), ("k_stride_h", C.c_int64),
        ("q_out_stride_t", C.c_int64), ("q_out_stride_h", C.c_int64),
        ("k_out_stride_t", C.c_int64), ("k_out_stride_h", C.c_int64),
        ("positions", C.c_void_p), ("freqs", C.c_void_p),
        ("attn_factor", C.c_float), ("total_tokens", C.c_int),
        ("hq", C.c_int), ("hkv", C.c_int), ("head_dim", C.c_int),
        ("rot_dim", C.c_int),
    ]


class AppendParams(C.Structure):
    """Mirror of tilemix_append_params (include/tilemix.h)."""
    _fields_ = [
        ("struct_size", C.c_uint32), ("dtype", C.c_int),
        ("kv_format", C.c_int), ("layout", C.c_int),
        ("k", C.c_void_p), ("v", C.c_void_p), ("q", C.c_void_p),
        ("q_out", C.c_void_p),
        ("k_stride_t", C.c_int64), ("k_stride_h", C.c_int64),
        ("v_stride_t", C.c_int64), ("v_stride_h", C.c_int64),
        ("q_stride_t", C.c_int64), ("q_stride_h", C.c_int64),
        ("q_out_stride_t", C.c_int64), ("q_out_stride_h", C.c_int64),
        ("positions", C.c_void_p), ("freqs", C.c_void_p),
        ("k_pages", C.c_void_p), ("v_pages", C.c_void_p),
        ("page_stride", C.c_int64), ("token_stride", C.c_int64),
        ("head_stride", C.c_int64),
        ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
        ("page_table", C.c_void_p), ("table_stride", C.c_int64),
        ("cu_seqlens", C.c_void_p), ("kv_lens", C.c_void_p),
        ("batch", C.c_int), ("total_tokens", C.c_int), ("hq", C.c_int),
        ("hkv", C.c_int), ("head_dim", C.c_int), ("rot_dim", C.c_int),
        ("num_pages", C.c_int), ("page_size", C.c_int),
        ("max_pages", C.c_int), ("attn_factor", C.c_float),
        ("status", C.c_void_p),
    ]


class AttnPagedParams(C.Structure):
    """Mirror of tilemix_attn_paged_params (include/tilemix.h)."""
    _fields_ = [
        ("struct_size", C.c_uint32), ("dtype", C.c_int),
        ("kv_format", C.c_int), ("causal", C.c_int),
        ("q", C.c_void_p), ("q_stride_t", C.c_int64),
        ("q_stride_h", C.c_int64),
        ("k_pages", C.c_void_p), ("v_pages", C.c_void_p),
        ("page_stride", C.c_int64), ("token_stride", C.c_int64),
        ("head_stride", C.c_int64),
        ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
        ("page_table", C.c_void_p), ("table_stride", C.c_int64),
        ("cu_seqlens", C.c_void_p), ("kv_lens", C.c_void_p),
        ("batch", C.c_int), ("total_tokens", C.c_int),
        ("max_q_len", C.c_int), ("max_kv_len", C.c_int),
        ("hq", C.c_int), ("hkv", C.c_int), ("head_dim", C.c_int),
        ("num_pages", C.c_int), ("page_size", C.c_int),
        ("max_pages", C.c_int), ("softmax_scale", C.c_float),
        ("flags", C.c_uint32), ("out", C.c_void_p), ("lse", C.c_void_p), ("workspace", C.c_void_p),
        ("workspace_bytes", C.c_size_t), ("status", C.c_void_p),
    ]


def library_path() -> Path:
    return _LIB_PATH


def _load() -> C.CDLL:
    if not _LIB_PATH.exists():
        raise ImportError(
            f"{_LIB_PATH} is missing: build the CUDA library with "
            "`python -m prefill_blockwise_int8_b200.build` (nvcc, sm_100a)")
    lib = C.CDLL(str(_LIB_PATH))
    vp, i32 = C.c_void_p, C.c_int
    lib.tilemix_quantize_blockwise.restype = i32
    lib.tilemix_quantize_blockwise.argtypes = [
        vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp]
    lib.tilemix_quantize_blockwise_qk.restype = i32
    lib.tilemix_quantize_blockwise_qk.argtypes = [
        vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp,
        vp, vp]
    lib.tilemix_pack_mask.restype = i32
    lib.tilemix_pack_mask.argtypes = [
        vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp]
    lib.tilemix_route_template.restype = i32
    lib.tilemix_route_template.argtypes = [
        i32, i32, C.c_uint64, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp]
    lib.tilemix_route_adaptive_workspace_bytes.restype = C.c_size_t
    lib.tilemix_route_adaptive_workspace_bytes.argtypes = [i32] * 5
    lib.tilemix_route_adaptive.restype = i32
    lib.tilemix_route_adaptive.argtypes = [
        vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, i32, i32, i32, i32, vp,
        C.c_size_t, vp, vp, vp, vp]
    lib.tilemix_route_adaptive_noalloc.restype = i32
    lib.tilemix_route_adaptive_noalloc.argtypes = [
        vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, i32, i32, i32, i32, vp,
        vp, vp, vp]
    lib.tilemix_attn_prefill.restype = i32
    lib.tilemix_attn_prefill.argtypes = [C.POINTER(AttnParams), vp]
    lib.tilemix_rope_frequencies.restype = i32
    lib.tilemix_rope_frequencies.argtypes = [
        i32, i32, C.c_double, C.c_double, C.c_double, C.c_double, i32,
        C.POINTER(C.c_double), C.POINTER(C.c_float)]
    lib.tilemix_rope.restype = i32
    lib.tilemix_rope.argtypes = [vp, vp]  # packed parameter structs
    lib.tilemix_paged_append.restype = i32
    lib.tilemix_paged_append.argtypes = [vp, vp]
    lib.tilemix_attn_paged_workspace_bytes.restype = C.c_size_t
    lib.tilemix_attn_paged_workspace_bytes.argtypes = [i32] * 4
    lib.tilemix_attn_paged.restype = i32
    lib.tilemix_attn_paged.argtypes = [vp, vp]
    lib.tilemix_status_string.restype = C.c_char_p
    lib.tilemix_status_string.argtypes = [i32]
    lib.tilemix_last_error.restype = C.c_char_p
    lib.tilemix_last_error.argtypes = []
    lib.tilemix_version.restype = C.c_uint32
    lib.tilemix_version.argtypes = []
    return lib


class _Missing:
    """Stands in for the library when it is missing or older than the
    sources (so the package imports for a build); any use raises."""

    def __init__(self, err: Exception):
        self._err = err

    def __getattr__(self, name):
        raise ImportError(f"libtilemix.so unusable ({self._err}); build it "
                          "with `python -m prefill_blockwise_int8_b200.build`")


class _Lazy:
    """The library, mapped into the process on the first attribute access
    (importing the package, or its host-side helpers such as ``roofline``,
    maps nothing).  A missing or unusable library raises at that access."""

    def __init__(self):
        self._lib = None

    def __getattr__(self, name):
        if self._lib is None:
            try:
                self._lib = _load()
            except (OSError, AttributeError, ImportError) as e:
                self._lib = _Missing(e)
        fn = getattr(self._lib, name)
        self.__dict__[name] = fn  # the next access is a plain attribute's
        return fn


lib = _Lazy()


def reload_library():
    """Load libtilemix.so now (again, after a build); raises if unusable."""
    loaded = _load()
    lib.__dict__.clear()
    lib._lib = loaded
    return lib


def tilemix_status_string(status: int) -> str:
    return lib.tilemix_status_string(status).decode()


def tilemix_last_error() -> str:
    return lib.tilemix_last_error().decode()


def tilemix_version() -> int:
    return int(lib.tilemix_version())


# ----------------------------------------------------------------------------
# torch marshalling
# ----------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _check(rc: int, where: str):
    if rc != 0:
        raise TilemixError(rc, where, tilemix_last_error())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dev(t, name, dtype=None):
    torch = _torch()
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def tilemix_quantize_blockwise(x, cu_seqlens, max_seqlen: int, block: int = 128,
                               *, x8=None, scale=None, status=None,
                               stream=None):
    """Blockwise symmetric INT8 quantisation of fp16 x [T, H, d].

    Returns (x8 int8 [T, H, d], scale fp32 [H, batch, ceil(max_seqlen/block)])."""
    torch = _torch()
    _dev(x, "x", torch.float16)
    _dev(cu_seqlens, "cu_seqlens", torch.int32)
    t, heads, d = x.shape
    batch = cu_seqlens.numel() - 1
    nblk = -(-max_seqlen // block)
    if x8 is None:
        x8 = torch.empty((t, heads, d), dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty((heads, batch, nblk), dtype=torch.float32,
                            device=x.device)
    _dev(x8, "x8", torch.int8)
    _dev(scale, "scale", torch.float32)
    _check(lib.tilemix_quantize_blockwise(
        _ptr(x), _ptr(cu_seqlens), batch, max_seqlen, t, heads, d, block,
        _ptr(x8), _ptr(scale), _ptr(status), _stream(stream)),
        "tilemix_quantize_blockwise")
    return x8, scale


def tilemix_quantize_blockwise_qk(q, k, cu_seqlens, max_seqlen: int,
                                  block_q: int = 128, block_k: int = 128, *,
                                  q8=None, q_scale=None, k8=None, k_scale=None,
                                  status=None, stream=None):
    """Q and K quantised in one launch: returns (q8, q_scale, k8, k_scale),
    equal to two tilemix_quantize_blockwise calls."""
    torch = _torch()
    _dev(q, "q", torch.float16)
    _dev(k, "k", torch.float16)
    _dev(cu_seqlens, "cu_seqlens", torch.int32)
    t, hq, d = q.shape
    tk, hkv, dk = k.shape
    if (tk, dk) != (t, d):
        raise ValueError("q and k must share tokens and head_dim")
    batch = cu_seqlens.numel() - 1
    if q8 is None:
        q8 = torch.empty((t, hq, d), dtype=torch.int8, device=q.device)
    if k8 is None:
        k8 = torch.empty((t, hkv, d), dtype=torch.int8, device=q.device)
    if q_scale is None:
        q_scale = torch.empty((hq, batch, -(-max_seqlen // block_q)),
                              dtype=torch.float32, device=q.device)
    if k_scale is None:
        k_scale = torch.empty((hkv, batch, -(-max_seqlen // block_k)),
                              dtype=torch.float32, device=q.device)
    for tns, nm, dt in ((q8, "q8", torch.int8), (k8, "k8", torch.int8),
                        (q_scale, "q_scale", torch.float32),
                        (k_scale, "k_scale", torch.float32)):
        _dev(tns, nm, dt)
    _check(lib.tilemix_quantize_blockwise_qk(
        _ptr(q), _ptr(k), _ptr(cu_seqlens), batch, max_seqlen, t, hq, hkv, d,
        block_q, block_k, _ptr(q8), _ptr(q_scale), _ptr(k8), _ptr(k_scale),
        _ptr(status), _stream(stream)), "tilemix_quantize_blockwise_qk")
    return q8, q_scale, k8, k_scale


def tilemix_pack_mask(route, cu_seqlens, max_seqlen: int, block_m: int,
                      block_n: int, group: int, *, mask=None, status=None,
                      stream=None):
    """uint8 route [B, Hkv, ceil(max_seqlen/block_m), 64] -> uint64 words
    [B, Hkv, ceil(max_seqlen/block_m)] (returned as torch.int64 storage)."""
    torch = _torch()
    _dev(route, "route", torch.uint8)
    _dev(cu_seqlens, "cu_seqlens", torch.int32)
    batch, hkv, tm, ng = route.shape
    if ng != 64:
        raise ValueError("route last dimension must be 64")
    if mask is None:
        mask = torch.empty((batch, hkv, tm), dtype=torch.int64,
                           device=route.device)
    _dev(mask, "mask")
    _check(lib.tilemix_pack_mask(
        _ptr(route), _ptr(cu_seqlens), batch, max_seqlen, hkv, block_m,
        block_n, group, _ptr(mask), _ptr(status), _stream(stream)),
        "tilemix_pack_mask")
    return mask


def tilemix_route_template(layout, int8_permille: int, cu_seqlens,
                           max_seqlen: int, hkv: int, block_m: int,
                           block_n: int, group: int, *, seed: int = 0,
                           route=None, status=None, stream=None):
    """Route bytes [B, Hkv, ceil(max_seqlen/block_m), 64] (uint8, 1 = INT8)
    of a named layout ("band", "bigbird", ... or a TILEMIX_LAYOUT_* value)
    with an INT8 share of int8_permille / 1000 of each row's legal groups."""
    torch = _torch()
    _dev(cu_seqlens, "cu_seqlens", torch.int32)
    code = LAYOUTS[layout] if isinstance(layout, str) else int(layout)
    batch = cu_seqlens.numel() - 1
    tm = -(-max_seqlen // block_m)
    if route is None:
        route = torch.empty((batch, hkv, tm, 64), dtype=torch.uint8,
                            device=cu_seqlens.device)
    _dev(route, "route", torch.uint8)
    _check(lib.tilemix_route_template(
        code, int8_permille, seed & 0xFFFFFFFFFFFFFFFF, _ptr(cu_seqlens), batch,
        max_seqlen, hkv, block_m, block_n, group, _ptr(route), _ptr(status),
        _stream(stream)), "tilemix_route_template")
    return route


def tilemix_route_adaptive_workspace_bytes(batch: int, max_seqlen: int,
                                           hkv: int, head_dim: int,
                                           block_m: int) -> int:
    """Bytes of device scratch tilemix_route_adaptive needs."""
    return int(lib.tilemix_route_adaptive_workspace_bytes(
        batch, max_seqlen, hkv, head_dim, block_m))


def tilemix_route_adaptive(q, k, cu_seqlens, max_seqlen: int, block_m: int,
                           block_n: int, group: int, int8_permille: int, *,
                           head_map=None, workspace=None, route=None,
                           mask=None, want_route: bool = True, status=None,
                           stream=None):
    """Route bytes [B, Hkv, ceil(max_seqlen/block_m), 64] (uint8, 1 = INT8)
    chosen from the data: per query-tile row, the groups whose summed raw
    logits with the row are largest stay FP16.  q fp16 [T, hq, d], k fp16
    [T, hkv, d].  `workspace` (uint8 CUDA tensor) is allocated here when not
    given.  Returns the route bytes, or (route, mask) when `mask` (uint64
    words [B, Hkv, Tm], int64 CUDA tensor) is given; want_route=False skips
    the bytes (route is then None)."""
    torch = _torch()
    _dev(q, "q", torch.float16)
    _dev(k, "k", torch.float16)
    _dev(cu_seqlens, "cu_seqlens", torch.int32)
    _dev(head_map, "head_map", torch.int32)
    t, hq, d = q.shape
    hkv = k.shape[1]
    batch = cu_seqlens.numel() - 1
    tm = -(-max_seqlen // block_m)
    need = tilemix_route_adaptive_workspace_bytes(batch, max_seqlen, hkv, d,
                                                  block_m)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8,
                                device=q.device)
    _dev(workspace, "workspace")
    if route is None and want_route:
        route = torch.empty((batch, hkv, tm, 64), dtype=torch.uint8,
                            device=q.device)
    _dev(route, "route", torch.uint8)
    _dev(mask, "mask", torch.int64)
    _check(lib.tilemix_route_adaptive(
        _ptr(q), _ptr(k), _ptr(cu_seqlens), batch, max_seqlen, t, hq, hkv, d,
        _ptr(head_map), block_m, block_n, group, int8_permille,
        _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(route), _ptr(mask), _ptr(status), _stream(stream)),
        "tilemix_route_adaptive")
    return route if mask is None else (route, mask)


def tilemix_route_adaptive_noalloc(q, k, cu_seqlens, max_seqlen: int,
                                   block_m: int, block_n: int, group: int,
                                   int8_permille: int, *, route, mask=None,
                                   head_map=None, status=None, stream=None):
    """tilemix_route_adaptive with the library's static device scratch: the
    C call allocates nothing (outputs are the caller's: `route` uint8
    [B, Hkv, Tm, 64] and/or `mask` int64 [B, Hkv, Tm], either may be None).
    Calls that can overlap on the device share that scratch and must be
    ordered (one stream, or events)."""
    torch = _torch()
    _dev(q, "q", torch.float16)
    _dev(k, "k", torch.float16)
    _dev(cu_seqlens, "cu_seqlens", torch.int32)
    _dev(head_map, "head_map", torch.int32)
    _dev(route, "route", torch.uint8)
    _dev(mask, "mask", torch.int64)
    t, hq, d = q.shape
    _check(lib.tilemix_route_adaptive_noalloc(
        _ptr(q), _ptr(k), _ptr(cu_seqlens), cu_seqlens.numel() - 1, max_seqlen,
        t, hq, k.shape[1], d, _ptr(head_map), block_m, block_n, group,
        int8_permille, _ptr(route), _ptr(mask), _ptr(status), _stream(stream)),
        "tilemix_route_adaptive_noalloc")
    return route, mask


def tilemix_attn_prefill(q, k, v, cu_seqlens, max_seqlen: int, *, q8=None,
                         q_scale=None, k8=None, k_scale=None, v8=None,
                         v_scale=None, mask=None, block_m: int = 128,
                         block_n: int = 128, group: int = 1,
                         quant_block_q: int = 128, quant_block_k: int = 128,
                         softmax_scale: float = 0.0, head_map=None,
                         fp16_only: bool = False, kv_format: int = KV_FP16,
                         quant_on_chip: bool = False,
                         test_expire_wait: bool = False,
                         pv_f16_acc: bool = False, out=None, lse=None,
                         qk_dump=None, status=None, stream=None):
    """Causal tile-routed attention.  q fp16 [T, hq, d]; k, v fp16
    [T, hkv, d] (or k8/v8 int8 + scales with kv_format=KV_INT8).
    Returns out fp16 [T, hq, d]."""
    torch = _torch()
    _dev(q, "q", torch.float16)
    _dev(cu_seqlens, "cu_seqlens", torch.int32)
    t, hq, d = q.shape
    kv_src = k8 if kv_format == KV_INT8 else k
    if kv_src is None:
        raise ValueError("k (or k8 for KV_INT8) is required")
    hkv = kv_src.shape[1]
    for name, tt, dt in (("k", k, torch.float16), ("v", v, torch.float16),
                         ("q8", q8, torch.int8), ("k8", k8, torch.int8),
                         ("v8", v8, torch.int8),
                         ("q_scale", q_scale, torch.float32),
                         ("k_scale", k_scale, torch.float32),
                         ("v_scale", v_scale, torch.float32),
                         ("head_map", head_map, torch.int32),
                         ("lse", lse, torch.float32),
                         ("qk_dump", qk_dump, torch.int32)):
        _dev(tt, name, dt)
    _dev(mask, "mask")
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out", torch.float16)
    p = AttnParams()
    p.struct_size = C.sizeof(AttnParams)
    p.kv_format = kv_format
    p.flags = (FLAG_FP16_ONLY if fp16_only else 0) | \
        (FLAG_QUANT_ON_CHIP if quant_on_chip else 0) | \
        (FLAG_TEST_EXPIRE_WAIT if test_expire_wait else 0) | \
        (FLAG_PV_F16_ACC if pv_f16_acc else 0)
    p.q, p.q8, p.q_scale = _ptr(q), _ptr(q8), _ptr(q_scale)
    p.k, p.k8, p.k_scale = _ptr(k), _ptr(k8), _ptr(k_scale)
    p.v, p.v8, p.v_scale = _ptr(v), _ptr(v8), _ptr(v_scale)
    p.cu_seqlens = _ptr(cu_seqlens)
    p.batch = cu_seqlens.numel() - 1
    p.max_seqlen = max_seqlen
    p.total_tokens = t
    p.hq, p.hkv, p.head_dim = hq, hkv, d
    p.head_map = _ptr(head_map)
    p.mask = _ptr(mask)
    p.block_m, p.block_n, p.group = block_m, block_n, group
    p.quant_block_q, p.quant_block_k = quant_block_q, quant_block_k
    p.softmax_scale = softmax_scale
    p.causal = 1
    p.out, p.lse, p.qk_dump, p.status = (_ptr(out), _ptr(lse), _ptr(qk_dump),
                                         _ptr(status))
    _check(lib.tilemix_attn_prefill(C.byref(p), _stream(stream)),
           "tilemix_attn_prefill")
    return out


# ----------------------------------------------------------------------------
# rotary positions and the paged KV cache
# ----------------------------------------------------------------------------

def _packer(struct):
    """Packs a parameter struct from its fields in order (a small call spends
    less host time here than in setting ctypes fields one by one)."""
    code = {C.c_uint32: "I", C.c_int: "i", C.c_void_p: "P", C.c_int64: "q",
            C.c_float: "f", C.c_size_t: "N"}
    layout = _struct.Struct("@" + "".join(code[t] for _, t in struct._fields_) +
                            "0q")
    assert layout.size == C.sizeof(struct)
    return functools.partial(layout.pack, layout.size)


_pack_rope = _packer(RopeParams)
_pack_append = _packer(AppendParams)
_pack_attn = _packer(AttnPagedParams)


def _check_device(index, names, *tensors):
    """Every tensor has to lie on GPU `index`."""
    for i, t in enumerate(tensors):
        if t is not None and t.get_device() != index:
            name = names.split()[i]
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")


def _on(torch, index, stream):
    """What makes GPU `index` and `stream` (None: that GPU's current stream)
    current, or None where they are already: tensors made in a call belong to
    the stream that uses them."""
    if index < 0:
        raise ValueError("the first argument must be a CUDA tensor")
    if stream is None:
        if index == torch.cuda.current_device():
            return None
        return torch.cuda.device(index)
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, not on cuda:{index}")
    return torch.cuda.stream(stream)


def _call(torch, fn, where, packed, index):
    rc = fn(packed, torch._C._cuda_getCurrentRawStream(index))
    if rc != 0:
        _check(rc, where)


def _dtype_code(torch, dtype, name):
    if dtype is torch.float16:
        return 0
    if dtype is torch.bfloat16:
        return 1
    raise ValueError(f"{name} must be float16 or bfloat16, got {dtype}")


def _rows(t, name, shape, dtype):
    """Token and head strides of a [T, heads, d] tensor (an axis of one
    counts as packed, whatever stride torch gives it)."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got "
                         f"{tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    n, h, d = shape
    st, sh, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{name} must have contiguous channels")
    if h <= 1:
        sh = d
    return (st if n > 1 else h * sh), sh


def _tokens(t, name):
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    return t.shape


def _vector(t, name, n, dtype):
    """Pointer of a contiguous vector of n elements."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {t.numel()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _status_ptr(status):
    """Pointer of the caller's status word (int32, at least one element)."""
    if status is None:
        return 0
    if status.numel() < 1:
        raise ValueError("status must hold at least one element")
    return _vector(status, "status", status.numel(), _torch().int32)


def _layout_code(layout):
    return ROPE_LAYOUTS[layout] if isinstance(layout, str) else int(layout)


def _frequencies(freqs, head_dim):
    """Pointer and rotated channels of a frequency vector."""
    n = freqs.numel()
    if not 0 < 2 * n <= head_dim:
        raise ValueError(f"freqs must have 1 .. head_dim / 2 elements, got {n}")
    return _vector(freqs, "freqs", n, _torch().float64), 2 * n


def _cache(torch, k_pages, v_pages, k_scale, v_scale, page_table, cu_seqlens,
           kv_lens, dtype):
    """Checks the cache arguments: (kv_format, page strides, scale pointers,
    table stride, batch, page array's shape, table width)."""
    if k_pages.dim() != 4:
        raise ValueError("k_pages must be [num_pages, page_size, hkv, head_dim]")
    shape = k_pages.shape
    if v_pages.shape != shape or v_pages.dtype != k_pages.dtype:
        raise ValueError("k_pages and v_pages must share shape and dtype")
    n, page, hkv, d = shape
    kind = k_pages.dtype
    int8 = kind is torch.int8
    if not int8 and kind is not dtype:
        raise ValueError(f"pages must be {dtype} or int8, got {kind}")
    strides = k_pages.stride()
    if v_pages.stride() != strides and any(
            a != b and m > 1
            for a, b, m in zip(strides, v_pages.stride(), shape)):
        raise ValueError("k_pages and v_pages must share their strides")
    sp, st, sh, sd = strides
    if sd != 1 and d > 1:
        raise ValueError("pages must have contiguous channels")
    if hkv <= 1:
        sh = d
    if page <= 1:
        st = hkv * sh
    if n <= 1:
        sp = page * st
    if int8 != (k_scale is not None) or int8 != (v_scale is not None):
        raise ValueError("k_scale and v_scale go with int8 pages, and only "
                         "with them")
    ks = vs = 0
    if int8:
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.shape != (n, hkv, page):
                raise ValueError(f"{name} must have shape {(n, hkv, page)}, "
                                 f"got {tuple(t.shape)}")
        ks = _vector(k_scale, "k_scale", n * hkv * page, torch.float32)
        vs = _vector(v_scale, "v_scale", n * hkv * page, torch.float32)
    batch = cu_seqlens.numel() - 1
    if batch < 0:
        raise ValueError("cu_seqlens must have batch + 1 elements")
    if (page_table.dim() != 2 or page_table.shape[0] != batch or
            page_table.dtype != torch.int32):
        raise ValueError(f"page_table must be int32 [{batch}, max_pages]")
    width = page_table.shape[1]
    ts, tw = page_table.stride()
    if width > 1 and tw != 1:
        raise ValueError("page_table must have contiguous rows")
    return (KV_INT8 if int8 else KV_FP16, sp, st, sh, ks, vs,
            page_table.data_ptr(), ts if batch > 1 else width,
            _vector(cu_seqlens, "cu_seqlens", batch + 1, torch.int32),
            _vector(kv_lens, "kv_lens", batch, torch.int32), batch, n, page,
            hkv, d, width)


def tilemix_rope_frequencies(rot_dim: int, base: float = 10000.0, *,
                             scaling: str = "none", factor: float = 1.0,
                             low_freq_factor: float = 1.0,
                             high_freq_factor: float = 4.0,
                             original_max_position: int = 0, device=None):
    """Rotary frequencies (radians per position) as a float64 tensor
    [rot_dim / 2] on `device` (host without one), and the attn_factor that
    goes with them.  `scaling`: one of ROPE_SCALINGS; "yarn" takes its two
    rotation counts (32 and 1 usually) as high_freq_factor and
    low_freq_factor."""
    torch = _torch()
    code = ROPE_SCALINGS[scaling] if isinstance(scaling, str) else int(scaling)
    buf = (C.c_double * max(1, rot_dim // 2))()
    att = C.c_float(1.0)
    _check(lib.tilemix_rope_frequencies(
        code, rot_dim, base, factor, low_freq_factor, high_freq_factor,
        original_max_position, buf, C.byref(att)), "tilemix_rope_frequencies")
    freqs = torch.tensor(list(buf), dtype=torch.float64, device=device)
    return freqs, float(att.value)


@functools.lru_cache(maxsize=None)
def _rope_function():
    """tilemix_rope as a node of autograd: its gradient is the rotation by the
    negative angle (with the same attn_factor), so it is one too."""
    torch = _torch()

    def rows(g):  # a gradient may be expanded, or lie anywhere
        if g.stride(-1) != 1 or any(s % 8 for s in g.stride()[:2]):
            g = g.contiguous()
        return g.clone() if g.data_ptr() % 16 else g

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, positions, freqs, layout, attn_factor, inverse):
            ctx.save_for_backward(positions, freqs)
            ctx.how = layout, attn_factor, inverse
            ctx.set_materialize_grads(False)
            return tilemix_rope(q, k, positions, freqs, layout=layout,
                                attn_factor=attn_factor, inverse=inverse)

        @staticmethod
        def backward(ctx, gq, gk):
            layout, attn_factor, inverse = ctx.how
            want = [g is not None and need
                    for g, need in zip((gq, gk), ctx.needs_input_grad)]
            grads = [rows(g) for g, w in zip((gq, gk), want) if w]
            done = iter(())
            if grads:
                done = iter(tilemix_rope(
                    grads[0], grads[1] if len(grads) > 1 else None,
                    *ctx.saved_tensors, layout=layout, attn_factor=attn_factor,
                    inverse=not inverse))
            return (*(next(done) if w else None for w in want),
                    None, None, None, None, None)

    return Rope


def tilemix_rope(q, k, positions, freqs, *, layout="half",
                 attn_factor: float = 1.0, inverse: bool = False, q_out=None,
                 k_out=None, stream=None):
    """Rotary positions of q [T, hq, d] and k [T, hkv, d] (k may be None) in
    one launch; fp16 or bf16, token and head strides free.  positions int32
    [T], freqs float64 [rot_dim / 2] on the device (channels past rot_dim are
    copied).  `inverse` rotates back, which is also the gradient; autograd
    records it where q or k requires one (not with q_out or k_out given;
    positions and freqs are constants).  As with any torch operation, a
    backward pass goes into a CUDA graph only while no earlier result of the
    same leaves is alive.
    Outputs default to new contiguous tensors; q_out=q rotates in place.
    Returns (q_out, k_out)."""
    torch = _torch()
    index = q.get_device()
    ctx = _on(torch, index, stream)
    if ctx is not None:
        with ctx:
            return tilemix_rope(q, k, positions, freqs, layout=layout,
                                attn_factor=attn_factor, inverse=inverse,
                                q_out=q_out, k_out=k_out)
    if torch.is_grad_enabled() and (q.requires_grad or
                                    k is not None and k.requires_grad):
        if q_out is not None or k_out is not None:
            raise ValueError("q_out and k_out take no part in autograd: leave "
                             "them out, or call under torch.no_grad()")
        return _rope_function().apply(q, k, positions, freqs, layout,
                                      attn_factor, inverse)
    _check_device(index, "k positions freqs q_out k_out", k, positions, freqs,
                  q_out, k_out)
    dtype = q.dtype
    code = _dtype_code(torch, dtype, "q")
    shape = _tokens(q, "q")
    t, hq, d = shape
    qt, qh = _rows(q, "q", shape, dtype)
    pos = _vector(positions, "positions", t, torch.int32)
    fp, rot = _frequencies(freqs, d)
    if q_out is None:
        q_out = q.new_empty(shape)
        qot, qoh = hq * d, d
    else:
        qot, qoh = _rows(q_out, "q_out", shape, dtype)
    kp = kop = hkv = kt = kh = kot = koh = 0
    if k is not None:
        kshape = _tokens(k, "k")
        _, hkv, _ = kshape
        if kshape[0] != t or kshape[2] != d:
            raise ValueError("q and k must share tokens and head_dim")
        kt, kh = _rows(k, "k", kshape, dtype)
        if k_out is None:
            k_out = k.new_empty(kshape)
            kot, koh = hkv * d, d
        else:
            kot, koh = _rows(k_out, "k_out", kshape, dtype)
        kp, kop = k.data_ptr(), k_out.data_ptr()
        if t and not (kp and hkv):
            raise ValueError("k has no heads")
    elif k_out is not None:
        raise ValueError("k_out without k")
    _call(torch, lib.tilemix_rope, "tilemix_rope",
          _pack_rope(code, _layout_code(layout), 1 if inverse else 0,
                     q.data_ptr(), kp, q_out.data_ptr(), kop, qt, qh, kt, kh,
                     qot, qoh, kot, koh, pos, fp, attn_factor, t, hq, hkv, d,
                     rot), index)
    return q_out, k_out


def tilemix_paged_append(k, v, page_table, cu_seqlens, kv_lens, k_pages,
                         v_pages, *, k_scale=None, v_scale=None, q=None,
                         q_out=None, positions=None, freqs=None,
                         layout="half", attn_factor: float = 1.0, status=None,
                         stream=None):
    """Writes the new tokens' k and v [T, hkv, d] into the pages of the cache
    in one launch: token i of sequence b (n_b of them) to position kv_lens[b]
    - n_b + i.  k_pages, v_pages [num_pages, page_size, hkv, d] of the same
    type, or int8 with k_scale, v_scale fp32 [num_pages, hkv, page_size].
    With freqs, k (and q, if given) is rotated on the way, by each token's
    position in the cache or by `positions`.  Returns the rotated q (rows
    past cu_seqlens[-1] are not written) or None.  Records no gradient."""
    torch = _torch()
    index = k.get_device()
    ctx = _on(torch, index, stream)
    if ctx is not None:
        with ctx:
            return tilemix_paged_append(
                k, v, page_table, cu_seqlens, kv_lens, k_pages, v_pages,
                k_scale=k_scale, v_scale=v_scale, q=q, q_out=q_out,
                positions=positions, freqs=freqs, layout=layout,
                attn_factor=attn_factor, status=status)
    _check_device(index, "v page_table cu_seqlens kv_lens k_pages v_pages "
                  "k_scale v_scale q q_out positions freqs status", v,
                  page_table, cu_seqlens, kv_lens, k_pages, v_pages, k_scale,
                  v_scale, q, q_out, positions, freqs, status)
    dtype = k.dtype
    code = _dtype_code(torch, dtype, "k")
    (fmt, sp, st, sh, ks, vs, table, ts, cu, lens, batch, n, page, hkv, d,
     width) = _cache(torch, k_pages, v_pages, k_scale, v_scale, page_table,
                     cu_seqlens, kv_lens, dtype)
    shape = _tokens(k, "k")
    t = shape[0]
    if shape[1:] != (hkv, d):
        raise ValueError("k and the pages must share heads and head_dim")
    kt, kh = _rows(k, "k", shape, dtype)
    vt, vh = _rows(v, "v", shape, dtype)
    fp = rot = pos = 0
    if freqs is not None:
        fp, rot = _frequencies(freqs, d)
    elif q is not None or positions is not None:
        raise ValueError("q and positions need freqs")
    if positions is not None:
        pos = _vector(positions, "positions", t, torch.int32)
    qp = qop = hq = qt = qh = qot = qoh = 0
    if q is not None:
        qshape = _tokens(q, "q")
        hq = qshape[1]
        if qshape[0] != t or qshape[2] != d:
            raise ValueError("q and k must share tokens and head_dim")
        qt, qh = _rows(q, "q", qshape, dtype)
        if q_out is None:
            q_out = q.new_empty(qshape)
            qot, qoh = hq * d, d
        else:
            qot, qoh = _rows(q_out, "q_out", qshape, dtype)
        qp, qop = q.data_ptr(), q_out.data_ptr()
        if t and not qp:
            raise ValueError("q has no heads")
    elif q_out is not None:
        raise ValueError("q_out without q")
    _call(torch, lib.tilemix_paged_append, "tilemix_paged_append",
          _pack_append(code, fmt, _layout_code(layout), k.data_ptr(),
                       v.data_ptr(), qp, qop, kt, kh, vt, vh, qt, qh, qot, qoh,
                       pos, fp, k_pages.data_ptr(), v_pages.data_ptr(), sp, st,
                       sh, ks, vs, table, ts, cu, lens, batch, t, hq, hkv, d,
                       rot, n, page, width, attn_factor, _status_ptr(status)),
          index)
    return q_out


@functools.lru_cache(maxsize=256)
def tilemix_attn_paged_workspace_bytes(max_q_len: int, hq: int, hkv: int,
                                       head_dim: int) -> int:
    """Bytes of device scratch tilemix_attn_paged needs; 0 for sizes it
    refuses."""
    if not all(-1 << 31 <= x < 1 << 31 for x in (max_q_len, hq, hkv, head_dim)):
        return 0  # (ctypes would pass the low 32 bits)
    return int(lib.tilemix_attn_paged_workspace_bytes(max_q_len, hq, hkv,
                                                      head_dim))


def tilemix_attn_paged(q, k_pages, v_pages, page_table, cu_seqlens, kv_lens,
                       max_q_len: int, max_kv_len: int, *, k_scale=None,
                       v_scale=None, causal: bool = True,
                       softmax_scale: float = 0.0, out=None, lse=None,
                       workspace=None, status=None,
                       test_expire_wait: bool = False, stream=None):
    """Attention of the new tokens q [T, hq, d] (fp16 or bf16) over the paged
    cache: kv_lens int32 [B] counts each sequence's keys, the new tokens' own
    among them when `causal`.  max_q_len and max_kv_len bound the sequences'
    new tokens and keys.  `workspace` (a CUDA tensor, 16-byte aligned, of
    tilemix_attn_paged_workspace_bytes) is allocated here when not given; two
    calls that may run at the same time need two.  Rows of q past
    cu_seqlens[-1] are neither read nor written.  Forward only: no gradient is
    recorded.  Returns out [T, hq, d]."""
    torch = _torch()
    index = q.get_device()
    ctx = _on(torch, index, stream)
    if ctx is not None:
        with ctx:
            return tilemix_attn_paged(
                q, k_pages, v_pages, page_table, cu_seqlens, kv_lens,
                max_q_len, max_kv_len, k_scale=k_scale, v_scale=v_scale,
                causal=causal, softmax_scale=softmax_scale, out=out, lse=lse,
                workspace=workspace, status=status,
                test_expire_wait=test_expire_wait)
    _check_device(index, "k_pages v_pages page_table cu_seqlens kv_lens "
                  "k_scale v_scale out lse workspace status", k_pages, v_pages,
                  page_table, cu_seqlens, kv_lens, k_scale, v_scale, out, lse,
                  workspace, status)
    if not (max_q_len < 1 << 31 and max_kv_len < 1 << 31):
        raise ValueError("max_q_len and max_kv_len must be below 2^31")
    dtype = q.dtype
    code = _dtype_code(torch, dtype, "q")
    (fmt, sp, st, sh, ks, vs, table, ts, cu, lens, batch, n, page, hkv, d,
     width) = _cache(torch, k_pages, v_pages, k_scale, v_scale, page_table,
                     cu_seqlens, kv_lens, dtype)
    shape = _tokens(q, "q")
    t, hq, dq = shape
    if dq != d:
        raise ValueError("q and the pages must share head_dim")
    qt, qh = _rows(q, "q", shape, dtype)
    if out is None:
        out = q.new_empty(shape)
    elif out.shape != shape or out.dtype != dtype or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape "
                         f"{tuple(shape)}")
    lp = 0 if lse is None else _vector(lse, "lse", hq * t, torch.float32)
    if workspace is None:
        need = tilemix_attn_paged_workspace_bytes(max_q_len, hq, hkv, d)
        workspace = q.new_empty(max(need, 16), dtype=torch.uint8)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _call(torch, lib.tilemix_attn_paged, "tilemix_attn_paged",
          _pack_attn(code, fmt, 1 if causal else 0, q.data_ptr(), qt, qh,
                     k_pages.data_ptr(), v_pages.data_ptr(), sp, st, sh, ks, vs,
                     table, ts, cu, lens, batch, t, max_q_len, max_kv_len, hq,
                     hkv, d, n, page, width, softmax_scale,
                     FLAG_TEST_EXPIRE_WAIT if test_expire_wait else 0,
                     out.data_ptr(), lp,
                     workspace.data_ptr(),
                     workspace.numel() * workspace.element_size(),
                     _status_ptr(status)), index)
    return out
