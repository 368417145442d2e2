"""ctypes binding of libtg_gemm.so (include/tg_gemm.h, include/tg_attention.h,
include/tg_cache.h), argument marshalling only.

The raw entry points keep the C names (``tg_gemm``, ``tg_gemm_ex``, ...) and
take integers for pointers and the stream.  ``gemm``, ``gemm_host``,
``attention``, ``cache_plan``, ``cache_write``, ``tree_mask`` and
``tree_attention`` are the torch-tensor conveniences: they check dtype, shape, contiguity and device,
pass ``data_ptr()`` and the current stream, and raise on a non-OK status.
Every step of the computation runs in the library's CUDA kernels; there is
no fallback of any kind, and a missing library is an error.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
from typing import NamedTuple

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtg_gemm.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "tg_gemm.h")
HEADERS = [HEADER, os.path.join(os.path.dirname(HERE), "include", "tg_attention.h"),
           os.path.join(os.path.dirname(HERE), "include", "tg_cache.h")]

TG_EPILOGUE_NONE = 0
TG_EPILOGUE_BIAS = 1
TG_EPILOGUE_BIAS_GELU = 2
TG_EPILOGUE_BIAS_GELU_TANH = 3
TG_EPILOGUE_BIAS_SOFTMAX = 4

TG_OK = 0
TG_ERR_INVALID_ARG = 1
TG_ERR_MISALIGNED = 2
TG_ERR_UNSUPPORTED_DEVICE = 3
TG_ERR_LAUNCH = 4
TG_ERR_TIMEOUT = 5
TG_ERR_OOM = 6
TG_ERR_CUDA = 7
TG_ERR_SCRATCH_LIMIT = 8

TG_INJECT_SKIP_FIRST_LOAD = 1
TG_ATTN_SPLIT_AUTO, TG_ATTN_SPLIT_NEVER, TG_ATTN_SPLIT_ALL = 0, 1, 2
TG_INJECT_SKIP_STREAMK_FLAGS = 2
TG_TYPE_FP16, TG_TYPE_BF16 = 0, 1
TG_CACHE_MAX_BATCH = 8192
TG_TREE_MAX_WORDS = 64
TG_PLAN_NO_PAGES, TG_PLAN_TABLE_FULL, TG_PLAN_BAD_LENGTH = 1, 2, 4
TG_PLAN_BAD_TOKENS, TG_PLAN_BAD_RING = 8, 16
TG_SPLIT_AUTO = 0
TG_SPLIT_TILES = 1
TG_SPLIT_STREAM_K = 2

EPILOGUES = {"none": TG_EPILOGUE_NONE, "bias": TG_EPILOGUE_BIAS, "bias_gelu": TG_EPILOGUE_BIAS_GELU,
             "bias_gelu_tanh": TG_EPILOGUE_BIAS_GELU_TANH, "bias_softmax": TG_EPILOGUE_BIAS_SOFTMAX}


class TgError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {tg_status_string(status)}" if what else tg_status_string(status))


class tg_config_t(ctypes.Structure):
    _fields_ = [("id", ctypes.c_int), ("block_m", ctypes.c_int), ("block_n", ctypes.c_int),
                ("block_k", ctypes.c_int), ("stages", ctypes.c_int), ("cta_pair", ctypes.c_int),
                ("group_m", ctypes.c_int), ("epi_warps", ctypes.c_int), ("split", ctypes.c_int),
                ("loader", ctypes.c_int)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class tg_attention_options_t(ctypes.Structure):
    _fields_ = [("wait_limit_ns", ctypes.c_uint64), ("inject", ctypes.c_int),
                ("kv_split", ctypes.c_int)]


class tg_options_t(ctypes.Structure):
    _fields_ = [("config_id", ctypes.c_int), ("wait_limit_ns", ctypes.c_uint64),
                ("inject", ctypes.c_int), ("group_m", ctypes.c_int), ("split", ctypes.c_int)]


class tg_tree_attention_t(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int)] + \
        [(n, ctypes.c_int64) for n in ("tokens", "batch", "kv_heads", "group", "head_dim")] + \
        [("scale", ctypes.c_float), ("q", ctypes.c_void_p), ("q_token_stride", ctypes.c_int64),
         ("q_head_stride", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
         ("kv_token_stride", ctypes.c_int64), ("kv_head_stride", ctypes.c_int64),
         ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p)] + \
        [(n, ctypes.c_int64) for n in ("num_pages", "page_size", "page_stride", "slot_stride",
                                       "cache_head_stride")] + \
        [("block_tables", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
         ("max_pages", ctypes.c_int64), ("lens", ctypes.c_void_p), ("starts", ctypes.c_void_p),
         ("mask", ctypes.c_void_p), ("words", ctypes.c_int64), ("mask_stride", ctypes.c_int64),
         ("out", ctypes.c_void_p), ("out_token_stride", ctypes.c_int64),
         ("out_head_stride", ctypes.c_int64), ("workspace", ctypes.c_void_p),
         ("workspace_bytes", ctypes.c_size_t), ("wait_limit_ns", ctypes.c_uint64),
         ("inject", ctypes.c_int), ("own_v_strides", ctypes.c_int),
         ("v_token_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64)]


# The same struct as bytes: packing it takes a quarter of the time of setting 39 ctypes fields.
_TREE_ARGS = struct.Struct("@" + "".join(
    {ctypes.c_int: "i", ctypes.c_int64: "q", ctypes.c_float: "f", ctypes.c_void_p: "P",
     ctypes.c_size_t: "N", ctypes.c_uint64: "Q"}[t] for _, t in tg_tree_attention_t._fields_)
    + "0q")

_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libtg_gemm.so not found at {path}; build it with "
                          "`python -m tensor_core_gemm_fp16_b200.build`")
    lib = ctypes.CDLL(path)
    vp, i64, c_int, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.tg_gemm.argtypes = [vp, vp, vp, vp, i64, i64, i64, c_int, vp]
    lib.tg_gemm.restype = c_int
    lib.tg_gemm_ex.argtypes = [vp, vp, vp, vp, i64, i64, i64, c_int,
                               ctypes.POINTER(tg_options_t), vp]
    lib.tg_gemm_ex.restype = c_int
    lib.tg_gemm_host.argtypes = [vp, vp, vp, vp, i64, i64, i64, c_int, vp, sz, vp]
    lib.tg_gemm_host.restype = c_int
    lib.tg_gemm_host_workspace_size.argtypes = [i64, i64, i64, c_int]
    lib.tg_gemm_host_workspace_size.restype = sz
    lib.tg_gemm_check_error.argtypes = [vp]
    lib.tg_gemm_check_error.restype = c_int
    lib.tg_status_string.argtypes = [c_int]
    lib.tg_status_string.restype = ctypes.c_char_p
    lib.tg_num_configs.argtypes = []
    lib.tg_num_configs.restype = c_int
    lib.tg_config_info.argtypes = [c_int, ctypes.POINTER(tg_config_t)]
    lib.tg_config_info.restype = c_int
    lib.tg_gemm_select_config.argtypes = [i64, i64, i64, c_int, c_int, ctypes.POINTER(tg_config_t)]
    lib.tg_gemm_select_config.restype = c_int
    lib.tg_gemm_launch_count.argtypes = [vp, vp, vp, vp, i64, i64, i64, c_int]
    lib.tg_gemm_launch_count.restype = c_int
    lib.tg_gemm_noalloc.argtypes = [vp, vp, vp, vp, i64, i64, i64, c_int, vp]
    lib.tg_gemm_noalloc.restype = c_int
    lib.tg_version.argtypes = []
    lib.tg_version.restype = c_int
    lib.tg_attention_fwd.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, c_int,
                                     ctypes.c_float, vp]
    lib.tg_attention_fwd.restype = c_int
    lib.tg_attention_fwd_ex.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, c_int,
                                        ctypes.c_float, ctypes.POINTER(tg_attention_options_t), vp]
    lib.tg_attention_fwd_ex.restype = c_int
    i64p = ctypes.POINTER(i64)
    lib.tg_attention_plan.argtypes = [i64, i64, i64, i64, i64, c_int, c_int, c_int, i64p, i64p,
                                      i64p]
    lib.tg_attention_plan.restype = c_int
    lib.tg_cache_plan.argtypes = [vp, vp, i64, vp, vp, i64, vp, i64, i64, i64, vp, i64, vp, vp, vp,
                                  vp, vp, vp, vp, vp]
    lib.tg_cache_plan.restype = c_int
    lib.tg_cache_write.argtypes = [vp, vp] + [i64] * 5 + [vp, vp, vp] + [i64] * 5 + [vp]
    lib.tg_cache_write.restype = c_int
    lib.tg_cache_write_ex.argtypes = [vp, i64, i64, vp] + [i64] * 5 + [vp, vp, vp] + [i64] * 5 + \
        [vp]
    lib.tg_cache_write_ex.restype = c_int
    lib.tg_tree_mask.argtypes = [vp, i64, vp, i64, i64, vp, vp, vp]
    lib.tg_tree_mask.restype = c_int
    lib.tg_tree_attention.argtypes = [ctypes.POINTER(tg_tree_attention_t), vp]
    lib.tg_tree_attention.restype = c_int
    lib._tree_attention_packed = lib["tg_tree_attention"]      # the struct as bytes
    lib._tree_attention_packed.argtypes = [ctypes.c_char_p, vp]
    lib._tree_attention_packed.restype = c_int
    lib.tg_tree_attention_workspace_size.argtypes = [i64]
    lib.tg_tree_attention_workspace_size.restype = sz
    lib._tree_workspace_halves = {d: (lib.tg_tree_attention_workspace_size(d) + 1) // 2
                                  for d in (64, 128)}
    _lib = lib
    return lib


def header_symbols(headers=None):
    """Function names declared in the library's headers (include/*.h)."""
    names = set()
    for header in ([headers] if isinstance(headers, str) else (headers or HEADERS)):
        with open(header) as f:
            text = f.read()
        text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
        names.update(re.findall(r"\b(tg_[a-z0-9_]+)\s*\(", text))
    return sorted(names)


# ---------------------------------------------------------------- raw entry points

def tg_gemm(A: int, B: int, bias: int | None, C: int, M: int, N: int, K: int, epilogue: int,
            stream: int | None = None) -> int:
    return load().tg_gemm(A, B, bias, C, M, N, K, epilogue, stream)


def tg_gemm_noalloc(A: int, B: int, bias: int | None, C: int, M: int, N: int, K: int,
                    epilogue: int, stream: int | None = None) -> int:
    """tg_gemm without any allocation: repacking scratch comes from the
    library's fixed device array (see tg_gemm.h)."""
    return load().tg_gemm_noalloc(A, B, bias, C, M, N, K, epilogue, stream)


def noalloc_scratch_bytes(header: str = HEADER) -> int:
    """TG_NOALLOC_SCRATCH_BYTES as declared in include/tg_gemm.h."""
    m = re.search(r"#define\s+TG_NOALLOC_SCRATCH_BYTES\s+\((\d+)u\s*<<\s*(\d+)\)",
                  open(header).read())
    return int(m.group(1)) << int(m.group(2))


def tg_gemm_ex(A, B, bias, C, M, N, K, epilogue, config_id=-1, wait_limit_ns=0, inject=0,
               stream=None, group_m=0, split=0) -> int:
    opts = tg_options_t(config_id, wait_limit_ns, inject, group_m, split)
    return load().tg_gemm_ex(A, B, bias, C, M, N, K, epilogue, ctypes.byref(opts), stream)


def tg_gemm_host(A_host, B_host, bias_host, C_host, M, N, K, epilogue, workspace,
                 workspace_bytes, stream=None) -> int:
    return load().tg_gemm_host(A_host, B_host, bias_host, C_host, M, N, K, epilogue, workspace,
                               workspace_bytes, stream)


def tg_gemm_host_workspace_size(M, N, K, has_bias) -> int:
    return load().tg_gemm_host_workspace_size(M, N, K, 1 if has_bias else 0)


def tg_gemm_check_error(stream=None) -> int:
    return load().tg_gemm_check_error(stream)


def tg_status_string(status: int) -> str:
    return load().tg_status_string(status).decode()


def tg_num_configs() -> int:
    return load().tg_num_configs()


def tg_config_info(config_id: int) -> dict:
    c = tg_config_t()
    st = load().tg_config_info(config_id, ctypes.byref(c))
    if st != TG_OK:
        raise TgError(st, "tg_config_info")
    return c.as_dict()


def tg_gemm_select_config(M, N, K, epilogue, num_sms=148) -> dict:
    c = tg_config_t()
    st = load().tg_gemm_select_config(M, N, K, epilogue, num_sms, ctypes.byref(c))
    if st != TG_OK:
        raise TgError(st, "tg_gemm_select_config")
    return c.as_dict()


def tg_gemm_launch_count(A, B, bias, C, M, N, K, epilogue) -> int:
    return load().tg_gemm_launch_count(A, B, bias, C, M, N, K, epilogue)


def tg_version() -> int:
    return load().tg_version()


# ---------------------------------------------------------------- torch conveniences

def _epi(epilogue):
    if isinstance(epilogue, str):
        return EPILOGUES[epilogue]
    return int(epilogue)


def _stream_handle(torch, device):
    return torch.cuda.current_stream(device).cuda_stream


def gemm(a, b, bias=None, epilogue=None, out=None, *, config_id=-1, wait_limit_ns=0, inject=0,
         group_m=0, split=0):
    """C = g(a @ b + bias) on the GPU through tg_gemm_ex.

    a: (M, K) fp16 CUDA, b: (K, N) fp16 CUDA, bias: (N,) fp16 CUDA or None,
    both row-major contiguous.  epilogue defaults to "bias_gelu" when a
    bias is given, else "none".  Returns ``out`` (allocated if None).
    """
    import torch
    if epilogue is None:
        epilogue = TG_EPILOGUE_BIAS_GELU if bias is not None else TG_EPILOGUE_NONE
    epi = _epi(epilogue)
    for name, t in (("a", a), ("b", b), ("bias", bias), ("out", out)):
        if t is None:
            continue
        if t.dtype != torch.float16:
            raise TypeError(f"{name} must be float16, got {t.dtype}")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous (row-major)")
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[0]:
        raise ValueError(f"shape mismatch: a {tuple(a.shape)} @ b {tuple(b.shape)}")
    M, K = a.shape
    N = b.shape[1]
    if bias is not None and tuple(bias.shape) != (N,):
        raise ValueError(f"bias must have shape ({N},)")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=a.device)
    elif tuple(out.shape) != (M, N):
        raise ValueError(f"out must have shape ({M}, {N})")
    with torch.cuda.device(a.device):
        st = tg_gemm_ex(a.data_ptr(), b.data_ptr(), bias.data_ptr() if bias is not None else None,
                        out.data_ptr(), M, N, K, epi, config_id=config_id,
                        wait_limit_ns=wait_limit_ns, inject=inject,
                        stream=_stream_handle(torch, a.device), group_m=group_m, split=split)
    if st != TG_OK:
        raise TgError(st, "tg_gemm")
    return out


def tg_attention_fwd(Q, K, V, O, batch, heads, seq_q, seq_k, head_dim, causal, scale,
                     stream=None) -> int:
    return load().tg_attention_fwd(Q, K, V, O, batch, heads, seq_q, seq_k, head_dim, int(causal),
                                   float(scale), stream)


def tg_attention_plan(batch, heads, seq_q, seq_k, head_dim, causal, kv_split=0,
                      num_sms=148) -> dict:
    """Host-only: units, split units and grid of the launch tg_attention_fwd_ex
    would make (no device needed)."""
    units, split, grid = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    st = load().tg_attention_plan(batch, heads, seq_q, seq_k, head_dim, int(causal), kv_split,
                                  num_sms, ctypes.byref(units), ctypes.byref(split),
                                  ctypes.byref(grid))
    if st != TG_OK:
        raise TgError(st, "tg_attention_plan")
    return {"units": units.value, "split": split.value, "grid": grid.value}


def tg_attention_fwd_ex(Q, K, V, O, batch, heads, seq_q, seq_k, head_dim, causal, scale,
                        wait_limit_ns=0, inject=0, stream=None, kv_split=0) -> int:
    opts = tg_attention_options_t(wait_limit_ns, inject, kv_split)
    return load().tg_attention_fwd_ex(Q, K, V, O, batch, heads, seq_q, seq_k, head_dim,
                                      int(causal), float(scale), ctypes.byref(opts), stream)


def attention(q, k, v, causal=False, scale=0.0, out=None, *, wait_limit_ns=0, inject=0,
              kv_split=0):
    """O = softmax(scale q k^T) v on the GPU through tg_attention_fwd_ex.

    q: (B, H, Sq, D), k and v: (B, H, Sk, D), fp16 contiguous CUDA tensors,
    D in {64, 128}; scale 0 means 1/sqrt(D).  kv_split: TG_ATTN_SPLIT_*.
    Returns ``out`` (allocated if None).
    """
    import torch
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if t is None:
            continue
        if t.dtype != torch.float16:
            raise TypeError(f"{name} must be float16, got {t.dtype}")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape or k.shape[:2] != q.shape[:2] \
            or k.shape[3] != q.shape[3]:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, "
                         f"v {tuple(v.shape)}")
    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape:
        raise ValueError(f"out must have shape {tuple(q.shape)}")
    with torch.cuda.device(q.device):
        st = tg_attention_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H,
                                 Sq, Sk, D, causal, scale, wait_limit_ns=wait_limit_ns,
                                 inject=inject, stream=_stream_handle(torch, q.device),
                                 kv_split=kv_split)
    if st != TG_OK:
        raise TgError(st, "tg_attention_fwd")
    return out


def gemm_host(a, b, bias=None, epilogue=None, out=None, workspace=None, device=None):
    """End-to-end GEMM on HOST tensors through tg_gemm_host.

    a, b, bias, out are CPU fp16 tensors (pinned for async copies).  The
    device workspace (uint8 CUDA tensor) is allocated when not given.
    Enqueues copies + GEMM + copy-back on the current stream and waits for
    them; returns ``out``.
    """
    import torch
    if epilogue is None:
        epilogue = TG_EPILOGUE_BIAS_GELU if bias is not None else TG_EPILOGUE_NONE
    epi = _epi(epilogue)
    M, K = a.shape
    N = b.shape[1]
    device = torch.device(device or "cuda")
    has_bias = bias is not None and epi != TG_EPILOGUE_NONE
    need = tg_gemm_host_workspace_size(M, N, K, has_bias)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, pin_memory=True)
    with torch.cuda.device(device):
        stream = torch.cuda.current_stream(device)
        st = tg_gemm_host(a.data_ptr(), b.data_ptr(), bias.data_ptr() if has_bias else None,
                          out.data_ptr(), M, N, K, epi, workspace.data_ptr(),
                          workspace.numel(), stream.cuda_stream)
        if st != TG_OK:
            raise TgError(st, "tg_gemm_host")
        stream.synchronize()
    return out


# ---------------------------------------------------------------- paged cache

def tg_cache_plan(lens, add, batch, starts, offsets, tokens, block_tables, table_stride, max_pages,
                  page_size, free_pages, num_pages, ring, lens_out, ring_out, starts_out, slots,
                  positions, status, stream=None) -> int:
    return load().tg_cache_plan(lens, add, batch, starts, offsets, tokens, block_tables,
                                table_stride, max_pages, page_size, free_pages, num_pages, ring,
                                lens_out, ring_out, starts_out, slots, positions, status, stream)


def tg_cache_write(k, v, tokens, heads, head_dim, token_stride, head_stride, slots, k_cache,
                   v_cache, num_pages, page_size, page_stride, slot_stride, cache_head_stride,
                   stream=None) -> int:
    return load().tg_cache_write(k, v, tokens, heads, head_dim, token_stride, head_stride, slots,
                                 k_cache, v_cache, num_pages, page_size, page_stride, slot_stride,
                                 cache_head_stride, stream)


def tg_cache_write_ex(k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, tokens,
                      heads, head_dim, slots, k_cache, v_cache, num_pages, page_size, page_stride,
                      slot_stride, cache_head_stride, stream=None) -> int:
    return load().tg_cache_write_ex(k, k_token_stride, k_head_stride, v, v_token_stride,
                                    v_head_stride, tokens, heads, head_dim, slots, k_cache,
                                    v_cache, num_pages, page_size, page_stride, slot_stride,
                                    cache_head_stride, stream)


def tg_tree_mask(parents, tokens, starts, batch, words, mask, depth, stream=None) -> int:
    return load().tg_tree_mask(parents, tokens, starts, batch, words, mask, depth, stream)


def tg_tree_attention(args: tg_tree_attention_t, stream=None) -> int:
    return load().tg_tree_attention(ctypes.byref(args), stream)


def tg_tree_attention_workspace_size(head_dim: int) -> int:
    return load().tg_tree_attention_workspace_size(head_dim)


class CachePlan(NamedTuple):
    """What ``cache_plan`` writes (see tg_cache_plan): lengths, ring and packing after the call,
    each token's slot and position, and the status word (0, or TG_PLAN_* bits)."""
    lens: "torch.Tensor"        # (B,) int32
    ring: "torch.Tensor"        # (2,) int32
    starts: "torch.Tensor"      # (B + 1,) int32
    slots: "torch.Tensor"       # (tokens,) int64
    positions: "torch.Tensor"   # (tokens,) int32
    status: "torch.Tensor"      # (1,) int32


def _refuse(name, t, dtype, shape, index):
    """The error for a tensor that is not a contiguous ``dtype`` tensor of ``shape`` (None: any
    extent) on CUDA device ``index``."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if t.dim() != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _vector(name, t, dtype, n, index):
    """Check a contiguous one-dimensional tensor of n elements; returns its address.  (These
    checks are most of the time of a short call, hence one test of all that may be wrong.)"""
    if t.dtype is not dtype or t.get_device() != index or t.shape != (n,) \
            or not t.is_contiguous():
        _refuse(name, t, dtype, (n,), index)
    return t.data_ptr()


def _table(name, t, dtype, rows, index):
    """Check an int32 table with contiguous rows; returns (address, row stride, columns)."""
    if t.dtype is not dtype or t.get_device() != index or t.dim() != 2 or t.shape[0] != rows:
        _refuse(name, t, dtype, (rows, None), index)
    cols, (row, col) = t.shape[1], t.stride()
    if rows < 2:
        row = max(cols, 1)
    if (cols > 1 and col != 1) or row < cols:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return t.data_ptr(), row, cols


def _rows(name, t, dtype, shape, index):
    """Check a (tokens, heads, dim) tensor whose last dimension is contiguous; returns its
    strides."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape:
        _refuse(name, t, dtype, shape, index)
    strides = t.stride()
    if strides[2] != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return strides


def _same_layout(shape, a, b):
    """Whether strides a and b reach the same elements of ``shape``: those of dimensions with one
    element reach nothing (torch leaves there what a slice or a view happened to have)."""
    return a == b or all(x == y for n, x, y in zip(shape, a, b) if n > 1)


def _caches(k_cache, v_cache, dtype, index):
    """Check both caches: (pages, page size, heads, dim) tensors of the same shape and strides,
    the last dimension contiguous; returns shape and strides."""
    shape, strides = k_cache.shape, k_cache.stride()
    if len(shape) != 4:
        raise ValueError("k_cache must be (pages, page size, heads, dim)")
    if k_cache.dtype is not dtype or k_cache.get_device() != index:
        _refuse("k_cache", k_cache, dtype, shape, index)
    if v_cache.dtype is not dtype or v_cache.get_device() != index:
        _refuse("v_cache", v_cache, dtype, shape, index)
    if v_cache.shape != shape or not _same_layout(shape, v_cache.stride(), strides):
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    if strides[3] != 1:
        raise ValueError("the caches must have a contiguous last dimension")
    return shape, strides


def _device_index(name, t):
    index = t.get_device() if t.is_cuda else -1
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return index


def _call(torch, index, what, f, *args):
    """Call an entry point on the current stream of CUDA device ``index``; raise on a non-OK
    status."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)     # without a Stream object
    stream = raw(index) if raw else torch.cuda.current_stream(index).cuda_stream
    if torch.cuda.current_device() == index:
        st = f(*args, stream)
    else:
        with torch.cuda.device(index):
            st = f(*args, stream)
    if st != TG_OK:
        raise TgError(st, what)


def cache_plan(lens, add, ring, free_pages, block_tables, page_size, tokens, *, starts=None,
               offsets=None, out=None):
    """Pages, block-table entries, slots and positions for a change of the requests' lengths, on
    the GPU through tg_cache_plan.

    lens, add: (B,) int32, tokens in the cache and tokens to append (negative: to drop);
    free_pages: (num_pages,) int32 ring of free pages with ring = (head, count); block_tables:
    (B, max_pages) int32, extended in place; tokens: rows of the slot map.  starts (B + 1,) and
    offsets (tokens,) int32 pick the kept ones of a packed batch of drafted tokens; without
    them request b's max(add[b], 0) tokens are packed in order.  Returns a CachePlan, ``out``
    (its six tensors) if given; with ``starts`` given, its starts are a copy.
    """
    import torch
    index = _device_index("lens", lens)
    B, i32 = lens.numel(), torch.int32
    if out is None:
        def new(n):
            return torch.empty(n, dtype=i32, device=lens.device)
        out = CachePlan(new(B), new(2), new(B + 1),
                        torch.empty(tokens, dtype=torch.int64, device=lens.device), new(tokens),
                        new(1))
    elif not isinstance(out, CachePlan):
        out = CachePlan(*out)
    pages = free_pages.numel()
    table, stride, max_pages = _table("block_tables", block_tables, i32, B, index)
    _call(torch, index, "tg_cache_plan", load().tg_cache_plan,
          _vector("lens", lens, i32, B, index), _vector("add", add, i32, B, index), B,
          None if starts is None else _vector("starts", starts, i32, B + 1, index),
          None if offsets is None else _vector("offsets", offsets, i32, tokens, index), tokens,
          table, stride, max_pages, page_size,
          _vector("free_pages", free_pages, i32, pages, index), pages,
          _vector("ring", ring, i32, 2, index), _vector("out.lens", out.lens, i32, B, index),
          _vector("out.ring", out.ring, i32, 2, index),
          _vector("out.starts", out.starts, i32, B + 1, index),
          _vector("out.slots", out.slots, torch.int64, tokens, index),
          _vector("out.positions", out.positions, i32, tokens, index),
          _vector("out.status", out.status, i32, 1, index))
    return out


def cache_write(k, v, slots, k_cache, v_cache):
    """k_cache[slots] = k, v_cache[slots] = v on the GPU through tg_cache_write_ex.

    k, v: (tokens, heads, D), any 16-bit type (slices of a fused projection will do); slots:
    (tokens,) int64, -1 skips a token; caches: (pages, page size, heads, D), D 64 or 128, any
    strides (both the same) with a contiguous last dimension.  Returns the caches.
    """
    import torch
    index, dt = _device_index("k", k), k.dtype
    if dt.itemsize != 2:
        raise TypeError(f"k must have a 16-bit type, got {dt}")
    (pages, page, heads, dim), cs = _caches(k_cache, v_cache, dt, index)
    n = k.shape[0] if k.dim() else 0
    ks = _rows("k", k, dt, (n, heads, dim), index)
    vs = _rows("v", v, dt, (n, heads, dim), index)
    _call(torch, index, "tg_cache_write", load().tg_cache_write_ex, k.data_ptr(), ks[0], ks[1],
          v.data_ptr(), vs[0], vs[1], n, heads, dim, _vector("slots", slots, torch.int64, n, index),
          k_cache.data_ptr(), v_cache.data_ptr(), pages, page, cs[0], cs[1], cs[2])
    return k_cache, v_cache


def tree_mask(parents, starts, words, out=None):
    """Ancestor masks and depths of drafted token trees on the GPU through tg_tree_mask.

    parents: (tokens,) int32, index of a token's parent among its request's tokens or -1;
    starts: (B + 1,) int32.  Returns (mask, depth): (tokens, words) and (tokens,) int32, ``out``
    if given.
    """
    import torch
    index, n, i32 = _device_index("parents", parents), parents.numel(), torch.int32
    batch = starts.numel() - 1
    if batch < 0:
        raise ValueError("starts must have shape (batch + 1,)")
    if out is None:
        out = (torch.empty((n, max(words, 0)), dtype=i32, device=parents.device),
               torch.empty(n, dtype=i32, device=parents.device))
    mask = out[0]
    if mask.dtype is not i32 or mask.get_device() != index or mask.shape != (n, words) \
            or not mask.is_contiguous():
        _refuse("out[0]", mask, i32, (n, max(words, 0)), index)
    _call(torch, index, "tg_tree_mask", load().tg_tree_mask,
          _vector("parents", parents, i32, n, index), n,
          _vector("starts", starts, i32, batch + 1, index), batch, words, mask.data_ptr(),
          _vector("out[1]", out[1], i32, n, index))
    return out


def tree_attention(q, k, v, k_cache, v_cache, block_tables, lens, starts, mask=None, scale=0.0,
                   out=None, *, workspace=None, wait_limit_ns=0, inject=0):
    """Attention of drafted tokens over a paged cache and over one another on the GPU through
    tg_tree_attention.

    q: (tokens, heads, D), k and v: (tokens, kv_heads, D), fp16 or bf16, D 64 or 128, heads a
    multiple of kv_heads; caches: (pages, page size, kv_heads, D); block_tables: (B, max_pages)
    int32; lens: (B,) int32 cached tokens; starts: (B + 1,) int32 packing of the rows; mask:
    (tokens, words) int32 from tree_mask, None: a token sees those of its request up to itself
    (one token: decoding).  scale 0 means 1/sqrt(D).  workspace: uint8 tensor of at least
    tg_tree_attention_workspace_size(D) bytes, allocated if None; calls that may overlap need
    one each.  Returns ``out`` (allocated if None; rows outside every request are left as they
    are).
    """
    import torch
    index, dt = _device_index("q", q), q.dtype
    if dt is not torch.float16 and dt is not torch.bfloat16:
        raise TypeError(f"q must be float16 or bfloat16, got {dt}")
    (pages, page, kv_heads, dim), cs = _caches(k_cache, v_cache, dt, index)
    if q.dim() != 3 or kv_heads < 1 or q.shape[1] % kv_heads:
        raise ValueError(f"q must have shape (tokens, a multiple of {kv_heads}, {dim}), got "
                         f"{tuple(q.shape)}")
    n, heads, _ = q.shape
    qs = _rows("q", q, dt, (n, heads, dim), index)
    ks = _rows("k", k, dt, (n, kv_heads, dim), index)
    vs = _rows("v", v, dt, (n, kv_heads, dim), index)
    B, i32 = lens.numel(), torch.int32
    table, stride, max_pages = _table("block_tables", block_tables, i32, B, index)
    bits, mask_stride, words = None, 0, 0
    if mask is not None:
        bits, mask_stride, words = _table("mask", mask, i32, n, index)
        if words < 1:
            raise ValueError("mask must have at least one word")
    if out is None:
        out = q.new_empty((n, heads, dim))
    os = _rows("out", out, dt, (n, heads, dim), index)
    if workspace is None:
        workspace = q.new_empty(load()._tree_workspace_halves.get(dim, 0))
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on cuda:{index}")
    args = _TREE_ARGS.pack(
        TG_TYPE_BF16 if dt is torch.bfloat16 else TG_TYPE_FP16, n, B, kv_heads,
        heads // kv_heads, dim, scale, q.data_ptr(), qs[0], qs[1], k.data_ptr(), v.data_ptr(),
        ks[0], ks[1], k_cache.data_ptr(), v_cache.data_ptr(), pages, page, cs[0], cs[1], cs[2],
        table, stride, max_pages, _vector("lens", lens, i32, B, index),
        _vector("starts", starts, i32, B + 1, index), bits or 0, words, mask_stride,
        out.data_ptr(), os[0], os[1], workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), wait_limit_ns, inject, 1, vs[0], vs[1])
    _call(torch, index, "tg_tree_attention", load()._tree_attention_packed, args)
    return out
