"""Python binding of libmsa, the B200 (sm_100a) MiniMax Sparse Attention hot path.

Thin ctypes marshalling over the C ABI in include/msa.h: every function here only checks shapes,
allocates outputs / workspace through PyTorch and calls the same-named C entry point on the
current CUDA stream. All arithmetic runs in the library's CUDA kernels; there is no other path.
Importing works without a GPU (the library loads without one); calling needs a CUDA device.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import struct
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmsa.so")

MSA_OK, MSA_ERR_INVALID_ARG, MSA_ERR_UNSUPPORTED, MSA_ERR_WORKSPACE, MSA_ERR_CUDA, MSA_ERR_TIMEOUT, \
    MSA_ERR_DEVICE_CHECK = range(7)
(MSA_OP_INDEX_TOPK, MSA_OP_INDEX_TOPK_LSE, MSA_OP_ATTN_FWD, MSA_OP_DECODE, MSA_OP_KL, MSA_OP_ATTN_BWD,
 MSA_OP_LSE_IDX_LOCAL, MSA_OP_KL_DENSE, MSA_OP_TREE_INDEX_TOPK, MSA_OP_TREE_ATTN) = range(10)
MSA_BF16, MSA_F32 = range(2)


class MsaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {msa_status_string(code)} ({code})")
        self.code = code


class _Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("H_q", ctypes.c_int), ("H_kv", ctypes.c_int),
                ("d", ctypes.c_int), ("d_idx", ctypes.c_int), ("block_k", ctypes.c_int), ("topk", ctypes.c_int),
                ("scale", ctypes.c_float), ("scale_idx", ctypes.c_float)]


class _KeyRanges(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("tok0", ctypes.c_int32 * 2), ("ntok", ctypes.c_int32 * 2)]


class _RopeSeg(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("y_stride", ctypes.c_int64), ("inv_freq", ctypes.c_void_p), ("heads", ctypes.c_int),
                ("dim", ctypes.c_int), ("rot", ctypes.c_int), ("amp", ctypes.c_float)]


_ROPE_SEG = struct.Struct("@PPqqPiiif")  # the same, packed (a quarter of the time of filling the structure)
assert _ROPE_SEG.size == ctypes.sizeof(_RopeSeg)


class _Pages(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("cache_len", ctypes.c_void_p), ("num_pages", ctypes.c_int)]


class _Tree(ctypes.Structure):
    _fields_ = [("parents", ctypes.c_void_p), ("n_nodes", ctypes.c_void_p), ("T", ctypes.c_int)]


def _held(held, k_idx_local) -> _KeyRanges:
    """msa_key_ranges from a list of one or two (tok0, ntok) ranges, or from a single first token
    (one range spanning k_idx_local); the tokens must add up to k_idx_local's length."""
    rng = [(int(held), int(k_idx_local.shape[1]))] if isinstance(held, int) else [(int(a), int(n)) for a, n in held]
    if not 1 <= len(rng) <= 2 or sum(n for _, n in rng) != k_idx_local.shape[1]:
        raise ValueError(f"held ranges {rng} do not describe k_idx_local of {k_idx_local.shape[1]} tokens")
    h = _KeyRanges()
    h.n = len(rng)
    for x, (a, n) in enumerate(rng):
        h.tok0[x], h.ntok[x] = a, n
    return h


@dataclass
class MsaDims:
    """msa_dims: B sequences of N tokens (cache capacity for decode), H_q / H_kv heads, head dim d,
    index dim d_idx, KV block size block_k, topk past blocks per (query, group).
    scale / scale_idx of 0 mean 1/sqrt(d) and 1/sqrt(d_idx)."""
    B: int
    N: int
    H_q: int
    H_kv: int
    d: int
    d_idx: int
    block_k: int
    topk: int
    scale: float = 0.0
    scale_idx: float = 0.0

    def c(self) -> _Dims:
        return _Dims(self.B, self.N, self.H_q, self.H_kv, self.d, self.d_idx, self.block_k, self.topk,
                     self.scale, self.scale_idx)


@dataclass
class MsaPages:
    """msa_pages: where each sequence's cached tokens lie. page_table int32 [B, ceil(N / block_k)] (page ids of
    the pools, in position order) and cache_len int32 [B], on the device."""
    page_table: torch.Tensor
    cache_len: torch.Tensor


@dataclass
class MsaTree:
    """msa_tree: T drafted tokens per sequence. parents int32 [B, T] (-1: follows the cache; else a lower
    node number) and n_nodes int32 [B], on the device."""
    parents: torch.Tensor
    n_nodes: torch.Tensor


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmsa.so; raises if it has not been built (there is no fallback path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmsa.so not found at {LIB_PATH}; build it with "
                               "`python -m block_sparse_attention_idx_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, D, S = ctypes.c_void_p, ctypes.POINTER(_Dims), ctypes.c_size_t
        L.msa_workspace_size.argtypes = [ctypes.c_int, D, ctypes.POINTER(ctypes.c_size_t)]
        L.msa_index_topk.argtypes = [D, P, P, P, P, P, S, P]
        L.msa_sparse_attn_fwd.argtypes = [D, P, P, P, P, P, P, P, S, P]
        L.msa_sparse_attn_fwd_bf16.argtypes = [D, P, P, P, P, P, P, P, S, P]
        L.msa_sparse_attn_decode.argtypes = [D, P, P, P, P, P, P, P, P, P, P, S, P]
        L.msa_sparse_attn_decode_fp8idx.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, S, P]
        L.msa_quantize_e4m3_rows.argtypes = [P, ctypes.c_int64, ctypes.c_int, P, P, P]
        L.msa_kl_fwd_grad.argtypes = [D, P, P, P, P, P, P, P, ctypes.c_float, P, P, P, P, S, P]
        L.msa_kl_dense_fwd_grad.argtypes = [D, P, P, P, P, ctypes.c_float, P, P, P, P, P, S, P]
        L.msa_sparse_attn_bwd.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, S, P]
        I = ctypes.c_int
        H = ctypes.POINTER(_KeyRanges)
        L.msa_index_topk_local.argtypes = [D, P, P, H, P, P, P, S, P]
        L.msa_topk_merge.argtypes = [D, I, P, P, P, P]
        L.msa_lse_idx_local.argtypes = [D, P, P, H, P, P, P, S, P]
        L.msa_lse_combine.argtypes = [D, I, P, P, P]
        L.msa_sparse_attn_decode_noalloc.argtypes = [D, P, P, P, P, P, P, P, P, P]
        L.msa_sparse_attn_decode_noalloc.restype = ctypes.c_int
        L.msa_get_device_status.argtypes = [P, P]
        L.msa_decode_noalloc_status.argtypes = [P]
        L.msa_decode_noalloc_status.restype = ctypes.c_int
        L.msa_debug_set_wait_ns.argtypes = [ctypes.c_ulonglong]
        L.msa_debug_set_wait_ns.restype = None
        L.msa_debug_wait_probe.argtypes = [P, S, P]
        L.msa_debug_wait_probe.restype = ctypes.c_int
        L.msa_debug_exp2_fma.argtypes = [P, P, ctypes.c_int64, P]
        L.msa_debug_exp2_fma.restype = ctypes.c_int
        PG, TR, I64 = ctypes.POINTER(_Pages), ctypes.POINTER(_Tree), ctypes.c_int64
        for fn in ("msa_rope_fwd", "msa_rope_bwd"):
            getattr(L, fn).argtypes = [P, I, I64, P, I, I, I, P]
        L.msa_cache_append.argtypes = [D, PG, I, P, P, P, I, P, P, P, P, P, P, S, P]
        L.msa_cache_copy_pages.argtypes = [D, I, I, P, P, P, P, P, P, S, P]
        L.msa_tree_workspace_size.argtypes = [I, D, I, ctypes.POINTER(ctypes.c_size_t)]
        L.msa_tree_index_topk.argtypes = [D, PG, TR, P, P, P, P, P, P, S, P]
        L.msa_tree_sparse_attn.argtypes = [D, PG, TR, P, P, P, P, P, P, P, P, P, S, P]
        L.msa_tree_sparse_attn_bf16.argtypes = [D, PG, TR, P, P, P, P, P, P, P, P, P, S, P]
        L.msa_profile_enable.argtypes = [ctypes.c_int]
        L.msa_profile_enable.restype = None
        L.msa_profile_read.argtypes = [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_double),
                                       ctypes.POINTER(ctypes.c_int), ctypes.c_int]
        L.msa_profile_read.restype = ctypes.c_int
        L.msa_status_string.argtypes = [ctypes.c_int]
        L.msa_status_string.restype = ctypes.c_char_p
        L.msa_version.restype = ctypes.c_char_p
        for fn in ("msa_workspace_size", "msa_index_topk", "msa_sparse_attn_fwd", "msa_sparse_attn_fwd_bf16",
                   "msa_sparse_attn_decode",
                   "msa_sparse_attn_decode_fp8idx", "msa_quantize_e4m3_rows", "msa_kl_fwd_grad",
                   "msa_sparse_attn_bwd", "msa_index_topk_local", "msa_topk_merge", "msa_lse_idx_local",
                   "msa_lse_combine", "msa_get_device_status", "msa_kl_dense_fwd_grad", "msa_rope_fwd",
                   "msa_rope_bwd", "msa_cache_append", "msa_cache_copy_pages", "msa_tree_workspace_size",
                   "msa_tree_index_topk", "msa_tree_sparse_attn", "msa_tree_sparse_attn_bf16"):
            getattr(L, fn).restype = ctypes.c_int
        _lib = L
    return _lib


def msa_status_string(code: int) -> str:
    return lib().msa_status_string(code).decode()


def msa_version() -> str:
    return lib().msa_version().decode()


def _check(fn: str, code: int):
    if code != MSA_OK:
        raise MsaError(fn, code)


def msa_workspace_size(op: int, dims: MsaDims) -> int:
    n = ctypes.c_size_t(0)
    _check("msa_workspace_size", lib().msa_workspace_size(op, ctypes.byref(dims.c()), ctypes.byref(n)))
    return n.value


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, dev: torch.device):
    """The stream to launch on. The library launches on the current CUDA device, so the tensors'
    device must be the current one (and an explicit stream must belong to it)."""
    cur = torch.cuda.current_device()
    if dev.type != "cuda" or (dev.index is not None and dev.index != cur):
        raise ValueError(f"tensors are on {dev}, but the current CUDA device is cuda:{cur}; "
                         "call under torch.cuda.device(...)")
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream(cur).cuda_stream)
    s = stream
    if s.device.index != cur:
        raise ValueError(f"stream belongs to {s.device}, not to the current device cuda:{cur}")
    return ctypes.c_void_p(s.cuda_stream)


def _raw_stream(stream, dev: torch.device):
    """_stream for the short calls: the current stream's handle without a Stream object."""
    if stream is None and dev.index == torch.cuda.current_device():
        return torch._C._cuda_getCurrentRawStream(dev.index)
    return _stream(stream, dev)


def _need(t: torch.Tensor, name: str, shape, dtype, device):
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda and t.get_device() == device.index:
        return
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (the library takes device pointers), got {t.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")


def workspace(op: int, dims: MsaDims, device) -> torch.Tensor:
    """A device workspace buffer of the size `op` needs (256-byte aligned by the allocator)."""
    return torch.empty(max(msa_workspace_size(op, dims), 256), dtype=torch.uint8, device=device)


def _ws(ws, op: int, dims: MsaDims, dev) -> torch.Tensor:
    """The caller's workspace, checked (a contiguous uint8 CUDA tensor on the inputs' device; the
    library checks its size and alignment), or a new one for `op`."""
    if ws is None:
        return workspace(op, dims, dev)
    if ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.device != dev:
        raise ValueError(f"ws must be a contiguous uint8 tensor on {dev}")
    return ws


def msa_index_topk(dims: MsaDims, q_idx, k_idx, want_lse: bool = False, ws=None, stream=None):
    """Block selection. Returns blocks int32 [B,N,H_kv,topk+1] (and LSE_idx fp32 [B,N,H_kv])."""
    dev = q_idx.device
    _need(q_idx, "q_idx", (dims.B, dims.N, dims.H_kv, dims.d_idx), torch.bfloat16, dev)
    _need(k_idx, "k_idx", (dims.B, dims.N, dims.d_idx), torch.bfloat16, dev)
    blocks = torch.empty(dims.B, dims.N, dims.H_kv, dims.topk + 1, dtype=torch.int32, device=dev)
    lse = torch.empty(dims.B, dims.N, dims.H_kv, dtype=torch.float32, device=dev) if want_lse else None
    ws = _ws(ws, MSA_OP_INDEX_TOPK_LSE if want_lse else MSA_OP_INDEX_TOPK, dims, dev)
    _check("msa_index_topk", lib().msa_index_topk(ctypes.byref(dims.c()), _p(q_idx), _p(k_idx), _p(blocks), _p(lse),
                                                  _p(ws), ws.numel(), _stream(stream, dev)))
    return (blocks, lse) if want_lse else blocks


def msa_sparse_attn_fwd(dims: MsaDims, q, k, v, blocks, want_lse: bool = True, ws=None, stream=None,
                        out_dtype=torch.float32, out=None):
    """Sparse attention forward. Returns out [B,N,H_q,d] (fp32, or with out_dtype=torch.bfloat16 the
    same values rounded to bf16 by msa_sparse_attn_fwd_bf16) and LSE fp32 [B,N,H_q] (or None).
    `out` may be given (contiguous, of out_dtype) to be written in place."""
    dev = q.device
    _need(q, "q", (dims.B, dims.N, dims.H_q, dims.d), torch.bfloat16, dev)
    _need(k, "k", (dims.B, dims.N, dims.H_kv, dims.d), torch.bfloat16, dev)
    _need(v, "v", (dims.B, dims.N, dims.H_kv, dims.d), torch.bfloat16, dev)
    _need(blocks, "blocks", (dims.B, dims.N, dims.H_kv, dims.topk + 1), torch.int32, dev)
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"out_dtype must be torch.float32 or torch.bfloat16, not {out_dtype}")
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=dev)
    _need(out, "out", tuple(q.shape), out_dtype, dev)
    lse = torch.empty(dims.B, dims.N, dims.H_q, dtype=torch.float32, device=dev) if want_lse else None
    ws = _ws(ws, MSA_OP_ATTN_FWD, dims, dev)
    fn = "msa_sparse_attn_fwd" if out_dtype == torch.float32 else "msa_sparse_attn_fwd_bf16"
    _check(fn, getattr(lib(), fn)(ctypes.byref(dims.c()), _p(q), _p(k), _p(v), _p(blocks), _p(out), _p(lse), _p(ws),
                                  ws.numel(), _stream(stream, dev)))
    return out, lse


def _decode_io(dims: MsaDims, cache_len, q, q_idx, k_cache, v_cache, want_blocks, want_margin):
    dev = q.device
    _need(cache_len, "cache_len", (dims.B,), torch.int32, dev)
    _need(q, "q", (dims.B, dims.H_q, dims.d), torch.bfloat16, dev)
    _need(q_idx, "q_idx", (dims.B, dims.H_kv, dims.d_idx), torch.bfloat16, dev)
    _need(k_cache, "k_cache", (dims.B, dims.N, dims.H_kv, dims.d), torch.bfloat16, dev)
    _need(v_cache, "v_cache", (dims.B, dims.N, dims.H_kv, dims.d), torch.bfloat16, dev)
    out = torch.empty(q.shape, dtype=torch.float32, device=dev)
    blocks = torch.empty(dims.B, dims.H_kv, dims.topk + 1, dtype=torch.int32, device=dev) if want_blocks else None
    margin = torch.empty(dims.B, dims.H_kv, dtype=torch.float32, device=dev) if want_margin else None
    return out, blocks, margin


def msa_sparse_attn_decode(dims: MsaDims, cache_len, q, q_idx, k_cache, v_cache, k_idx_cache, want_blocks=True,
                           ws=None, stream=None, want_margin=False):
    """One decode step. dims.N is the cache capacity. Returns out fp32 [B,H_q,d] and the selected
    blocks int32 [B,H_kv,topk+1] (or None); with want_margin, also the cutoff margins fp32 [B,H_kv]."""
    out, blocks, margin = _decode_io(dims, cache_len, q, q_idx, k_cache, v_cache, want_blocks, want_margin)
    _need(k_idx_cache, "k_idx_cache", (dims.B, dims.N, dims.d_idx), torch.bfloat16, q.device)
    ws = _ws(ws, MSA_OP_DECODE, dims, q.device)
    _check("msa_sparse_attn_decode",
           lib().msa_sparse_attn_decode(ctypes.byref(dims.c()), _p(cache_len), _p(q), _p(q_idx), _p(k_cache),
                                        _p(v_cache), _p(k_idx_cache), _p(out), _p(blocks), _p(margin), _p(ws),
                                        ws.numel(), _stream(stream, q.device)))
    return (out, blocks, margin) if want_margin else (out, blocks)


def msa_quantize_e4m3_rows(x, codes=None, scale=None, stream=None):
    """Row-wise e4m3 quantisation of a bf16 tensor [..., n]: codes uint8 [..., n] (e4m3 bit
    patterns) and scales fp32 [...], scale = max|row| / 448."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous bf16 CUDA tensor")
    n = x.shape[-1]
    rows = x.numel() // n if n else 0
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _need(codes, "codes", tuple(x.shape), torch.uint8, x.device)
    _need(scale, "scale", tuple(x.shape[:-1]), torch.float32, x.device)
    _check("msa_quantize_e4m3_rows",
           lib().msa_quantize_e4m3_rows(_p(x), rows, n, _p(codes), _p(scale), _stream(stream, x.device)))
    return codes, scale


def msa_sparse_attn_decode_fp8idx(dims: MsaDims, cache_len, q, q_idx, k_cache, v_cache, k_idx_codes, k_idx_scale,
                                  want_blocks=True, ws=None, stream=None, want_margin=False):
    """Decode step with FP8 index scoring: the K_idx cache as e4m3 codes uint8 [B,N,d_idx] plus
    per-token scales fp32 [B,N] (msa_quantize_e4m3_rows). Returns as msa_sparse_attn_decode."""
    out, blocks, margin = _decode_io(dims, cache_len, q, q_idx, k_cache, v_cache, want_blocks, want_margin)
    _need(k_idx_codes, "k_idx_codes", (dims.B, dims.N, dims.d_idx), torch.uint8, q.device)
    _need(k_idx_scale, "k_idx_scale", (dims.B, dims.N), torch.float32, q.device)
    ws = _ws(ws, MSA_OP_DECODE, dims, q.device)
    _check("msa_sparse_attn_decode_fp8idx",
           lib().msa_sparse_attn_decode_fp8idx(ctypes.byref(dims.c()), _p(cache_len), _p(q), _p(q_idx),
                                               _p(k_cache), _p(v_cache), _p(k_idx_codes), _p(k_idx_scale),
                                               _p(out), _p(blocks), _p(margin), _p(ws), ws.numel(),
                                               _stream(stream, q.device)))
    return (out, blocks, margin) if want_margin else (out, blocks)


_HERE = contextlib.nullcontext()


def _on(stream):
    """Context in which new buffers belong to `stream` (the allocator reuses them in its order)."""
    return _HERE if stream is None else torch.cuda.stream(stream)


def msa_rope_inv_freq(rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                      orig_len: int = 0, device=None):
    """Inverse frequencies fp64 [rot / 2] and the amplitude, as (inv_freq, amp), for msa_rope_fwd / _bwd.

    base ** (-2 i / rot), and for contexts `factor` times longer than the trained one:
      None      as is
      "linear"  positions divided by factor (every frequency / factor)
      "ntk"     base * factor ** (rot / (rot - 2)): the lowest frequency is divided by factor, the highest kept
      "yarn"    frequencies that turn at least 32 times over orig_len tokens are kept, those that turn at most
                once are divided by factor, a linear ramp over i between (from pair 0 where none turns 32 times);
                amp = 0.1 ln(factor) + 1
    """
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and at least 2, got {rot}")
    if not (base > 1.0 and factor >= 1.0):
        raise ValueError(f"base must exceed 1 and factor be at least 1, got {base} and {factor}")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', not {scaling!r}")
    amp = 1.0
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** -(torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if orig_len < 1:
            raise ValueError("yarn needs orig_len, the trained context length")

        def pair(turns):  # the (fractional) pair that turns that often over orig_len
            return rot * math.log(orig_len / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        if orig_len <= 2 * math.pi:  # not even pair 0 turns more than once
            ramp = torch.ones_like(ramp)
        f = f / factor * ramp + f * (1 - ramp)
        amp = 0.1 * math.log(factor) + 1
    return f.to(device) if device is not None else f, amp


def _token_rows(t: torch.Tensor, name: str):
    """(tokens, heads, dim, elements between tokens) of a [..., heads, dim] tensor whose last two dims are
    contiguous and whose leading dims have one stride (a column slice of a projection's output qualifies)."""
    if t.dim() < 3:
        raise ValueError(f"{name}: expected [..., heads, dim], got {tuple(t.shape)}")
    heads, dim = t.shape[-2:]
    if t.is_contiguous():
        return t.numel() // (heads * dim) if heads * dim else 0, heads, dim, heads * dim
    if (dim > 1 and t.stride(-1) != 1) or (heads > 1 and t.stride(-2) != dim):
        raise ValueError(f"{name}: heads and dim must be contiguous")
    tokens, stride = 1, heads * dim
    for size, st in zip(reversed(t.shape[:-2]), reversed(t.stride()[:-2])):
        if size == 1:
            continue
        if tokens == 1:
            stride = st
        elif st != tokens * stride:
            raise ValueError(f"{name}: the leading dimensions must have one stride")
        tokens *= size
    return tokens, heads, dim, stride


_ROPE_TYPES = {torch.bfloat16: MSA_BF16, torch.float32: MSA_F32}


def _rope(fn: str, xs, freqs, positions, interleaved, outs, out_dtype, stream):
    xs, freqs = list(xs), list(freqs)
    if not xs or len(freqs) != len(xs) or (outs is not None and len(outs) != len(xs)):
        raise ValueError("need one (inv_freq, amp) pair, and with outs one output, per tensor")
    dev, dtype = xs[0].device, xs[0].dtype
    given = outs is not None
    if given:
        outs = list(outs)
        if out_dtype not in (None, outs[0].dtype):
            raise ValueError(f"outs are {outs[0].dtype}, out_dtype is {out_dtype}")
        out_dtype = outs[0].dtype
    elif out_dtype is None:
        out_dtype = dtype
    if dtype not in _ROPE_TYPES or out_dtype not in _ROPE_TYPES:
        raise ValueError(f"tensors must be torch.bfloat16 or torch.float32, got {dtype} -> {out_dtype}")
    seg, made, tokens, seen, idx = b"", [], None, None, xs[0].get_device()
    for i, (x, (f, amp)) in enumerate(zip(xs, freqs)):
        if not x.is_cuda:
            raise ValueError(f"xs[{i}] must be a CUDA tensor (the library takes device pointers), got {x.device}")
        if x.get_device() != idx or x.dtype is not dtype:
            raise ValueError(f"xs[{i}]: expected {dtype} on {dev}, got {x.dtype} on {x.device}")
        n, heads, dim, sx = _token_rows(x, f"xs[{i}]" if i else "xs[0]")
        if n != tokens:
            if tokens is not None:
                raise ValueError(f"xs[{i}] has {n} tokens, xs[0] has {tokens}")
            tokens = n
        if given:
            y = outs[i]
            if y.get_device() != idx or y.dtype is not out_dtype:
                raise ValueError(f"outs[{i}]: expected {out_dtype} on {dev}, got {y.dtype} on {y.device}")
            if x.shape != y.shape:
                raise ValueError(f"outs[{i}]: expected shape {tuple(x.shape)}, got {tuple(y.shape)}")
            sy = _token_rows(y, f"outs[{i}]")[3]
        else:
            if stream is not None:
                with torch.cuda.stream(stream):
                    y = x.new_empty(x.shape, dtype=out_dtype)
            elif out_dtype is dtype and sx == heads * dim:
                y = torch.empty_like(x)
            else:
                y = x.new_empty(x.shape, dtype=out_dtype)
            sy = heads * dim
        made.append(y)
        if f is not seen:
            if f.dim() != 1:
                raise ValueError("inv_freq must be fp64 [rot / 2]")
            _need(f, "inv_freq", f.shape, torch.float64, dev)
            seen, at, rot = f, f.data_ptr(), 2 * f.numel()
        seg += _ROPE_SEG.pack(x.data_ptr(), y.data_ptr(), sx, sy, at, heads, dim, rot, amp)
    if positions is not None:
        _need(positions, "positions", positions.shape, torch.int32, dev)
        if positions.numel() != tokens:
            raise ValueError(f"positions: expected {tokens} values, got {positions.numel()}")
    st = _raw_stream(stream, dev)
    if tokens:
        code = getattr(_lib or lib(), fn)(seg, len(xs), tokens, positions.data_ptr() if positions is not None else None,
                                          int(interleaved), _ROPE_TYPES[dtype], _ROPE_TYPES[out_dtype], st)
        if code:
            _check(fn, code)
    return made


def msa_rope_fwd(xs, freqs, positions=None, interleaved: bool = False, outs=None, out_dtype=None, stream=None):
    """Rotary positions of up to 8 tensors [..., heads, dim] (Q, K, Q_idx, K_idx of a step) in one launch.
    freqs: one (inv_freq fp64 [rot / 2], amp) per tensor, e.g. from msa_rope_inv_freq; positions int32 with one
    value per token (None: the token's index). Returns outs (new, contiguous, of out_dtype or the inputs' type,
    unless given; an input itself for in place)."""
    return _rope("msa_rope_fwd", xs, freqs, positions, interleaved, outs, out_dtype, stream)


def msa_rope_bwd(dys, freqs, positions=None, interleaved: bool = False, outs=None, out_dtype=None, stream=None):
    """Gradient of msa_rope_fwd with respect to its tensors: the upstream gradients (fp32, as the attention and
    KL gradients are, or bf16) through the transposed rotation."""
    return _rope("msa_rope_bwd", dys, freqs, positions, interleaved, outs, out_dtype, stream)


def _status_ws(ws, dev):
    """The optional status workspace of the cache operations."""
    if ws is not None and (ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.device != dev):
        raise ValueError(f"ws must be a contiguous uint8 tensor on {dev}")
    return _p(ws), 0 if ws is None else ws.numel()


def _pools(dims: MsaDims, pools, names, dev) -> int:
    """Checks the pools and returns their number of pages."""
    n = pools[0].shape[0] if pools[0].dim() else 0
    kv, idx = (n, dims.block_k, dims.H_kv, dims.d), (n, dims.block_k, dims.d_idx)
    for t, name in zip(pools, names):
        _need(t, name, idx if name.startswith("k_idx") else kv, torch.bfloat16, dev)
    return n


def _pages(dims: MsaDims, pages: MsaPages, num_pages: int, dev) -> _Pages:
    _need(pages.page_table, "page_table", (dims.B, -(-dims.N // dims.block_k)), torch.int32, dev)
    _need(pages.cache_len, "cache_len", (dims.B,), torch.int32, dev)
    return _Pages(pages.page_table.data_ptr(), pages.cache_len.data_ptr(), num_pages)


def msa_cache_append(dims: MsaDims, pages: MsaPages, k, v, k_idx, k_pool, v_pool, k_idx_pool, n_new, rows=None, ws=None,
                     stream=None):
    """Writes n_new[b] (int32 [B]) new tokens of each sequence behind its cache_len[b] cached ones: rows 0, 1, ...
    of k, v bf16 [B,T,H_kv,d] and k_idx bf16 [B,T,d_idx], or with rows (int32 [B,T_new]) row rows[b,i] for the
    i-th. cache_len is the caller's to advance. ws (256 bytes) receives the status word if given."""
    dev = k.device
    T = k.shape[1] if k.dim() == 4 else 0
    _need(k, "k", (dims.B, T, dims.H_kv, dims.d), torch.bfloat16, dev)
    _need(v, "v", (dims.B, T, dims.H_kv, dims.d), torch.bfloat16, dev)
    _need(k_idx, "k_idx", (dims.B, T, dims.d_idx), torch.bfloat16, dev)
    _need(n_new, "n_new", (dims.B,), torch.int32, dev)
    T_new = T
    if rows is not None:
        T_new = rows.shape[1] if rows.dim() == 2 else 0
        _need(rows, "rows", (dims.B, T_new), torch.int32, dev)
    n = _pools(dims, (k_pool, v_pool, k_idx_pool), ("k_pool", "v_pool", "k_idx_pool"), dev)
    pg = _pages(dims, pages, n, dev)
    wp, wn = (None, 0) if ws is None else _status_ws(ws, dev)
    code = (_lib or lib()).msa_cache_append(
        ctypes.byref(dims.c()), ctypes.byref(pg), T, k.data_ptr(), v.data_ptr(), k_idx.data_ptr(), T_new, n_new.data_ptr(),
        None if rows is None else rows.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), k_idx_pool.data_ptr(), wp, wn,
        _raw_stream(stream, dev))
    if code:
        _check("msa_cache_append", code)


def msa_cache_copy_pages(dims: MsaDims, src, dst, k_pool, v_pool, k_idx_pool, ws=None, stream=None):
    """Page dst[i] of the three pools becomes a copy of page src[i]. src and dst are int32 CUDA tensors [n], or
    sequences of page numbers, which are then checked here: in range, dst distinct, and no page in both."""
    dev = k_pool.device
    n_pages = _pools(dims, (k_pool, v_pool, k_idx_pool), ("k_pool", "v_pool", "k_idx_pool"), dev)
    if not torch.is_tensor(src) and not torch.is_tensor(dst):
        src, dst = [int(p) for p in src], [int(p) for p in dst]
        if len(src) != len(dst):
            raise ValueError(f"src has {len(src)} pages, dst {len(dst)}")
        if any(not 0 <= p < n_pages for p in src + dst):
            raise ValueError(f"page numbers must be in [0, {n_pages})")
        if len(set(dst)) != len(dst) or set(dst) & set(src):
            raise ValueError("dst pages must be distinct and none of them a src page")
        with _on(stream):
            src = torch.tensor(src, dtype=torch.int32, device=dev)
            dst = torch.tensor(dst, dtype=torch.int32, device=dev)
    elif not (torch.is_tensor(src) and torch.is_tensor(dst)):
        raise ValueError("src and dst must both be tensors or both sequences")
    _need(src, "src", (src.numel(),), torch.int32, dev)
    _need(dst, "dst", (src.numel(),), torch.int32, dev)
    wp, wn = (None, 0) if ws is None else _status_ws(ws, dev)
    code = (_lib or lib()).msa_cache_copy_pages(
        ctypes.byref(dims.c()), n_pages, src.numel(), src.data_ptr() or None, dst.data_ptr() or None, k_pool.data_ptr(),
        v_pool.data_ptr(), k_idx_pool.data_ptr(), wp, wn, _raw_stream(stream, dev))
    if code:
        _check("msa_cache_copy_pages", code)


def msa_tree_workspace_size(op: int, dims: MsaDims, T: int) -> int:
    n = ctypes.c_size_t(0)
    _check("msa_tree_workspace_size", lib().msa_tree_workspace_size(op, ctypes.byref(dims.c()), T, ctypes.byref(n)))
    return n.value


def tree_workspace(op: int, dims: MsaDims, T: int, device) -> torch.Tensor:
    """A device workspace buffer of the size a tree operation needs (256-byte aligned by the allocator)."""
    return torch.empty((max(msa_tree_workspace_size(op, dims, T), 256),), dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=256)
def _tree_ws_size(op, B, N, H_q, H_kv, d, d_idx, block_k, topk, T, device) -> int:
    """msa_tree_workspace_size for sizes seen before on a device (it depends on the SM count of the current one)."""
    if device != torch.cuda.current_device():
        raise ValueError(f"tensors are on cuda:{device}, but the current CUDA device is cuda:{torch.cuda.current_device()}; "
                         "call under torch.cuda.device(...)")
    return max(256, msa_tree_workspace_size(op, MsaDims(B, N, H_q, H_kv, d, d_idx, block_k, topk), T))


def _tree(dims: MsaDims, tree: MsaTree, dev):
    T = tree.parents.shape[1] if tree.parents.dim() == 2 else 0
    _need(tree.parents, "parents", (dims.B, T), torch.int32, dev)
    _need(tree.n_nodes, "n_nodes", (dims.B,), torch.int32, dev)
    return T, _Tree(tree.parents.data_ptr(), tree.n_nodes.data_ptr(), T)


def _tree_ws(ws, op: int, dims: MsaDims, T: int, like: torch.Tensor) -> torch.Tensor:
    """The caller's workspace, checked, or a new one next to `like`, on the current stream."""
    if ws is None:
        n = _tree_ws_size(op, dims.B, dims.N, dims.H_q, dims.H_kv, dims.d, dims.d_idx, dims.block_k, dims.topk, T, like.get_device())
        return like.new_empty(n, dtype=torch.uint8)
    if ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.device != like.device:
        raise ValueError(f"ws must be a contiguous uint8 tensor on {like.device}")
    return ws


def msa_tree_index_topk(dims: MsaDims, pages: MsaPages, tree: MsaTree, q_idx, k_idx, k_idx_pool, want_margin=False, ws=None,
                        stream=None):
    """Block selection of drafted tokens over a paged cache: q_idx bf16 [B,T,H_kv,d_idx], the drafted k_idx bf16
    [B,T,d_idx], the cache's k_idx_pool. dims.N is the page table's capacity. Returns blocks int32
    [B,T,H_kv,topk+1]; with want_margin, also the cutoff margins fp32 [B,T,H_kv]."""
    dev = q_idx.device
    T, tr = _tree(dims, tree, dev)
    _need(q_idx, "q_idx", (dims.B, T, dims.H_kv, dims.d_idx), torch.bfloat16, dev)
    _need(k_idx, "k_idx", (dims.B, T, dims.d_idx), torch.bfloat16, dev)
    pg = _pages(dims, pages, _pools(dims, (k_idx_pool,), ("k_idx_pool",), dev), dev)
    with _on(stream):
        ws = _tree_ws(ws, MSA_OP_TREE_INDEX_TOPK, dims, T, q_idx)
        blocks = q_idx.new_empty((dims.B, T, dims.H_kv, dims.topk + 1), dtype=torch.int32)
        margin = q_idx.new_empty((dims.B, T, dims.H_kv), dtype=torch.float32) if want_margin else None
    code = (_lib or lib()).msa_tree_index_topk(
        ctypes.byref(dims.c()), ctypes.byref(pg), ctypes.byref(tr), q_idx.data_ptr(), k_idx.data_ptr(), k_idx_pool.data_ptr(),
        blocks.data_ptr(), None if margin is None else margin.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(stream, dev))
    if code:
        _check("msa_tree_index_topk", code)
    return (blocks, margin) if want_margin else blocks


def msa_tree_sparse_attn(dims: MsaDims, pages: MsaPages, tree: MsaTree, q, k, v, k_pool, v_pool, blocks, want_lse=False,
                         out_dtype=torch.float32, out=None, ws=None, stream=None):
    """Sparse attention of drafted tokens: q bf16 [B,T,H_q,d], the drafted k, v bf16 [B,T,H_kv,d], the cache's
    pools, blocks from msa_tree_index_topk. Returns out [B,T,H_q,d] (fp32, or bf16 by
    msa_tree_sparse_attn_bf16) and LSE fp32 [B,T,H_q] (or None). `out` may be given to be written in place."""
    dev = q.device
    T, tr = _tree(dims, tree, dev)
    _need(q, "q", (dims.B, T, dims.H_q, dims.d), torch.bfloat16, dev)
    _need(k, "k", (dims.B, T, dims.H_kv, dims.d), torch.bfloat16, dev)
    _need(v, "v", (dims.B, T, dims.H_kv, dims.d), torch.bfloat16, dev)
    _need(blocks, "blocks", (dims.B, T, dims.H_kv, dims.topk + 1), torch.int32, dev)
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"out_dtype must be torch.float32 or torch.bfloat16, not {out_dtype}")
    pg = _pages(dims, pages, _pools(dims, (k_pool, v_pool), ("k_pool", "v_pool"), dev), dev)
    given = out is not None
    with _on(stream):
        ws = _tree_ws(ws, MSA_OP_TREE_ATTN, dims, T, q)
        if not given:
            out = torch.empty_like(q) if out_dtype is torch.bfloat16 else q.new_empty(q.shape, dtype=out_dtype)
        lse = q.new_empty((dims.B, T, dims.H_q), dtype=torch.float32) if want_lse else None
    if given:
        _need(out, "out", tuple(q.shape), out_dtype, dev)
    fn = "msa_tree_sparse_attn" if out_dtype is torch.float32 else "msa_tree_sparse_attn_bf16"
    code = getattr(_lib or lib(), fn)(
        ctypes.byref(dims.c()), ctypes.byref(pg), ctypes.byref(tr), q.data_ptr(), k.data_ptr(), v.data_ptr(), k_pool.data_ptr(),
        v_pool.data_ptr(), blocks.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel(),
        _raw_stream(stream, dev))
    if code:
        _check(fn, code)
    return out, lse


def msa_sparse_attn_decode_noalloc(dims: MsaDims, cache_len, q, q_idx, k_cache, v_cache, k_idx_cache, out=None,
                                   blocks=None, stream=None):
    """Decode step through the allocation-free entry point (the library's static 16 MiB device scratch
    instead of a workspace). For callers that cannot allocate device memory while decoding; outputs may
    be passed in preallocated. Calls on one device share the scratch and must not overlap on the GPU."""
    dev = q.device
    _need(cache_len, "cache_len", (dims.B,), torch.int32, dev)
    _need(q, "q", (dims.B, dims.H_q, dims.d), torch.bfloat16, dev)
    _need(q_idx, "q_idx", (dims.B, dims.H_kv, dims.d_idx), torch.bfloat16, dev)
    _need(k_cache, "k_cache", (dims.B, dims.N, dims.H_kv, dims.d), torch.bfloat16, dev)
    _need(v_cache, "v_cache", (dims.B, dims.N, dims.H_kv, dims.d), torch.bfloat16, dev)
    _need(k_idx_cache, "k_idx_cache", (dims.B, dims.N, dims.d_idx), torch.bfloat16, dev)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=dev)
    _need(out, "out", (dims.B, dims.H_q, dims.d), torch.float32, dev)
    if blocks is not None:
        _need(blocks, "blocks", (dims.B, dims.H_kv, dims.topk + 1), torch.int32, dev)
    _check("msa_sparse_attn_decode_noalloc",
           lib().msa_sparse_attn_decode_noalloc(ctypes.byref(dims.c()), _p(cache_len), _p(q), _p(q_idx),
                                                _p(k_cache), _p(v_cache), _p(k_idx_cache), _p(out), _p(blocks),
                                                _stream(stream, dev)))
    return out, blocks


def msa_sparse_attn_bwd(dims: MsaDims, q, k, v, blocks, out, lse, dout, ws=None, stream=None):
    """Backward of the sparse attention with the selection fixed. out / lse are the forward's
    (fp32), dout bf16 [B,N,H_q,d]. Returns dq fp32 [B,N,H_q,d], dk and dv fp32 [B,N,H_kv,d]."""
    dev = q.device
    _need(q, "q", (dims.B, dims.N, dims.H_q, dims.d), torch.bfloat16, dev)
    _need(k, "k", (dims.B, dims.N, dims.H_kv, dims.d), torch.bfloat16, dev)
    _need(v, "v", (dims.B, dims.N, dims.H_kv, dims.d), torch.bfloat16, dev)
    _need(blocks, "blocks", (dims.B, dims.N, dims.H_kv, dims.topk + 1), torch.int32, dev)
    _need(out, "out", (dims.B, dims.N, dims.H_q, dims.d), torch.float32, dev)
    _need(lse, "lse", (dims.B, dims.N, dims.H_q), torch.float32, dev)
    _need(dout, "dout", (dims.B, dims.N, dims.H_q, dims.d), torch.bfloat16, dev)
    dq = torch.empty(dims.B, dims.N, dims.H_q, dims.d, dtype=torch.float32, device=dev)
    dk = torch.empty(dims.B, dims.N, dims.H_kv, dims.d, dtype=torch.float32, device=dev)
    dv = torch.empty(dims.B, dims.N, dims.H_kv, dims.d, dtype=torch.float32, device=dev)
    ws = _ws(ws, MSA_OP_ATTN_BWD, dims, dev)
    _check("msa_sparse_attn_bwd",
           lib().msa_sparse_attn_bwd(ctypes.byref(dims.c()), _p(q), _p(k), _p(v), _p(blocks), _p(out), _p(lse),
                                     _p(dout), _p(dq), _p(dk), _p(dv), _p(ws), ws.numel(), _stream(stream, dev)))
    return dq, dk, dv


def msa_index_topk_local(dims: MsaDims, q_idx, k_idx_local, held, ws=None, stream=None):
    """This rank's candidates for the sequence-parallel selection: k_idx_local bf16 [B, ntok, d_idx]
    holds the tokens of `held`, one or two (tok0, ntok) ranges in order (or a single tok0: one range
    of ntok tokens). Returns (raw block maxima fp32, block ids int32), each [B, N, H_kv, topk], best
    first, -inf / -1 padded."""
    dev = q_idx.device
    _need(q_idx, "q_idx", (dims.B, dims.N, dims.H_kv, dims.d_idx), torch.bfloat16, dev)
    ntok = k_idx_local.shape[1]
    _need(k_idx_local, "k_idx_local", (dims.B, ntok, dims.d_idx), torch.bfloat16, dev)
    h = _held(held, k_idx_local)
    cs = torch.empty(dims.B, dims.N, dims.H_kv, dims.topk, dtype=torch.float32, device=dev)
    ci = torch.empty(dims.B, dims.N, dims.H_kv, dims.topk, dtype=torch.int32, device=dev)
    ws = _ws(ws, MSA_OP_INDEX_TOPK, dims, dev)
    _check("msa_index_topk_local",
           lib().msa_index_topk_local(ctypes.byref(dims.c()), _p(q_idx), _p(k_idx_local), ctypes.byref(h), _p(cs),
                                      _p(ci), _p(ws), ws.numel(), _stream(stream, dev)))
    return cs, ci


def msa_topk_merge(dims: MsaDims, cand_scores, cand_ids, stream=None):
    """Merge of P ranks' candidates [P, B, N, H_kv, topk] into blocks int32 [B, N, H_kv, topk+1]."""
    P = cand_scores.shape[0]
    dev = cand_scores.device
    _need(cand_scores, "cand_scores", (P, dims.B, dims.N, dims.H_kv, dims.topk), torch.float32, dev)
    _need(cand_ids, "cand_ids", (P, dims.B, dims.N, dims.H_kv, dims.topk), torch.int32, dev)
    blocks = torch.empty(dims.B, dims.N, dims.H_kv, dims.topk + 1, dtype=torch.int32, device=dev)
    _check("msa_topk_merge", lib().msa_topk_merge(ctypes.byref(dims.c()), P, _p(cand_scores), _p(cand_ids), _p(blocks),
                                                  _stream(stream, dev)))
    return blocks


def msa_lse_idx_local(dims: MsaDims, q_idx, k_idx_local, held, blocks, ws=None, stream=None):
    """This rank's (max, exp-sum) of the index scores over the selected tokens it holds (`held` as in
    msa_index_topk_local): fp32 [B, N, H_kv, 2]."""
    dev = q_idx.device
    ntok = k_idx_local.shape[1]
    _need(q_idx, "q_idx", (dims.B, dims.N, dims.H_kv, dims.d_idx), torch.bfloat16, dev)
    _need(k_idx_local, "k_idx_local", (dims.B, ntok, dims.d_idx), torch.bfloat16, dev)
    _need(blocks, "blocks", (dims.B, dims.N, dims.H_kv, dims.topk + 1), torch.int32, dev)
    h = _held(held, k_idx_local)
    ml = torch.empty(dims.B, dims.N, dims.H_kv, 2, dtype=torch.float32, device=dev)
    ws = _ws(ws, MSA_OP_LSE_IDX_LOCAL, dims, dev)
    _check("msa_lse_idx_local",
           lib().msa_lse_idx_local(ctypes.byref(dims.c()), _p(q_idx), _p(k_idx_local), ctypes.byref(h), _p(blocks),
                                   _p(ml), _p(ws), ws.numel(), _stream(stream, dev)))
    return ml


def msa_lse_combine(dims: MsaDims, ml, stream=None):
    """Eq (16) over the P ranks' pairs ml [P, B, N, H_kv, 2]: LSE_idx fp32 [B, N, H_kv]."""
    P = ml.shape[0]
    _need(ml, "ml", (P, dims.B, dims.N, dims.H_kv, 2), torch.float32, ml.device)
    lse = torch.empty(dims.B, dims.N, dims.H_kv, dtype=torch.float32, device=ml.device)
    _check("msa_lse_combine", lib().msa_lse_combine(ctypes.byref(dims.c()), P, _p(ml), _p(lse), _stream(stream, ml.device)))
    return lse


def msa_kl_fwd_grad(dims: MsaDims, q, k, q_idx, k_idx, blocks, lse, lse_idx=None, grad_scale: float = 1.0, ws=None,
                    stream=None):
    """KL alignment. Returns loss fp32 [1], dq_idx fp32 [B,N,H_kv,d_idx], dk_idx fp32 [B,N,d_idx]."""
    dev = q.device
    _need(q, "q", (dims.B, dims.N, dims.H_q, dims.d), torch.bfloat16, dev)
    _need(k, "k", (dims.B, dims.N, dims.H_kv, dims.d), torch.bfloat16, dev)
    _need(q_idx, "q_idx", (dims.B, dims.N, dims.H_kv, dims.d_idx), torch.bfloat16, dev)
    _need(k_idx, "k_idx", (dims.B, dims.N, dims.d_idx), torch.bfloat16, dev)
    _need(blocks, "blocks", (dims.B, dims.N, dims.H_kv, dims.topk + 1), torch.int32, dev)
    _need(lse, "lse", (dims.B, dims.N, dims.H_q), torch.float32, dev)
    if lse_idx is not None:
        _need(lse_idx, "lse_idx", (dims.B, dims.N, dims.H_kv), torch.float32, dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    dq = torch.empty(dims.B, dims.N, dims.H_kv, dims.d_idx, dtype=torch.float32, device=dev)
    dk = torch.empty(dims.B, dims.N, dims.d_idx, dtype=torch.float32, device=dev)
    ws = _ws(ws, MSA_OP_KL, dims, dev)
    _check("msa_kl_fwd_grad",
           lib().msa_kl_fwd_grad(ctypes.byref(dims.c()), _p(q), _p(k), _p(q_idx), _p(k_idx), _p(blocks), _p(lse),
                                 _p(lse_idx), ctypes.c_float(grad_scale), _p(loss), _p(dq), _p(dk), _p(ws),
                                 ws.numel(), _stream(stream, dev)))
    return loss, dq, dk


def msa_kl_dense_fwd_grad(dims: MsaDims, q, k, q_idx, k_idx, grad_scale: float = 1.0, want_lse: bool = False,
                          ws=None, stream=None):
    """Dense warm-up KL (every causal block selected). Returns (loss fp32 [1], dq_idx [B,N,H_kv,d_idx],
    dk_idx [B,N,d_idx]) and, with want_lse, the teacher LSE fp32 [B,N,H_q]."""
    dev = q.device
    _need(q, "q", (dims.B, dims.N, dims.H_q, dims.d), torch.bfloat16, dev)
    _need(k, "k", (dims.B, dims.N, dims.H_kv, dims.d), torch.bfloat16, dev)
    _need(q_idx, "q_idx", (dims.B, dims.N, dims.H_kv, dims.d_idx), torch.bfloat16, dev)
    _need(k_idx, "k_idx", (dims.B, dims.N, dims.d_idx), torch.bfloat16, dev)
    ws = _ws(ws, MSA_OP_KL_DENSE, dims, dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    dq = torch.empty(dims.B, dims.N, dims.H_kv, dims.d_idx, dtype=torch.float32, device=dev)
    dk = torch.empty(dims.B, dims.N, dims.d_idx, dtype=torch.float32, device=dev)
    lse = torch.empty(dims.B, dims.N, dims.H_q, dtype=torch.float32, device=dev) if want_lse else None
    _check("msa_kl_dense_fwd_grad",
           lib().msa_kl_dense_fwd_grad(ctypes.byref(dims.c()), _p(q), _p(k), _p(q_idx), _p(k_idx),
                                       ctypes.c_float(grad_scale), _p(loss), _p(dq), _p(dk), _p(lse), _p(ws),
                                       ws.numel(), _stream(stream, dev)))
    return (loss, dq, dk, lse) if want_lse else (loss, dq, dk)


def msa_profile_enable(on: bool = True) -> None:
    """Record CUDA events around every kernel the library launches (on the launching stream)."""
    lib().msa_profile_enable(1 if on else 0)


def msa_profile_read() -> dict:
    """{kernel name: (total ms, launches)} since the last read; synchronises on the events."""
    cap = 64
    names = (ctypes.c_char_p * cap)()
    ms = (ctypes.c_double * cap)()
    n = (ctypes.c_int * cap)()
    k = lib().msa_profile_read(names, ms, n, cap)
    if k < 0:
        raise MsaError("msa_profile_read", MSA_ERR_CUDA)
    return {names[x].decode(): (ms[x], n[x]) for x in range(k)}


def msa_get_device_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronise the stream and return the status code recorded by the last call using `ws`."""
    return lib().msa_get_device_status(_p(ws), _stream(stream, ws.device))


def msa_decode_noalloc_status(stream=None) -> int:
    """Synchronise the stream and return the status code of the last allocation-free decode call on
    the current device (its status word lives in the library's static scratch array)."""
    return lib().msa_decode_noalloc_status(_stream(stream, torch.device("cuda", torch.cuda.current_device())))


def msa_debug_set_wait_ns(ns: int) -> None:
    """Test hook: time limit (ns) of every bounded device wait of later calls (0: the 2 s default)."""
    lib().msa_debug_set_wait_ns(int(ns))


def msa_debug_exp2_fma(x: torch.Tensor, stream=None) -> torch.Tensor:
    """2^x by the library's FMA-pipe exponential (fp32 device tensor in, same shape out)."""
    if not (x.is_cuda and x.dtype == torch.float32 and x.is_contiguous()):
        raise ValueError("msa_debug_exp2_fma: x must be a contiguous float32 CUDA tensor")
    y = torch.empty_like(x)
    _check("msa_debug_exp2_fma", lib().msa_debug_exp2_fma(_p(x), _p(y), x.numel(), _stream(stream, x.device)))
    return y


def msa_debug_wait_probe(ws: torch.Tensor, stream=None) -> None:
    """Test hook: enqueue the launch whose bounded wait can only run out (status MSA_ERR_TIMEOUT).
    ws: a uint8 CUDA tensor of at least 256 + 4096 bytes."""
    if ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.device.type != "cuda":
        raise ValueError("ws must be a contiguous uint8 CUDA tensor")
    _check("msa_debug_wait_probe", lib().msa_debug_wait_probe(_p(ws), ws.numel(), _stream(stream, ws.device)))


__all__ = ["MsaDims", "MsaError", "msa_workspace_size", "msa_index_topk", "msa_sparse_attn_fwd",
           "msa_sparse_attn_decode", "msa_sparse_attn_decode_noalloc", "msa_sparse_attn_decode_fp8idx",
           "msa_quantize_e4m3_rows", "msa_kl_fwd_grad", "msa_sparse_attn_bwd", "msa_index_topk_local",
           "msa_topk_merge", "msa_lse_idx_local", "msa_lse_combine", "msa_get_device_status", "msa_status_string",
           "msa_version", "msa_profile_enable", "msa_profile_read", "msa_decode_noalloc_status",
           "msa_debug_set_wait_ns", "msa_debug_wait_probe", "msa_debug_exp2_fma", "msa_kl_dense_fwd_grad", "MsaPages", "MsaTree",
           "msa_rope_inv_freq", "msa_rope_fwd", "msa_rope_bwd", "msa_cache_append", "msa_cache_copy_pages",
           "msa_tree_workspace_size", "msa_tree_index_topk", "msa_tree_sparse_attn", "tree_workspace", "workspace",
           "lib", "LIB_PATH"]
