"""sl8 -- W8A8 INT8 attention for NVIDIA GB300 (sm_103a).

A thin Python binding over the C ABI of ``libsl8.so`` (declared in
``include/sl8.h``).  This module only marshals arguments: it takes torch CUDA
tensors, allocates outputs and workspaces with torch, and calls the library on
torch's current stream.  Every step of the computation runs in the library's
CUDA kernels; there is no CPU or PyTorch fallback, and a missing library is an
error.

Operations (the "SuperL8" README, github.com/jajmangold/superl8): symmetric
per-row int8 quantisation ("Supporting kernels" table, quant_rowwise; "Quantization"
table, per-row int8 with K-smoothing), W8A8 INT8 FlashAttention prefill, dense and
varlen ("Attention kernels" table, attn_int8_fwd / attn_varlen_fwd; "Quick start"
layouts) and split-KV decode over an int8 KV cache ("Attention kernels" table,
attn_decode, int8-V variant); and what serving from the paged int8 cache takes ("Engine"
table, "Paged KV cache" row): the page plan of a step, the rotary append, page bounds,
page selection and decode over page lists; and that cache in 4 bits: the rotary append to it,
reading it back as dense keys and values, and decode attention over it.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsl8.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "sl8.h")

SL8_F16, SL8_BF16, SL8_F32, SL8_I8 = 0, 1, 2, 3
SL8_OK, SL8_ERR_INVALID_ARG, SL8_ERR_UNSUPPORTED, SL8_ERR_WORKSPACE, SL8_ERR_CUDA, SL8_ERR_TIMEOUT, \
    SL8_ERR_DEVICE_ARG = range(7)

_DTYPES = {torch.float16: SL8_F16, torch.bfloat16: SL8_BF16, torch.float32: SL8_F32, torch.int8: SL8_I8}
_TORCH_DTYPES = {v: k for k, v in _DTYPES.items()}


class SL8Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = f"{what}: {status_string(status)} (status {status})"
        if status == SL8_ERR_CUDA:
            try:
                msg += ": " + lib().sl8_last_cuda_error_string().decode()
            except Exception:  # noqa: BLE001 - used while formatting another error
                pass
        super().__init__(msg)


_lock = threading.Lock()
_lib = None

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_SZ = ctypes.c_size_t
_U64 = ctypes.c_uint64

_SIGNATURES = {
    "sl8_status_string": (ctypes.c_char_p, [_INT]),
    "sl8_last_cuda_error_string": (ctypes.c_char_p, []),
    "sl8_version": (_INT, []),
    "sl8_quant_rowwise": (_INT, [_P, _INT, _I64, _I32, _I64, _P, _I64, _P, _P, _P]),
    "sl8_k_channel_mean_workspace_size": (_SZ, [_I32, _I32, _I32, _I32]),
    "sl8_k_channel_mean": (_INT, [_P, _INT, _I32, _I32, _I32, _I32, _P, _I64, _P, _P, _SZ, _P]),
    "sl8_attn_int8_fwd_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I64]),
    "sl8_attn_int8_fwd": (_INT, [_P, _P, _P, _INT, _INT, _I32, _I32, _I32, _I32, _I32, _P, _I64, _INT, _INT, _P,
                                 _INT, _P, _P, _SZ, _P]),
    "sl8_attn_int8_fwd_chunk_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32]),
    "sl8_attn_int8_fwd_chunk": (_INT, [_P, _P, _P, _INT, _INT, _I32, _I32, _I32, _I32, _I32, _I32, _INT, _INT, _P,
                                       _INT, _P, _P, _SZ, _P]),
    "sl8_attn_int8_fwd_chunk_cache": (_INT, [_P, _INT, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _INT,
                                             _P, _INT, _P, _P, _SZ, _P]),
    "sl8_attn_int8_qk_logits_debug": (_INT, [_P, _P, _INT, _I32, _I32, _I32, _I32, _I32, _P, _I64, _INT, _I32, _I32,
                                             _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "sl8_attn_w8a8_fwd": (_INT, [_P, _P, _P, _INT, _INT, _I32, _I32, _I32, _I32, _I32, _P, _I64, _INT, _INT, _I32,
                                 _I32, ctypes.c_float, _P, _INT, _P, _P, _SZ, _P]),
    "sl8_attn_w8a8_qk_logits_debug": (_INT, [_P, _P, _INT, _I32, _I32, _I32, _I32, _I32, _P, _I64, _INT, _I32,
                                             _I32, ctypes.c_float, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "sl8_attn_decode_num_splits": (_I32, [_I32, _I32, _I32, _I32, _I32]),
    "sl8_attn_decode_split_size": (_I32, [_I32, _I32, _I32, _I32, _I32]),
    "sl8_attn_decode_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32]),
    "sl8_attn_decode_lse_offset": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32]),
    "sl8_attn_int8_decode_splitkv": (_INT, [_P, _INT, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _P,
                                            _P, _P]),
    "sl8_attn_decode_verify_num_splits": (_I32, [_I32, _I32, _I32, _I32, _I32, _I32, _I32]),
    "sl8_attn_int8_decode_verify": (_INT, [_P, _INT, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32,
                                           _I32, _P, _P, _P, _INT, _P, _P]),
    "sl8_attn_int8_decode_splitkv_f16v": (_INT, [_P, _INT, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _P,
                                                 _P, _P]),
    "sl8_attn_int8_paged_decode_splitkv": (_INT, [_P, _INT, _P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _I32, _I32,
                                                  _I32, _I32, _I32, _P, _P, _P]),
    "sl8_attn_decode_combine": (_INT, [_P, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _INT, _P, _P]),
    "sl8_attn_int8_decode_logits_debug": (_INT, [_P, _INT, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _P,
                                                 _P, _P, _P, _P]),
    "sl8_attn_int8_decode_noalloc": (_INT, [_P, _INT, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _INT,
                                            _P]),
    "sl8_paged_assign": (_INT, [_P, _P, _P, _I32, _I32, _I32, _P, _P, _I32, _P, _P, _I32, _P, _P, _P, _P, _P, _P]),
    "sl8_rope_append": (_INT, [_P, _P, _P, _INT, _I64, _I64, _I64, _I32, _I32, _I32, _I32, _P, _I32, _I32, _P,
                               ctypes.c_char_p, _INT, _P, _I64, _P, _P, _P, _P, _P, _I32, _I32, _P]),
    "sl8_page_bounds": (_INT, [_P, _P, _I32, _I32, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _P, _P, _P]),
    "sl8_page_select": (_INT, [_P, _INT, _P, _P, _I32, _I32, _P, _I32, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                               _I32, _P, _P, _P, _P, _P]),
    "sl8_attn_int8_sparse_decode_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32, _I32]),
    "sl8_attn_int8_sparse_decode": (_INT, [_P, _INT, _P, _P, _P, _P, _I32, _I32, _P, _P, _I32, _I32, _I32, _I32, _I32,
                                           _I32, _P, _INT, _P, _P, _SZ, _P]),
    "sl8_rope_append_int4": (_INT, [_P, _P, _P, _INT, _I64, _I64, _I64, _I32, _I32, _I32, _I32, _P, _I32, _I32, _P,
                                    ctypes.c_char_p, _INT, _P, _I64, _P, _P, _P, _P, _P, _P, _I32, _I32, _P]),
    "sl8_paged_read_int4": (_INT, [_P, _P, _P, _P, _I32, _I32, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _I64, _P, _P, _P,
                                   _INT, _P]),
    "sl8_attn_int4_paged_decode_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32]),
    "sl8_attn_int4_paged_decode": (_INT, [_P, _INT, _P, _P, _P, _P, _I32, _I32, _P, _I32, _P, _P, _I32, _I32, _I32, _I32,
                                          _I32, _I32, _P, _INT, _P, _P, _SZ, _P]),
    "sl8_last_device_status": (_INT, [_P, ctypes.POINTER(_INT)]),
    "sl8_set_spin_limit_ns": (None, [_U64]),
    "sl8_get_spin_limit_ns": (_U64, []),
    "sl8_selftest_timeout": (_INT, [_U64, _P]),
    "sl8_trace_enable": (None, [_INT]),
    "sl8_trace_collect": (_INT, [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(_I64),
                                 ctypes.POINTER(ctypes.c_double), _INT]),
}


def lib() -> ctypes.CDLL:
    """The loaded libsl8 (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libsl8.so not found at {LIB_PATH}: build it first "
                                   "(python -c 'import __graft_entry__ as g; g.build()'); there is no fallback")
            l = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _SIGNATURES.items():
                f = getattr(l, name)
                f.restype = res
                f.argtypes = args
            _lib = l
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/sl8.h declares."""
    src = open(HEADER_PATH).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(sl8_[a-z0-9_]+)\s*\(", src)))


def status_string(status: int) -> str:
    try:
        return lib().sl8_status_string(status).decode()
    except Exception:  # noqa: BLE001 - used while formatting another error
        return f"status {status}"


def _check(status: int, what: str) -> None:
    if status != SL8_OK:
        raise SL8Error(status, what)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DTYPES[t.dtype]


def _need_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("sl8 takes CUDA tensors only (no CPU fallback)")
            if not t.is_contiguous():
                raise ValueError("sl8 takes contiguous tensors")


# ------------------------------------------------------------------ quantisation

def quant_rowwise(x: torch.Tensor, sub_mean: torch.Tensor | None = None, rows_per_group: int | None = None):
    """Symmetric per-row int8 quantisation of the last axis of x (f16/bf16/f32).

    Returns (codes int8 like x, scales fp32 x.shape[:-1]).  sub_mean [groups, cols]
    fp32 is subtracted from row r (flattened) with group r // rows_per_group."""
    _need_cuda(x, sub_mean)
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    codes = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    scales = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    rpg = 0
    if sub_mean is not None:
        rpg = rows_per_group or rows
    _check(lib().sl8_quant_rowwise(_ptr(x), _dt(x), rows, cols, cols, _ptr(sub_mean), rpg, _ptr(codes),
                                   _ptr(scales), _stream(x.device)), "sl8_quant_rowwise")
    return codes, scales


def k_channel_mean(k: torch.Tensor, cu_seqlens: torch.Tensor | None = None, max_seqlen: int | None = None):
    """Per-(sequence, kv head, channel) mean of K.  Dense k [B,Hkv,N,d] or packed
    k [T,Hkv,d] with cu_seqlens.  Returns fp32 [B, Hkv, d]."""
    _need_cuda(k, cu_seqlens)
    if cu_seqlens is None:
        B, Hkv, N, d = k.shape
        T = 0
    else:
        T, Hkv, d = k.shape
        B = cu_seqlens.numel() - 1
        N = int(max_seqlen) if max_seqlen is not None else T
    mean = torch.empty((B, Hkv, d), dtype=torch.float32, device=k.device)
    ws_bytes = lib().sl8_k_channel_mean_workspace_size(B, Hkv, N, d)
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=k.device)
    _check(lib().sl8_k_channel_mean(_ptr(k), _dt(k), B, Hkv, N, d, _ptr(cu_seqlens), T, _ptr(mean), _ptr(ws),
                                    ws.numel(), _stream(k.device)), "sl8_k_channel_mean")
    return mean


# ------------------------------------------------------------------ prefill

def prefill_workspace_bytes(B, Hq, Hkv, N, d, total_tokens=0) -> int:
    return int(lib().sl8_attn_int8_fwd_workspace_size(B, Hq, Hkv, N, d, total_tokens))


def attn_int8_fwd(q, k, v, causal=True, smooth_k=True, cu_seqlens=None, max_seqlen=None, out_dtype=None,
                  return_lse=False, workspace=None, out=None, lse=None):
    """W8A8 INT8 attention prefill.

    Dense: q [B,Hq,N,d], k/v [B,Hkv,N,d].  Varlen: q [T,Hq,d], k/v [T,Hkv,d] with
    cu_seqlens int32 [B+1] (CUDA) and max_seqlen (host int >= every length).
    Returns out (q's layout, dtype v.dtype or out_dtype=float32) and, with
    return_lse, the fp32 log-sum-exp per query row."""
    return _prefill("sl8_attn_int8_fwd", (), q, k, v, causal, smooth_k, cu_seqlens, max_seqlen, out_dtype,
                    return_lse, workspace, out, lse)


def attn_w8a8_fwd(q, k, v, causal=True, smooth_k=True, q_group=32, k_group=32, q_outlier_ratio=4.0,
                  cu_seqlens=None, max_seqlen=None, out_dtype=None, return_lse=False, workspace=None, out=None,
                  lse=None):
    """W8A8 prefill with grouped scales: rows of a (sequence, head) share one scale per
    group of q_group (Q) / k_group (K) consecutive positions; a Q row above
    q_outlier_ratio times its group's lower median row maximum keeps its own scale
    (0 turns that off).  Groups are powers of two up to 64; q_group = k_group = 1 is
    attn_int8_fwd.  Layouts and the rest as attn_int8_fwd."""
    return _prefill("sl8_attn_w8a8_fwd", (int(q_group), int(k_group), float(q_outlier_ratio)), q, k, v, causal,
                    smooth_k, cu_seqlens, max_seqlen, out_dtype, return_lse, workspace, out, lse)


def _prefill(fn, extra, q, k, v, causal, smooth_k, cu_seqlens, max_seqlen, out_dtype, return_lse, workspace, out,
             lse):
    _need_cuda(q, k, v, cu_seqlens, workspace)
    if cu_seqlens is None:
        B, Hq, N, d = q.shape
        Hkv = k.shape[1]
        T = 0
    else:
        T, Hq, d = q.shape
        Hkv = k.shape[1]
        B = cu_seqlens.numel() - 1
        if max_seqlen is None:
            raise ValueError("varlen prefill needs max_seqlen")
        N = int(max_seqlen)
        if cu_seqlens.dtype != torch.int32:
            raise TypeError("cu_seqlens must be int32")
    out_dtype = out_dtype or v.dtype
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    if return_lse and lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    ws_bytes = prefill_workspace_bytes(B, Hq, Hkv, N, d, T)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device)
    _check(getattr(lib(), fn)(_ptr(q), _ptr(k), _ptr(v), _dt(q), _dt(v), B, Hq, Hkv, N, d, _ptr(cu_seqlens), T,
                              int(bool(causal)), int(bool(smooth_k)), *extra, _ptr(out), _dt(out),
                              _ptr(lse) if return_lse else None, _ptr(workspace), workspace.numel(),
                              _stream(q.device)), fn)
    return (out, lse) if return_lse else out


def attn_int8_fwd_chunk(q, k, v, causal=True, smooth_k=True, out_dtype=None, return_lse=False, workspace=None,
                        out=None, lse=None):
    """Prefill of a query chunk: q [B,Hq,Nq,d] holds the last Nq positions of sequences
    whose keys/values k, v [B,Hkv,Nk,d] cover all Nk >= Nq positions (bottom-right causal
    alignment).  Returns out [B,Hq,Nq,d] (and the fp32 LSE with return_lse)."""
    _need_cuda(q, k, v, workspace)
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    out_dtype = out_dtype or v.dtype
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    if return_lse and lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    if workspace is None:
        # room for the key-split partials, which the library uses when the chunk is small
        ws_bytes = int(lib().sl8_attn_int8_fwd_chunk_workspace_size(B, Hq, Hkv, Nq, Nk, d))
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device)
    _check(lib().sl8_attn_int8_fwd_chunk(_ptr(q), _ptr(k), _ptr(v), _dt(q), _dt(v), B, Hq, Hkv, Nq, Nk, d,
                                         int(bool(causal)), int(bool(smooth_k)), _ptr(out), _dt(out),
                                         _ptr(lse) if return_lse else None, _ptr(workspace), workspace.numel(),
                                         _stream(q.device)), "sl8_attn_int8_fwd_chunk")
    return (out, lse) if return_lse else out


def attn_int8_fwd_chunk_cache(q, k_cache, k_scale, v_cache, v_scale, Nk=None, causal=True, out_dtype=None,
                              return_lse=False, workspace=None, out=None, lse=None):
    """Prefill of a query chunk onto an int8 KV cache: q [B,Hq,Nq,d] (fp16/bf16) holds
    positions Nk-Nq .. Nk-1; the caches k_cache, v_cache [B,Hkv,Lmax,d] int8 with scales
    [B,Hkv,Lmax] fp32 hold Nk (default Lmax) positions of every sequence.  Returns out
    [B,Hq,Nq,d] (and the fp32 LSE with return_lse)."""
    _need_cuda(q, k_cache, k_scale, v_cache, v_scale, workspace)
    B, Hq, Nq, d = q.shape
    Hkv, Lmax = k_cache.shape[1], k_cache.shape[2]
    Nk = Lmax if Nk is None else int(Nk)
    out_dtype = out_dtype or q.dtype
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    if return_lse and lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    if workspace is None:
        ws_bytes = int(lib().sl8_attn_int8_fwd_chunk_workspace_size(B, Hq, Hkv, Nq, Nk, d))
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device)
    _check(lib().sl8_attn_int8_fwd_chunk_cache(_ptr(q), _dt(q), _ptr(k_cache), _ptr(k_scale), _ptr(v_cache),
                                               _ptr(v_scale), B, Hq, Hkv, Nq, Nk, Lmax, d, int(bool(causal)),
                                               _ptr(out), _dt(out), _ptr(lse) if return_lse else None,
                                               _ptr(workspace), workspace.numel(), _stream(q.device)),
           "sl8_attn_int8_fwd_chunk_cache")
    return (out, lse) if return_lse else out


def attn_int8_qk_logits_debug(q, k, smooth_k=True, row_begin=0, row_end=None, want_codes=True, groups=None,
                              cu_seqlens=None, max_seqlen=None, want_logits=True, workspace=None):
    """Exact int32 logits of the prefill tensor-core path for query rows
    [row_begin, row_end) of every sequence against every key of that sequence, plus the
    int8 codes and fp32 scales of Q and (smoothed) K.  Dense q [B,Hq,N,d], k [B,Hkv,N,d],
    or varlen q [T,Hq,d], k [T,Hkv,d] with cu_seqlens and max_seqlen; logits are
    [B,Hq,row_end-row_begin,N] (entries past a sequence's length stay 0).
    groups = (q_group, k_group, q_outlier_ratio) selects the grouped quantisation of
    attn_w8a8_fwd.  Returns a dict."""
    _need_cuda(q, k, cu_seqlens, workspace)
    if cu_seqlens is None:
        B, Hq, N, d = q.shape
        T = 0
        code_shape = lambda H: (B, H, N)  # noqa: E731
    else:
        T, Hq, d = q.shape
        B = cu_seqlens.numel() - 1
        if max_seqlen is None:
            raise ValueError("varlen logits need max_seqlen")
        N = int(max_seqlen)
        code_shape = lambda H: (T, H)  # noqa: E731
    Hkv = k.shape[-2] if cu_seqlens is not None else k.shape[1]
    row_end = N if row_end is None else row_end
    dev = q.device
    logits = (torch.zeros((B, Hq, row_end - row_begin, N), dtype=torch.int32, device=dev) if want_logits else None)
    res = dict(logits=logits)
    if want_codes:
        res.update(q_codes=torch.empty((*code_shape(Hq), d), dtype=torch.int8, device=dev),
                   q_scales=torch.empty(code_shape(Hq), dtype=torch.float32, device=dev),
                   k_codes=torch.empty((*code_shape(Hkv), d), dtype=torch.int8, device=dev),
                   k_scales=torch.empty(code_shape(Hkv), dtype=torch.float32, device=dev))
    ws_bytes = prefill_workspace_bytes(B, Hq, Hkv, N, d, T)
    ws = workspace if workspace is not None else torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=dev)
    head = (_ptr(q), _ptr(k), _dt(q), B, Hq, Hkv, N, d, _ptr(cu_seqlens), T, int(bool(smooth_k)))
    tail = (row_begin, row_end, _ptr(logits), _ptr(res.get("q_codes")), _ptr(res.get("q_scales")),
            _ptr(res.get("k_codes")), _ptr(res.get("k_scales")), _ptr(ws), ws.numel(), _stream(dev))
    if groups is None:
        _check(lib().sl8_attn_int8_qk_logits_debug(*head, *tail), "sl8_attn_int8_qk_logits_debug")
    else:
        g = (int(groups[0]), int(groups[1]), float(groups[2]))
        _check(lib().sl8_attn_w8a8_qk_logits_debug(*head, *g, *tail), "sl8_attn_w8a8_qk_logits_debug")
    return res


# ------------------------------------------------------------------ decode

def decode_num_splits(B: int, Hkv: int, Lmax: int, d: int, num_splits: int = 0) -> int:
    """Effective split count of the decode for this shape (0 = automatic)."""
    return int(lib().sl8_attn_decode_num_splits(B, Hkv, Lmax, d, num_splits))


def decode_workspace(B: int, Hq: int, Hkv: int, Lmax: int, d: int, num_splits: int = 0, device=None):
    """The decode's split partials carved from one buffer of
    sl8_attn_decode_workspace_size bytes: (o_partial [B,Hq,S,d], lse_partial [B,Hq,S])
    fp32 views, at the offsets the header states."""
    S = decode_num_splits(B, Hkv, Lmax, d, num_splits)
    nbytes = int(lib().sl8_attn_decode_workspace_size(B, Hq, Hkv, Lmax, d, num_splits))
    off = int(lib().sl8_attn_decode_lse_offset(B, Hq, Hkv, Lmax, d, num_splits))
    if S <= 0 or nbytes == 0:
        raise SL8Error(SL8_ERR_UNSUPPORTED, "sl8_attn_decode_workspace_size")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    o_partial = ws[:B * Hq * S * d * 4].view(torch.float32).view(B, Hq, S, d)
    lse_partial = ws[off:off + B * Hq * S * 4].view(torch.float32).view(B, Hq, S)
    return o_partial, lse_partial


def attn_int8_decode_splitkv(q, k_cache, k_scale, v_cache, v_scale, seqlens, num_splits=0, o_partial=None,
                             lse_partial=None):
    """Split-KV partials (normalised O [B,Hq,S,d] fp32, lse [B,Hq,S] fp32)."""
    _need_cuda(q, k_cache, k_scale, v_cache, v_scale, seqlens)
    B, Hq, d = q.shape
    _, Hkv, Lmax, _ = k_cache.shape
    S = decode_num_splits(B, Hkv, Lmax, d, num_splits)
    if o_partial is None and lse_partial is None and S > 0:
        o_partial, lse_partial = decode_workspace(B, Hq, Hkv, Lmax, d, num_splits, q.device)
    if o_partial is None:
        o_partial = torch.empty((B, Hq, max(S, 1), d), dtype=torch.float32, device=q.device)
    if lse_partial is None:
        lse_partial = torch.empty((B, Hq, max(S, 1)), dtype=torch.float32, device=q.device)
    _check(lib().sl8_attn_int8_decode_splitkv(_ptr(q), _dt(q), _ptr(k_cache), _ptr(k_scale), _ptr(v_cache),
                                              _ptr(v_scale), _ptr(seqlens), B, Hq, Hkv, Lmax, d, num_splits,
                                              _ptr(o_partial), _ptr(lse_partial), _stream(q.device)),
           "sl8_attn_int8_decode_splitkv")
    return o_partial, lse_partial


def attn_decode_combine(o_partial, lse_partial, seqlens, Lmax, out_dtype=torch.bfloat16, return_lse=False, out=None):
    _need_cuda(o_partial, lse_partial, seqlens)
    B, Hq, S, d = o_partial.shape
    if out is None:
        out = torch.empty((B, Hq, d), dtype=out_dtype, device=o_partial.device)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=o_partial.device) if return_lse else None
    _check(lib().sl8_attn_decode_combine(_ptr(o_partial), _ptr(lse_partial), _ptr(seqlens), B, Hq, Lmax, d, S,
                                         _ptr(out), _dt(out), _ptr(lse), _stream(o_partial.device)),
           "sl8_attn_decode_combine")
    return (out, lse) if return_lse else out


def attn_int8_decode(q, k_cache, k_scale, v_cache, v_scale, seqlens, num_splits=0, out_dtype=None, return_lse=False,
                     o_partial=None, lse_partial=None, out=None):
    """Split-KV decode plus combine: out [B, Hq, d] (dtype q.dtype unless given)."""
    o_p, l_p = attn_int8_decode_splitkv(q, k_cache, k_scale, v_cache, v_scale, seqlens, num_splits, o_partial,
                                        lse_partial)
    return attn_decode_combine(o_p, l_p, seqlens, k_cache.shape[2], out_dtype or q.dtype, return_lse, out)


def attn_int8_decode_verify(q, k_cache, k_scale, v_cache, v_scale, seqlens, tree_mask, num_splits=0, out_dtype=None,
                            return_lse=False, o_partial=None, lse_partial=None, out=None):
    """Speculative-decode verification: q [B, T, Hq, d] draft queries, tree_mask [B, T] int32
    (bit u of row (b, t): query t sees draft token u, which sits at position L_b - T + u of
    the cache).  Returns out [B, T, Hq, d] (and the LSE [B, T, Hq] with return_lse)."""
    _need_cuda(q, k_cache, k_scale, v_cache, v_scale, seqlens, tree_mask)
    if tree_mask.dtype != torch.int32:
        raise TypeError("tree_mask must be int32 (bit u: draft token u is visible)")
    B, T, Hq, d = q.shape
    _, Hkv, Lmax, _ = k_cache.shape
    S = int(lib().sl8_attn_decode_verify_num_splits(B, T, Hq, Hkv, Lmax, d, num_splits))
    if o_partial is None:
        o_partial = torch.empty((B * T, Hq, max(S, 1), d), dtype=torch.float32, device=q.device)
    if lse_partial is None:
        lse_partial = torch.empty((B * T, Hq, max(S, 1)), dtype=torch.float32, device=q.device)
    if out is None:
        out = torch.empty((B, T, Hq, d), dtype=out_dtype or q.dtype, device=q.device)
    lse = torch.empty((B, T, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    _check(lib().sl8_attn_int8_decode_verify(_ptr(q), _dt(q), _ptr(k_cache), _ptr(k_scale), _ptr(v_cache),
                                             _ptr(v_scale), _ptr(seqlens), _ptr(tree_mask), T, B, Hq, Hkv, Lmax, d,
                                             num_splits, _ptr(o_partial), _ptr(lse_partial), _ptr(out), _dt(out),
                                             _ptr(lse), _stream(q.device)), "sl8_attn_int8_decode_verify")
    return (out, lse) if return_lse else out


def attn_int8_decode_splitkv_f16v(q, k_cache, k_scale, v_cache, seqlens, num_splits=0, o_partial=None,
                                  lse_partial=None):
    """Split-KV partials with an int8 K cache and an fp16 V cache [B, Hkv, Lmax, d]."""
    _need_cuda(q, k_cache, k_scale, v_cache, seqlens)
    if v_cache.dtype != torch.float16:
        raise ValueError("v_cache must be float16")
    B, Hq, d = q.shape
    _, Hkv, Lmax, _ = k_cache.shape
    S = decode_num_splits(B, Hkv, Lmax, d, num_splits)
    if o_partial is None:
        o_partial = torch.empty((B, Hq, max(S, 1), d), dtype=torch.float32, device=q.device)
    if lse_partial is None:
        lse_partial = torch.empty((B, Hq, max(S, 1)), dtype=torch.float32, device=q.device)
    _check(lib().sl8_attn_int8_decode_splitkv_f16v(_ptr(q), _dt(q), _ptr(k_cache), _ptr(k_scale), _ptr(v_cache),
                                                   _ptr(seqlens), B, Hq, Hkv, Lmax, d, num_splits, _ptr(o_partial),
                                                   _ptr(lse_partial), _stream(q.device)),
           "sl8_attn_int8_decode_splitkv_f16v")
    return o_partial, lse_partial


def attn_int8_decode_f16v(q, k_cache, k_scale, v_cache, seqlens, num_splits=0, out_dtype=None, return_lse=False,
                          o_partial=None, lse_partial=None, out=None):
    """Split-KV decode (int8 K, fp16 V) plus combine: out [B, Hq, d] (dtype q.dtype unless given)."""
    o_p, l_p = attn_int8_decode_splitkv_f16v(q, k_cache, k_scale, v_cache, seqlens, num_splits, o_partial,
                                             lse_partial)
    return attn_decode_combine(o_p, l_p, seqlens, k_cache.shape[2], out_dtype or q.dtype, return_lse, out)


def attn_int8_paged_decode_splitkv(q, k_pages, k_scale_pages, v_pages, v_scale_pages, block_table, seqlens,
                                   num_splits=0, o_partial=None, lse_partial=None):
    """Split-KV partials over a paged k8v8 cache: pages [num_pages, Hkv, page_size, d] int8,
    scales [num_pages, Hkv, page_size] fp32, block_table [B, max_blocks] int32."""
    _need_cuda(q, k_pages, k_scale_pages, v_pages, v_scale_pages, block_table, seqlens)
    B, Hq, d = q.shape
    num_pages, Hkv, page_size, _ = k_pages.shape
    max_blocks = block_table.shape[1]
    S = decode_num_splits(B, Hkv, max_blocks * page_size, d, num_splits)
    if o_partial is None:
        o_partial = torch.empty((B, Hq, max(S, 1), d), dtype=torch.float32, device=q.device)
    if lse_partial is None:
        lse_partial = torch.empty((B, Hq, max(S, 1)), dtype=torch.float32, device=q.device)
    _check(lib().sl8_attn_int8_paged_decode_splitkv(_ptr(q), _dt(q), _ptr(k_pages), _ptr(k_scale_pages),
                                                    _ptr(v_pages), _ptr(v_scale_pages), _ptr(block_table),
                                                    max_blocks, page_size, num_pages, _ptr(seqlens), B, Hq, Hkv, d,
                                                    num_splits, _ptr(o_partial), _ptr(lse_partial),
                                                    _stream(q.device)),
           "sl8_attn_int8_paged_decode_splitkv")
    return o_partial, lse_partial


def attn_int8_paged_decode(q, k_pages, k_scale_pages, v_pages, v_scale_pages, block_table, seqlens, num_splits=0,
                           out_dtype=None, return_lse=False, o_partial=None, lse_partial=None, out=None):
    """Paged split-KV decode plus combine: out [B, Hq, d] (dtype q.dtype unless given)."""
    o_p, l_p = attn_int8_paged_decode_splitkv(q, k_pages, k_scale_pages, v_pages, v_scale_pages, block_table,
                                              seqlens, num_splits, o_partial, lse_partial)
    lmax = block_table.shape[1] * k_pages.shape[2]
    return attn_decode_combine(o_p, l_p, seqlens, lmax, out_dtype or q.dtype, return_lse, out)


def attn_int8_decode_logits_debug(q, k_cache, k_scale, v_cache, v_scale, seqlens):
    """Exact int32 decode logits [B, Hq, Lmax] (entries t >= L_b stay 0) and q codes/scales."""
    _need_cuda(q, k_cache, k_scale, v_cache, v_scale, seqlens)
    B, Hq, d = q.shape
    _, Hkv, Lmax, _ = k_cache.shape
    dev = q.device
    S = decode_num_splits(B, Hkv, Lmax, d, 0)
    logits = torch.zeros((B, Hq, Lmax), dtype=torch.int32, device=dev)
    q_codes = torch.empty((B, Hq, d), dtype=torch.int8, device=dev)
    q_scales = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    o_p = torch.empty((B, Hq, max(S, 1), d), dtype=torch.float32, device=dev)
    l_p = torch.empty((B, Hq, max(S, 1)), dtype=torch.float32, device=dev)
    _check(lib().sl8_attn_int8_decode_logits_debug(_ptr(q), _dt(q), _ptr(k_cache), _ptr(k_scale), _ptr(v_cache),
                                                   _ptr(v_scale), _ptr(seqlens), B, Hq, Hkv, Lmax, d, _ptr(logits),
                                                   _ptr(q_codes), _ptr(q_scales), _ptr(o_p), _ptr(l_p),
                                                   _stream(dev)), "sl8_attn_int8_decode_logits_debug")
    return dict(logits=logits, q_codes=q_codes, q_scales=q_scales)


# ------------------------------------------------------------------ serving from the paged cache

_I32T, _F32T, _I8T = torch.int32, torch.float32, torch.int8
_SELECT_HELD = 4096  # blocks up to which a selection needs no scores (kPageSelectHeld of the library)


def _index(t) -> int:
    """The CUDA device that a tensor lives on."""
    i = t.get_device()
    if i < 0:
        raise ValueError("sl8 takes CUDA tensors only (no CPU fallback)")
    return i


def _ptrs(dev, dtype, names, *ts):
    """Addresses of contiguous tensors of one device and dtype (None stays None); names: theirs,
    for the error."""
    out = []
    for t in ts:
        if t is None:
            out.append(None)
        elif t.get_device() == dev and t.dtype is dtype and t.is_contiguous():
            out.append(t.data_ptr())
        else:
            name = names.split()[len(out)]
            if t.get_device() != dev:
                _index(t)
                raise ValueError(f"{name} is on another device")
            if t.dtype is not dtype:
                raise TypeError(f"{name} must be {dtype}")
            raise ValueError(f"{name} must be contiguous")
    return out


def _shaped(t, shape, name) -> None:
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def _call(fn: str, dev: int, *args) -> None:
    """Call an entry point on the device's current stream, with that device current."""
    f = getattr(_lib or lib(), fn)
    if dev == torch._C._cuda_getDevice():
        status = f(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = f(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status != SL8_OK:
        raise SL8Error(status, fn)


def paged_assign(ctx_lens, new_lens, block_table, free_pages, free_count, page_size, max_tokens, release=None,
                 out=None):
    """The page plan of one serving step: block tables, slot map and free list from request
    lengths.  ctx_lens, new_lens [B] int32; release [B] int32 (nonzero: the slot's request
    has ended, its pages go back first); block_table [B, max_blocks] and free_pages
    [capacity] are updated, free_count [1] int32 is read.  Returns a dict of int32 tensors:
    seqlens, granted [B], cu_new [B + 1], slot_map, token_pos [max_tokens], free_count [1]
    (out: a dict returned earlier, whose tensors are written again)."""
    dev = _index(block_table)
    p = _ptrs(dev, _I32T, "ctx_lens new_lens release block_table free_pages free_count", ctx_lens, new_lens, release,
              block_table, free_pages, free_count)
    B, max_blocks = block_table.shape
    max_tokens = int(max_tokens)
    if ctx_lens.numel() != B or new_lens.numel() != B or (release is not None and release.numel() != B):
        raise ValueError("ctx_lens, new_lens and release need one entry per row of block_table")
    if free_count.numel() < 1:
        raise ValueError("free_count needs one entry")
    if out is None:
        sizes = dict(seqlens=B, granted=B, cu_new=B + 1, slot_map=max_tokens, token_pos=max_tokens, free_count=1)
        out = {n: torch.empty(size, dtype=_I32T, device=block_table.device) for n, size in sizes.items()}
    elif (out["seqlens"].numel() != B or out["granted"].numel() != B or out["cu_new"].numel() != B + 1 or
          out["slot_map"].numel() != max_tokens or out["token_pos"].numel() != max_tokens or
          out["free_count"].numel() < 1):
        raise ValueError("out holds tensors of another batch or max_tokens")
    o = _ptrs(dev, _I32T, "free_count seqlens granted cu_new slot_map token_pos", out["free_count"], out["seqlens"],
              out["granted"], out["cu_new"], out["slot_map"], out["token_pos"])
    _call("sl8_paged_assign", dev, p[0], p[1], p[2], B, int(page_size), max_blocks, p[3], p[4], free_pages.numel(), p[5],
          o[0], max_tokens, o[1], o[2], o[3], o[4], o[5])
    return out


def _tokens(x, name, dev, dtype, T, d):
    """(address, heads, stride in elements) of [T, heads, d] whose tokens may be strided."""
    if x.get_device() != dev:
        _index(x)
        raise ValueError(f"{name} is on another device")
    if x.dtype is not dtype:
        raise TypeError("q, k, v and q_out must have one dtype")
    shape, stride = x.shape, x.stride()
    if len(shape) != 3 or shape[0] != T or shape[2] != d or stride[2] != 1 or (shape[1] > 1 and stride[1] != d):
        raise ValueError(f"{name} must be [{T}, heads, {d}] with each token's heads contiguous")
    return x.data_ptr(), shape[1], (stride[0] if T > 1 else shape[1] * d)


def _pages_of(dev, k_pages, k_scale_pages, v_pages=None, v_scale_pages=None):
    """((num_pages, Hkv, page_size, d), code addresses, scale addresses)."""
    c = _ptrs(dev, _I8T, "k_pages v_pages", k_pages, v_pages)
    s = _ptrs(dev, _F32T, "k_scale_pages v_scale_pages", k_scale_pages, v_scale_pages)
    shape = k_pages.shape
    if len(shape) != 4:
        raise ValueError("pages must be [num_pages, Hkv, page_size, d]")
    num_pages, hkv, page_size, _ = shape
    rows = (num_pages, hkv, page_size)
    _shaped(k_scale_pages, rows, "k_scale_pages")
    if v_pages is not None:
        _shaped(v_pages, shape, "v_pages")
        _shaped(v_scale_pages, rows, "v_scale_pages")
    return shape, c, s


def rope_pair_axis(sections, interleaved=False) -> bytes:
    """The axis of each rotary pair for rope_append: sections[a] pairs turn with axis a, in
    that order, or (interleaved) dealt out in turn until an axis has all of its pairs."""
    if not interleaved:
        return bytes(a for a, n in enumerate(sections) for _ in range(n))
    left, pairs = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                pairs.append(a)
                left[a] -= 1
    return bytes(pairs)


def rope_append(q, k, v, positions, inv_freq, slot_map, k_pages, k_scale_pages, v_pages, v_scale_pages,
                pair_axis=None, adjacent=False, q_out=None):
    """Rotary positions and the int8 append: q [T,Hq,d] and k [T,Hkv,d] are rotated, k and v
    quantised per row and stored at slot_map [T] int32 (negative: not stored) of the pages
    [num_pages,Hkv,page_size,d] int8 with scales [num_pages,Hkv,page_size].  positions int32
    [T] or [axes,T]; inv_freq fp32 [rot_dim / 2]; pair_axis (bytes or ints, one per pair;
    see rope_pair_axis) for several axes; adjacent: pairs (2p, 2p+1) instead of halves.
    positions = inv_freq = None: no rotation.  q may be None.  Returns the rotated q (q_out,
    which may be q itself)."""
    dev = _index(k_pages)
    (num_pages, hkv, page_size, d), codes, scales = _pages_of(dev, k_pages, k_scale_pages, v_pages, v_scale_pages)
    return _append("sl8_rope_append", dev, hkv, d, q, k, v, positions, inv_freq, slot_map, pair_axis, adjacent, q_out,
                   (codes[0], scales[0], codes[1], scales[1], num_pages, page_size))


def _append(fn, dev, hkv, d, q, k, v, positions, inv_freq, slot_map, pair_axis, adjacent, q_out, pages):
    """The appends' checks and call; pages: the arguments after slot_map."""
    pos, slots = _ptrs(dev, _I32T, "positions slot_map", positions, slot_map)
    freq, = _ptrs(dev, _F32T, "inv_freq", inv_freq)
    T, dtype = k.shape[0], k.dtype
    kp, kh, k_stride = _tokens(k, "k", dev, dtype, T, d)
    vp, vh, v_stride = _tokens(v, "v", dev, dtype, T, d)
    if kh != hkv or vh != hkv or slot_map.numel() != T:
        raise ValueError("k, v and slot_map must hold the same tokens, with the pages' kv heads")
    qp = op = None
    hq = q_stride = out_stride = 0
    if q is not None:
        qp, hq, q_stride = _tokens(q, "q", dev, dtype, T, d)
        if q_out is None:
            q_out = torch.empty((T, hq, d), dtype=dtype, device=q.device)
        op, oh, out_stride = _tokens(q_out, "q_out", dev, dtype, T, d)
        if oh != hq:
            raise ValueError("q_out must have q's heads")
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    axes, rot = 1, 0
    if positions is not None:
        axes, rot = (1 if positions.dim() == 1 else positions.shape[0]), 2 * inv_freq.numel()
        if positions.numel() != axes * T:
            raise ValueError("positions must be [T] or [axes, T]")
    if pair_axis is not None:
        pair_axis = bytes(pair_axis)
        if len(pair_axis) != rot // 2:
            raise ValueError("pair_axis needs one entry per rotary pair")
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    _call(fn, dev, qp, kp, vp, _DTYPES[dtype], q_stride, k_stride, v_stride, T, hq, hkv, d, pos, axes, rot, freq,
          pair_axis, 1 if adjacent else 0, op, out_stride, slots, *pages)
    return q_out


def page_bounds(k_pages, k_scale_pages, block_table, seqlens, bounds, bound_scale, new_lens=None, max_new=None):
    """Per-channel key bounds (bounds [num_pages,Hkv,2,d] int8, bound_scale [num_pages,Hkv]
    fp32, updated) of the pages that the last new_lens [B] int32 tokens of each sequence lie
    in (max_new: a host int >= every entry), or of every page without new_lens.
    seqlens [B] int32 counts the new tokens."""
    dev = _index(k_pages)
    (num_pages, hkv, page_size, d), codes, scales = _pages_of(dev, k_pages, k_scale_pages)
    bp, = _ptrs(dev, _I8T, "bounds", bounds)
    sp, = _ptrs(dev, _F32T, "bound_scale", bound_scale)
    _shaped(bounds, (num_pages, hkv, 2, d), "bounds")
    _shaped(bound_scale, (num_pages, hkv), "bound_scale")
    p = _ptrs(dev, _I32T, "block_table seqlens new_lens", block_table, seqlens, new_lens)
    B, max_blocks = block_table.shape
    if seqlens.numel() != B or (new_lens is not None and new_lens.numel() != B):
        raise ValueError("seqlens and new_lens need one entry per row of block_table")
    if (new_lens is None) != (max_new is None):
        raise ValueError("new_lens and max_new go together")
    _call("sl8_page_bounds", dev, codes[0], scales[0], num_pages, page_size, p[0], max_blocks, p[1], p[2],
          0 if max_new is None else int(max_new), B, hkv, d, bp, sp)


def page_select(q, bounds, bound_scale, block_table, seqlens, page_size, max_sel, first=1, last=2, out=None,
                scores=None):
    """The max_sel pages of each query and kv head whose keys can reach the largest logits,
    the first `first` and last `last` ones always among them.  q [B,Hq,d] (the decode's
    queries) or [B,T,Hq,d] (query t at position seqlens - T + t); bounds as page_bounds leaves
    them.  Returns a dict of int32 tensors: blocks and pages [B,T,Hkv,max_sel] (ascending
    blocks; -1 past the list) and lens [B,T,Hkv], the tokens listed (out: a dict returned
    earlier, written again).  scores fp32 [B,T,Hkv,max_blocks] receives the scores of
    the pages of every range longer than max_sel (allocated here where none is given and the
    table is wider than the 4,096 blocks whose scores stay on chip)."""
    dev = _index(q)
    if q.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {q.dtype}")
    qp, = _ptrs(dev, q.dtype, "q", q)
    bp, = _ptrs(dev, _I8T, "bounds", bounds)
    sp, scp = _ptrs(dev, _F32T, "bound_scale scores", bound_scale, scores)
    table, lens = _ptrs(dev, _I32T, "block_table seqlens", block_table, seqlens)
    if bounds.dim() != 4 or bounds.shape[2] != 2:
        raise ValueError("bounds must be [num_pages, Hkv, 2, d]")
    num_pages, hkv, _, d = bounds.shape
    _shaped(bound_scale, (num_pages, hkv), "bound_scale")
    B, max_blocks = block_table.shape
    shape = q.shape
    if len(shape) not in (3, 4):
        raise ValueError("q must be [B, Hq, d] or [B, T, Hq, d]")
    T, hq = (1, shape[1]) if len(shape) == 3 else (shape[1], shape[2])
    if shape[0] != B or shape[-1] != d or seqlens.numel() != B:
        raise ValueError("q, block_table, seqlens and bounds do not belong together")
    max_sel, rows = int(max_sel), B * T * hkv
    if out is None:
        new = lambda *n: torch.empty(n, dtype=_I32T, device=q.device)  # noqa: E731
        out = {"blocks": new(B, T, hkv, max_sel), "pages": new(B, T, hkv, max_sel), "lens": new(B, T, hkv)}
    elif (out["blocks"].numel() != rows * max_sel or out["pages"].numel() != rows * max_sel or
          out["lens"].numel() != rows):
        raise ValueError("out holds tensors of another shape")
    o = _ptrs(dev, _I32T, "blocks pages lens", out["blocks"], out["pages"], out["lens"])
    if scores is not None:
        _shaped(scores, (B, T, hkv, max_blocks), "scores")
    elif max_blocks > _SELECT_HELD:
        scores = torch.empty((B, T, hkv, max_blocks), dtype=_F32T, device=q.device)
        scp = scores.data_ptr()
    _call("sl8_page_select", dev, qp, _DTYPES[q.dtype], bp, sp, num_pages, int(page_size), table, max_blocks, lens, B, T,
          hq, hkv, d, max_sel, int(first), int(last), o[0], o[1], o[2], scp)
    return out


def sparse_decode_workspace_bytes(rows: int, Hq: int, Hkv: int, max_sel: int, page_size: int, d: int,
                                  num_splits: int = 0) -> int:
    return int(lib().sl8_attn_int8_sparse_decode_workspace_size(rows, Hq, Hkv, max_sel, page_size, d, num_splits))


def attn_int8_sparse_decode(q, k_pages, k_scale_pages, v_pages, v_scale_pages, pages, lens, num_splits=0,
                            out_dtype=None, return_lse=False, workspace=None, out=None, lse=None):
    """Decode attention of each query over a page list of its own per kv head: q [B,Hq,d] or
    [B,T,Hq,d], pages [B(,T),Hkv,max_sel] int32 and lens [B(,T),Hkv] int32 as page_select
    returns them (or from any other policy: full pages, the last one up to the length).
    Returns out like q (dtype q.dtype unless given) and, with return_lse, the fp32 LSE: 0 and
    -inf for an empty list, NaN where a logit is NaN (rows quantised with infinities).
    workspace: uint8, at least sparse_decode_workspace_bytes (16: none is used)."""
    dev = _index(q)
    (num_pages, hkv, page_size, d), codes, scales = _pages_of(dev, k_pages, k_scale_pages, v_pages, v_scale_pages)
    list_p, lens_p = _ptrs(dev, _I32T, "pages lens", pages, lens)
    shape = q.shape
    hq, max_sel = shape[-2], pages.shape[-1]
    rows = q.numel() // (hq * d) if hq * d else 0
    if shape[-1] != d or lens.numel() != rows * hkv or pages.numel() != rows * hkv * max_sel:
        raise ValueError("q, pages and lens do not belong together")
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or q.dtype, device=q.device)
    elif out.shape != shape:
        raise ValueError("out must have q's shape")
    if q.dtype not in _DTYPES or out.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {q.dtype} or {out.dtype}")
    qp, = _ptrs(dev, q.dtype, "q", q)
    op, = _ptrs(dev, out.dtype, "out", out)
    lse_p = None
    if return_lse:
        if lse is None:
            lse = torch.empty(shape[:-1], dtype=_F32T, device=q.device)
        elif lse.shape != shape[:-1]:
            raise ValueError("lse must have one entry per query head")
        lse_p, = _ptrs(dev, _F32T, "lse", lse)
    if workspace is None:
        need = sparse_decode_workspace_bytes(rows, hq, hkv, max_sel, page_size, d, num_splits)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need > 16 else None
    ws, nbytes = None, 0
    if workspace is not None:
        ws, = _ptrs(dev, workspace.dtype, "workspace", workspace)
        nbytes = workspace.numel() * workspace.element_size()
    _call("sl8_attn_int8_sparse_decode", dev, qp, _DTYPES[q.dtype], codes[0], scales[0], codes[1], scales[1], num_pages,
          page_size, list_p, lens_p, max_sel, rows, hq, hkv, d, num_splits, op, _DTYPES[out.dtype], lse_p, ws, nbytes)
    return (out, lse) if return_lse else out


# ------------------------------------------------------------------ the paged cache in 4 bits

_U8T, _BF16T = torch.uint8, torch.bfloat16


def _one(t, dev, dtype, name):
    """Address of a contiguous tensor of this device and dtype."""
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    return _ptrs(dev, dtype, name, t)[0]


def _pages4_of(dev, k_pages, k_scale_pages, v_pages, v_scale_pages):
    """num_pages, Hkv, page_size, d and the addresses of codes and scales of 4-bit pages."""
    shape, scales = k_pages.shape, k_scale_pages.shape
    if len(shape) != 4:
        raise ValueError("4-bit pages must be [num_pages, Hkv, page_size, d / 2]")
    num_pages, hkv, page_size, half = shape
    if v_pages.shape != shape:
        _shaped(v_pages, shape, "v_pages")
    if scales != (num_pages, hkv, page_size, half // 16) or v_scale_pages.shape != scales:
        _shaped(k_scale_pages, (num_pages, hkv, page_size, half // 16), "k_scale_pages")
        _shaped(v_scale_pages, scales, "v_scale_pages")
    return (num_pages, hkv, page_size, 2 * half, _one(k_pages, dev, _U8T, "k_pages"), _one(k_scale_pages, dev, _BF16T, "k_scale_pages"),
            _one(v_pages, dev, _U8T, "v_pages"), _one(v_scale_pages, dev, _BF16T, "v_scale_pages"))


def _mean_of(dev, k_mean, hkv, d):
    _shaped(k_mean, (hkv, d), "k_mean")
    return _one(k_mean, dev, _F32T, "k_mean")


def int4_pages(num_pages, Hkv, page_size, d, device=None):
    """An empty 4-bit pool (zeros): k_pages, k_scale_pages, v_pages, v_scale_pages."""
    def codes():
        return torch.full((num_pages, Hkv, page_size, d // 2), 0x88, dtype=_U8T, device=device or "cuda")

    def scales():
        return torch.zeros((num_pages, Hkv, page_size, d // 32), dtype=_BF16T, device=device or "cuda")

    return codes(), scales(), codes(), scales()


def rope_append_int4(q, k, v, positions, inv_freq, slot_map, k_pages, k_scale_pages, v_pages, v_scale_pages,
                     pair_axis=None, adjacent=False, q_out=None, k_mean=None):
    """rope_append to 4-bit pages: codes [num_pages,Hkv,page_size,d/2] uint8 (channel 2i in the low
    half of byte i) with a bf16 scale for each group of 32 channels [num_pages,Hkv,page_size,d/32].
    k_mean fp32 [Hkv,d] is taken off the rotated keys before they are quantised.  The rest, and what
    is returned, as rope_append."""
    dev = _index(k_pages)
    num_pages, hkv, page_size, d, kc, ks, vc, vs = _pages4_of(dev, k_pages, k_scale_pages, v_pages, v_scale_pages)
    mean = None if k_mean is None else _mean_of(dev, k_mean, hkv, d)
    return _append("sl8_rope_append_int4", dev, hkv, d, q, k, v, positions, inv_freq, slot_map, pair_axis, adjacent, q_out,
                   (mean, kc, ks, vc, vs, num_pages, page_size))


def paged_read_int4(k_pages, k_scale_pages, v_pages, v_scale_pages, block_table, seqlens, cu_seqlens=None,
                    max_seqlen=None, total_tokens=None, k_mean=None, out_dtype=None, k_out=None, v_out=None):
    """The first seqlens [B] int32 tokens of each sequence as dense keys and values: [B,Hkv,N,d] with
    N = max_seqlen (default: block_table's width in tokens), as attn_int8_fwd_chunk takes them; or,
    with cu_seqlens [B + 1] int32, packed [total_tokens,Hkv,d], token i of sequence b at row
    cu_seqlens[b] + i.  k_mean: as in the append, added to the keys.  Rows past a sequence's tokens are
    left as they were (zeros where the outputs, of out_dtype, default bfloat16, are made here).
    Returns (k_out, v_out)."""
    dev = _index(k_pages)
    num_pages, hkv, page_size, d, kc, ks, vc, vs = _pages4_of(dev, k_pages, k_scale_pages, v_pages, v_scale_pages)
    B, max_blocks = block_table.shape
    if seqlens.numel() != B or (cu_seqlens is not None and cu_seqlens.numel() != B + 1):
        raise ValueError("seqlens and cu_seqlens need one entry per row of block_table (and one more)")
    N = max_blocks * page_size if max_seqlen is None else int(max_seqlen)
    given = k_out if k_out is not None else v_out
    cu, total = None, 0
    if cu_seqlens is None:
        shape = (B, hkv, N, d)
    else:
        cu = _one(cu_seqlens, dev, _I32T, "cu_seqlens")
        if total_tokens is None and given is None:
            raise ValueError("a packed read needs total_tokens or an output")
        total = int(total_tokens) if total_tokens is not None else given.shape[0]
        shape = (total, hkv, d)
    dtype = given.dtype if given is not None else (out_dtype or _BF16T)
    if dtype not in _DTYPES or (out_dtype is not None and out_dtype is not dtype):
        raise TypeError(f"unsupported dtype {dtype}")
    if k_out is None:
        k_out = torch.zeros(shape, dtype=dtype, device=k_pages.device)
    if v_out is None:
        v_out = torch.zeros(shape, dtype=dtype, device=k_pages.device)
    if k_out.shape != shape or v_out.shape != shape:
        _shaped(k_out, shape, "k_out")
        _shaped(v_out, shape, "v_out")
    _call("sl8_paged_read_int4", dev, kc, ks, vc, vs, num_pages, page_size, _one(block_table, dev, _I32T, "block_table"), max_blocks,
          _one(seqlens, dev, _I32T, "seqlens"), cu, B, hkv, N, d, total, None if k_mean is None else _mean_of(dev, k_mean, hkv, d),
          _one(k_out, dev, dtype, "k_out"), _one(v_out, dev, dtype, "v_out"), _DTYPES[dtype])
    return k_out, v_out


def int4_decode_workspace_bytes(B: int, T: int, Hq: int, Hkv: int, max_blocks: int, page_size: int, d: int,
                                num_splits: int = 0) -> int:
    return int(lib().sl8_attn_int4_paged_decode_workspace_size(B, T, Hq, Hkv, max_blocks, page_size, d, num_splits))


def attn_int4_paged_decode(q, k_pages, k_scale_pages, v_pages, v_scale_pages, block_table, seqlens, tree_mask=None,
                           num_splits=0, out_dtype=None, return_lse=False, workspace=None, out=None, lse=None):
    """Decode attention over the paged 4-bit cache: q [B,Hq,d], or [B,T,Hq,d] with T <= 32 drafts whose
    tokens the cache holds (query t at position seqlens - T + t).  tree_mask [B,T] int32: bit u says
    that the query sees draft u (without it each sees the tokens up to itself).  Returns out like q
    (dtype q.dtype unless given) and, with return_lse, the fp32 LSE: 0 and -inf for a query that sees no
    token.  workspace: uint8, at least int4_decode_workspace_bytes (16: none is used)."""
    dev = _index(k_pages)
    num_pages, hkv, page_size, d, kc, ks, vc, vs = _pages4_of(dev, k_pages, k_scale_pages, v_pages, v_scale_pages)
    B, max_blocks = block_table.shape
    shape, dtype = q.shape, q.dtype
    if len(shape) not in (3, 4):
        raise ValueError("q must be [B, Hq, d] or [B, T, Hq, d]")
    T, hq = (1, shape[1]) if len(shape) == 3 else (shape[1], shape[2])
    if shape[0] != B or shape[-1] != d or seqlens.numel() != B:
        raise ValueError("q, block_table, seqlens and the pages do not belong together")
    mask = None
    if tree_mask is not None:
        if tree_mask.numel() != B * T:
            raise ValueError("tree_mask needs one entry per query")
        mask = _one(tree_mask, dev, _I32T, "tree_mask")
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or dtype, device=q.device)
    elif out.shape != shape:
        raise ValueError("out must have q's shape")
    odt = out.dtype
    if dtype not in _DTYPES or odt not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype} or {odt}")
    lse_p = None
    if return_lse:
        if lse is None:
            lse = torch.empty(shape[:-1], dtype=_F32T, device=q.device)
        elif lse.shape != shape[:-1]:
            raise ValueError("lse must have one entry per query head")
        lse_p = _one(lse, dev, _F32T, "lse")
    ws, nbytes = None, 0
    if workspace is None:
        need = int4_decode_workspace_bytes(B, T, hq, hkv, max_blocks, page_size, d, num_splits)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need > 16 else None
    if workspace is not None:
        ws = _one(workspace, dev, workspace.dtype, "workspace")
        nbytes = workspace.numel() * workspace.element_size()
    _call("sl8_attn_int4_paged_decode", dev, _one(q, dev, dtype, "q"), _DTYPES[dtype], kc, ks, vc, vs, num_pages, page_size,
          _one(block_table, dev, _I32T, "block_table"), max_blocks, _one(seqlens, dev, _I32T, "seqlens"), mask, T, B, hq, hkv, d,
          num_splits, _one(out, dev, odt, "out"), _DTYPES[odt], lse_p, ws, nbytes)
    return (out, lse) if return_lse else out


# ------------------------------------------------------------------ status / tracing

def last_device_status(device=None) -> tuple[int, int]:
    """(status, site) of the device's status word after synchronising the current stream; clears it."""
    site = _INT(0)
    dev = torch.device("cuda") if device is None else torch.device(device)
    st = lib().sl8_last_device_status(_stream(dev), ctypes.byref(site))
    return int(st), int(site.value)


def set_spin_limit_ns(ns: int) -> None:
    lib().sl8_set_spin_limit_ns(int(ns))


def get_spin_limit_ns() -> int:
    return int(lib().sl8_get_spin_limit_ns())


def selftest_timeout(limit_ns: int, device=None) -> None:
    dev = torch.device("cuda") if device is None else torch.device(device)
    _check(lib().sl8_selftest_timeout(int(limit_ns), _stream(dev)), "sl8_selftest_timeout")


def trace_enable(on: bool = True) -> None:
    lib().sl8_trace_enable(int(bool(on)))


def trace_collect(max_names: int = 64) -> dict[str, tuple[int, float]]:
    """{kernel name: (launches, total ms)} since the last collect (synchronises the traced events)."""
    names = (ctypes.c_char_p * max_names)()
    launches = (_I64 * max_names)()
    ms = (ctypes.c_double * max_names)()
    n = lib().sl8_trace_collect(names, launches, ms, max_names)
    return {names[i].decode(): (int(launches[i]), float(ms[i])) for i in range(n)}
