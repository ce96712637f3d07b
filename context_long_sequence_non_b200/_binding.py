"""ctypes binding of libcpattn.so (include/cpattn.h).  Argument marshalling only: every
step of the path runs in the library's CUDA kernels.  PyTorch provides device memory and
the current stream; nothing here computes on the host.  There is no fallback: if the
library is missing or a call fails, an exception is raised.
"""

from __future__ import annotations

import ctypes
import math
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcpattn.so")

BF16, F32 = 0, 1
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_CUDA, ERR_DEVICE_TIMEOUT = range(7)

_lock = threading.Lock()
_lib = None


class CpattnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)}")


def library_path() -> str:
    return LIB_PATH


def lib() -> ctypes.CDLL:
    """Load libcpattn.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m context_long_sequence_non_b200.build` (no CPU fallback exists)")
            L = ctypes.CDLL(LIB_PATH)
            vp, i, f, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong
            L.cpattn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
            L.cpattn_fwd_accumulate.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
            L.cpattn_ulysses_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
            L.cpattn_ulysses_fwd_split.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp,
                                                   ctypes.c_size_t, vp]
            L.cpattn_ulysses_fwd_workspace.argtypes = [i, i, i, i, i]
            L.cpattn_ulysses_fwd_workspace.restype = ctypes.c_size_t
            L.cpattn_ulysses_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i,
                                              f, i, i, vp]
            L.cpattn_fwd_split.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, i, vp,
                                           ctypes.c_size_t, vp]
            L.cpattn_fwd_split_workspace.argtypes = [i, i, i, i, i, i]
            L.cpattn_fwd_split_workspace.restype = ctypes.c_size_t
            L.cpattn_fwd_split_workspace_kv.argtypes = [i, i, i, i, i, i, i]
            L.cpattn_fwd_split_workspace_kv.restype = ctypes.c_size_t
            L.cpattn_split_suggest.argtypes = [i, i, i, i]
            L.cpattn_merge.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp]
            L.cpattn_seq2head.argtypes = [vp, vp, i, i, i, i, i, vp]
            L.cpattn_head2seq.argtypes = [vp, vp, i, i, i, i, i, vp]
            L.cpattn_seq2head_qkv.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp]
            L.cpattn_rmsnorm.argtypes = [vp, vp, vp, i, i, f, f, vp]
            L.cpattn_seq2head_qkv_norm.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f,
                                                   f, vp]
            d = ctypes.c_double
            L.cpattn_window_fwd.argtypes = [vp] * 7 + [i] * 6 + [ll] * 3 + [f] + [i] * 8 + [vp]
            L.cpattn_window_decode.argtypes = [vp] * 6 + [i] * 6 + [ll] * 3 + [f] + [i] * 4 + [vp]
            L.cpattn_rope_frequencies.argtypes = [vp, vp, i, d, i, d, d, d, d]
            L.cpattn_rope.argtypes = [vp] * 4 + [i] * 7 + [f, ll, ll, i, vp]
            L.cpattn_qk_norm_rope.argtypes = [vp] * 8 + [i] * 8 + [f] * 3 + [ll] * 4 + [i, vp]
            L.cpattn_seq2head_qkv_norm_rope.argtypes = [vp] * 10 + [i] * 7 + [f] * 3 + [vp]
            L.cpattn_call.argtypes = [i, ctypes.c_char_p, i]
            L.cpattn_status_str.argtypes = [i]
            L.cpattn_status_str.restype = ctypes.c_char_p
            L.cpattn_device_error.argtypes = []
            L.cpattn_selftest_wait_timeout.argtypes = [ll, vp]
            L.cpattn_version.argtypes = []
            L.cpattn_selftest_exp2.argtypes = [vp, vp, i, vp]
            for name in ("cpattn_fwd", "cpattn_fwd_accumulate", "cpattn_ulysses_fwd",
                         "cpattn_ulysses_fwd_split", "cpattn_ulysses_host",
                         "cpattn_fwd_split", "cpattn_split_suggest", "cpattn_merge", "cpattn_seq2head_qkv", "cpattn_seq2head", "cpattn_head2seq",
                         "cpattn_device_error", "cpattn_selftest_wait_timeout", "cpattn_version",
                         "cpattn_selftest_exp2", "cpattn_window_fwd", "cpattn_window_decode",
                         "cpattn_rope_frequencies", "cpattn_rope", "cpattn_qk_norm_rope",
                         "cpattn_seq2head_qkv_norm_rope", "cpattn_call"):
                getattr(L, name).restype = ctypes.c_int
            _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().cpattn_status_str(int(status)).decode()


def _check(status: int, what: str):
    if status != OK:
        raise CpattnError(status, what)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return BF16
    if t == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensors must live on a CUDA device")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")


def _need_shape(t, shape, name, dtype=None):
    """A caller-provided output must have exactly the size the call writes: the library
    receives only its pointer."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def on_stream(stream, device, make):
    """``make()``, tensors for a call that runs on ``stream`` (None: the current one), with that stream
    current, so that they come from its memory.  The current stream's could be memory that work queued
    there still uses, and would go to its next allocation as soon as Python drops the tensor, both while
    the call runs.  They are marked as used on the current stream too, where the caller reads them."""
    if stream is None:
        return make()
    here = torch.cuda.current_stream(device)
    if stream == here:
        return make()
    with torch.cuda.stream(stream):
        made = make()
    for t in made if isinstance(made, tuple) else (made,):
        t.record_stream(here)
    return made


def _empty(stream, shape, dtype, device):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return on_stream(stream, device, lambda: torch.empty(shape, dtype=dtype, device=device))


def fwd(q, k, v, out=None, lse=None, scale=None, out_dtype=None, want_lse=True, stream=None):
    """Non-causal attention ``softmax(scale * Q K^T) V`` with its log-sum-exp.

    q: [B][Sq][H][D], k/v: [B][Skv][H][D] (bf16 -> tcgen05 kernel, fp32 -> CUDA-core
    kernel).  Returns ``(out [B][Sq][H][D], lse [B][H][Sq] float32)``.
    """
    B, Sq, H, D = q.shape
    Skv = k.shape[1]
    if k.shape != (B, Skv, H, D) or v.shape != (B, Skv, H, D):
        raise ValueError("k and v must be [B][Skv][H][D] matching q")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out_dtype is None:
        out_dtype = q.dtype
    if out is None:
        out = _empty(stream, (B, Sq, H, D), out_dtype, q.device)
    if lse is None and want_lse:
        lse = _empty(stream, (B, H, Sq), torch.float32, q.device)
    _need_shape(out, (B, Sq, H, D), "out")
    _need_shape(lse, (B, H, Sq), "lse", torch.float32)
    _need_cuda(q, k, v, out, lse)
    st = lib().cpattn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Sq, Skv, D,
                          float(scale), _dtype_code(q.dtype), _dtype_code(out.dtype),
                          _stream(stream))
    _check(st, "cpattn_fwd")
    return out, lse


def ulysses_fwd(q, k, v, P, out=None, lse=None, scale=None, out_dtype=None, want_lse=True,
                stream=None):
    """Ulysses attention in one kernel: q/k/v/out are [P][S_l][H][D] rank shards; returns
    ``(out, lse [P][H/P][P*S_l])`` equal to seq2head -> fwd -> head2seq."""
    P_, S_l, H, D = q.shape
    if P_ != P or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must be same-shaped [P][S_l][H][D] shards")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _empty(stream, (P, S_l, H, D), out_dtype or q.dtype, q.device)
    if lse is None and want_lse:
        lse = _empty(stream, (P, H // P, P * S_l), torch.float32, q.device)
    _need_shape(out, (P, S_l, H, D), "out")
    _need_shape(lse, (P, H // P, P * S_l), "lse", torch.float32)
    _need_cuda(q, k, v, out, lse)
    st = lib().cpattn_ulysses_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), P, S_l, H, D,
                                  float(scale), _dtype_code(out.dtype), _stream(stream))
    _check(st, "cpattn_ulysses_fwd")
    return out, lse


def ulysses_workspace_bytes(P, S_l, H, D, out_dtype=torch.bfloat16) -> int:
    """Workspace bytes of ulysses_fwd_split for these shards (0: nothing to split)."""
    return int(lib().cpattn_ulysses_fwd_workspace(P, S_l, H, D, _dtype_code(out_dtype)))


def ulysses_fwd_split(q, k, v, P, out=None, lse=None, scale=None, out_dtype=None,
                      want_lse=True, workspace=None, stream=None):
    """ulysses_fwd with the tail split (the items of the GPU's last wave or two computed
    as key ranges and folded exactly).  ``workspace``: a uint8 CUDA tensor of at least
    ``ulysses_workspace_bytes(...)`` bytes, allocated here (by PyTorch) when omitted."""
    P_, S_l, H, D = q.shape
    if P_ != P or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must be same-shaped [P][S_l][H][D] shards")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _empty(stream, (P, S_l, H, D), out_dtype or q.dtype, q.device)
    if lse is None and want_lse:
        lse = _empty(stream, (P, H // P, P * S_l), torch.float32, q.device)
    _need_shape(out, (P, S_l, H, D), "out")
    _need_shape(lse, (P, H // P, P * S_l), "lse", torch.float32)
    need = ulysses_workspace_bytes(P, S_l, H, D, out.dtype)
    if workspace is None and need > 0:
        workspace = _empty(stream, (need,), torch.uint8, q.device)
    _need_cuda(q, k, v, out, lse, workspace)
    st = lib().cpattn_ulysses_fwd_split(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), P, S_l,
                                        H, D, float(scale), _dtype_code(out.dtype),
                                        _ptr(workspace), _nbytes(workspace), _stream(stream))
    _check(st, "cpattn_ulysses_fwd_split")
    return out, lse


def ulysses_host(hq, hk, hv, h_out, h_lse, dq, dk, dv, d_out, d_lse, P, scale=None,
                 n_chunks=None, stream=None):
    """Ulysses attention from host shards to host O/LSE through cpattn_ulysses_host: the
    copies are pipelined with the attention over head-group chunks.  h_*: CPU tensors
    (pinned for asynchronous copies); d_*: same-shaped CUDA work buffers.  The host
    outputs are valid once ``stream`` (default: the current stream) has passed the call."""
    P_, S_l, H, D = hq.shape
    for t in (hk, hv, dq, dk, dv):
        if t.shape != hq.shape:
            raise ValueError("all shard tensors must be [P][S_l][H][D]")
    if h_out.shape != hq.shape or d_out.shape != hq.shape or h_out.dtype != d_out.dtype:
        raise ValueError("h_out and d_out must be [P][S_l][H][D] of one dtype")
    if (h_lse is None) != (d_lse is None):
        raise ValueError("h_lse and d_lse go together")
    for t in (hq, hk, hv, h_out, h_lse):
        if t is not None and (t.is_cuda or not t.is_contiguous()):
            raise ValueError("host tensors must be contiguous CPU tensors")
    _need_cuda(dq, dk, dv, d_out, d_lse)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if n_chunks is None:
        n_chunks = P
    st = lib().cpattn_ulysses_host(_ptr(hq), _ptr(hk), _ptr(hv), _ptr(h_out), _ptr(h_lse),
                                   _ptr(dq), _ptr(dk), _ptr(dv), _ptr(d_out), _ptr(d_lse), P,
                                   S_l, H, D, float(scale), _dtype_code(d_out.dtype),
                                   int(n_chunks), _stream(stream))
    _check(st, "cpattn_ulysses_host")
    return h_out, h_lse


def split_workspace_bytes(B, H, Sq, D, n_split, out_dtype=torch.bfloat16, Skv=None) -> int:
    """Workspace bytes of fwd_split: exact for the key count ``Skv`` when given, else (for
    the tail split, n_split = 0) the largest any key count can need."""
    if Skv is not None:
        return int(lib().cpattn_fwd_split_workspace_kv(B, H, Sq, Skv, D, n_split,
                                                       _dtype_code(out_dtype)))
    return int(lib().cpattn_fwd_split_workspace(B, H, Sq, D, n_split, _dtype_code(out_dtype)))


def split_suggest(B, H, Sq, Skv) -> int:
    return int(lib().cpattn_split_suggest(B, H, Sq, Skv))


def fwd_split(q, k, v, out=None, lse=None, scale=None, out_dtype=None, accumulate=False,
              n_split=None, workspace=None, stream=None):
    """Split-KV attention: ``n_split`` key ranges computed as separate CTAs, their partials
    folded exactly (into the running (out, lse) when ``accumulate``).  ``workspace`` is a
    uint8 CUDA tensor of at least ``split_workspace_bytes(...)`` bytes (allocated here when
    omitted -- by PyTorch; the library allocates nothing)."""
    B_, Sq, H, D = q.shape
    Skv = k.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _empty(stream, (B_, Sq, H, D), out_dtype or q.dtype, q.device)
    if lse is None:
        lse = _empty(stream, (B_, H, Sq), torch.float32, q.device)
    if k.shape != (B_, Skv, H, D) or v.shape != (B_, Skv, H, D):
        raise ValueError("k and v must be [B][Skv][H][D] matching q")
    _need_shape(out, (B_, Sq, H, D), "out")
    _need_shape(lse, (B_, H, Sq), "lse", torch.float32)
    if n_split is None:
        n_split = split_suggest(B_, H, Sq, Skv)
    need = split_workspace_bytes(B_, H, Sq, D, n_split, out.dtype, Skv=Skv)
    if workspace is None:
        workspace = _empty(stream, (max(need, 256),), torch.uint8, q.device)
    _need_cuda(q, k, v, out, lse, workspace)
    st = lib().cpattn_fwd_split(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B_, H, Sq, Skv,
                                D, float(scale), _dtype_code(out.dtype), 1 if accumulate else 0,
                                int(n_split), _ptr(workspace), _nbytes(workspace),
                                _stream(stream))
    _check(st, "cpattn_fwd_split")
    return out, lse


def fwd_accumulate(q, k, v, o_acc, lse_acc, scale=None, stream=None):
    """Ring Attention step with the merge fused into the attention epilogue: attention of
    q over this K/V chunk, merged in place into the running (o_acc, lse_acc)."""
    B, Sq, H, D = q.shape
    Skv = k.shape[1]
    if k.shape != (B, Skv, H, D) or v.shape != (B, Skv, H, D):
        raise ValueError("k and v must be [B][Skv][H][D] matching q")
    if o_acc.shape != (B, Sq, H, D) or lse_acc.shape != (B, H, Sq):
        raise ValueError("o_acc must be [B][Sq][H][D] and lse_acc [B][H][Sq]")
    _need_shape(lse_acc, (B, H, Sq), "lse_acc", torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    _need_cuda(q, k, v, o_acc, lse_acc)
    st = lib().cpattn_fwd_accumulate(_ptr(q), _ptr(k), _ptr(v), _ptr(o_acc), _ptr(lse_acc), B, H,
                                     Sq, Skv, D, float(scale), _dtype_code(q.dtype),
                                     _dtype_code(o_acc.dtype), _stream(stream))
    _check(st, "cpattn_fwd_accumulate")
    return o_acc, lse_acc


def merge(o_a, lse_a, o_b, lse_b, out=None, lse=None, stream=None):
    """Exact merge of two partial (O, LSE) results; ``out``/``lse`` may be o_a/lse_a."""
    B, S, H, D = o_a.shape
    if out is None:
        out = _empty(stream, o_a.shape, o_a.dtype, o_a.device)
    if lse is None:
        lse = _empty(stream, lse_a.shape, lse_a.dtype, lse_a.device)
    _need_shape(o_b, (B, S, H, D), "o_b", o_a.dtype)
    _need_shape(out, (B, S, H, D), "out", o_a.dtype)
    for name, t in (("lse_a", lse_a), ("lse_b", lse_b), ("lse", lse)):
        _need_shape(t, (B, H, S), name, torch.float32)
    _need_cuda(o_a, lse_a, o_b, lse_b, out, lse)
    st = lib().cpattn_merge(_ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), _ptr(out), _ptr(lse),
                            B, H, S, D, _dtype_code(o_a.dtype), _stream(stream))
    _check(st, "cpattn_merge")
    return out, lse


def seq2head(src, P, out=None, stream=None):
    """[P][S_l][H][D] sequence shards -> [P][P*S_l][H/P][D] head groups (bit copy)."""
    P_, S_l, H, D = src.shape
    if P_ != P:
        raise ValueError("src.shape[0] must equal P")
    if out is None:
        out = _empty(stream, (P, P * S_l, H // P, D), src.dtype, src.device)
    _need_shape(out, (P, P * S_l, H // P, D), "out", src.dtype)
    _need_cuda(src, out)
    st = lib().cpattn_seq2head(_ptr(src), _ptr(out), P, S_l, H, D, src.element_size(),
                               _stream(stream))
    _check(st, "cpattn_seq2head")
    return out


def seq2head_qkv(q, k, v, P, out=None, stream=None):
    """seq2head of Q, K and V in one launch; ``out`` is an optional (qh, kh, vh) triple."""
    P_, S_l, H, D = q.shape
    if P_ != P or k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must be same-shaped [P][S_l][H][D] tensors")
    if out is None:
        out = tuple(_empty(stream, (P, P * S_l, H // P, D), q.dtype, q.device)
                    for _ in range(3))
    for i, t in enumerate(out):
        _need_shape(t, (P, P * S_l, H // P, D), f"out[{i}]", q.dtype)
    _need_cuda(q, k, v, *out)
    st = lib().cpattn_seq2head_qkv(_ptr(q), _ptr(k), _ptr(v), *(_ptr(t) for t in out), P, S_l, H,
                                   D, q.element_size(), _stream(stream))
    _check(st, "cpattn_seq2head_qkv")
    return out


def rmsnorm(x, gamma, eps=1e-6, out_scale=1.0, out=None, stream=None):
    """RMSNorm of every head row (last axis, D) of a bf16 tensor with fp32 weights
    ``gamma[D]``; ``out=x`` normalises in place.  See cpattn_rmsnorm."""
    if x.dtype != torch.bfloat16 or gamma.dtype != torch.float32 or gamma.shape != (x.shape[-1],):
        raise ValueError("x must be bf16 [..., D] and gamma float32 [D]")
    if out is None:
        out = _empty(stream, x.shape, x.dtype, x.device)
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out must match x")
    _need_cuda(x, gamma, out)
    D = x.shape[-1]
    st = lib().cpattn_rmsnorm(_ptr(x), _ptr(out), _ptr(gamma), x.numel() // D, D, float(eps),
                              float(out_scale), _stream(stream))
    _check(st, "cpattn_rmsnorm")
    return out


def seq2head_qkv_norm(q, k, v, P, gamma_q, gamma_k, eps=1e-6, out_scale=1.0, out=None,
                      stream=None):
    """seq2head of Q, K, V in one launch with Q and K head rows RMS-normalised on the way
    (weights gamma_q / gamma_k, float32 [D]); ``out`` is an optional (qh, kh, vh) triple."""
    P_, S_l, H, D = q.shape
    if P_ != P or k.shape != q.shape or v.shape != q.shape or any(
            t.dtype != torch.bfloat16 for t in (q, k, v)):
        raise ValueError("q, k, v must be same-shaped bf16 [P][S_l][H][D] tensors")
    for g in (gamma_q, gamma_k):
        if g.dtype != torch.float32 or g.shape != (D,):
            raise ValueError("gamma_q and gamma_k must be float32 [D]")
    if out is None:
        out = tuple(_empty(stream, (P, P * S_l, H // P, D), q.dtype, q.device)
                    for _ in range(3))
    for i, t in enumerate(out):
        _need_shape(t, (P, P * S_l, H // P, D), f"out[{i}]", q.dtype)
    _need_cuda(q, k, v, gamma_q, gamma_k, *out)
    st = lib().cpattn_seq2head_qkv_norm(_ptr(q), _ptr(k), _ptr(v), *(_ptr(t) for t in out),
                                        _ptr(gamma_q), _ptr(gamma_k), P, S_l, H, D, float(eps),
                                        float(out_scale), _stream(stream))
    _check(st, "cpattn_seq2head_qkv_norm")
    return out


def head2seq(src, P, out=None, stream=None):
    """[P][P*S_l][Hp][D] head groups -> [P][S_l][P*Hp][D] sequence shards (bit copy)."""
    P_, S_full, Hp, D = src.shape
    if P_ != P or S_full % P:
        raise ValueError("src must be [P][P*S_l][Hp][D]")
    S_l, H = S_full // P, Hp * P
    if out is None:
        out = _empty(stream, (P, S_l, H, D), src.dtype, src.device)
    _need_shape(out, (P, S_l, H, D), "out", src.dtype)
    _need_cuda(src, out)
    st = lib().cpattn_head2seq(_ptr(src), _ptr(out), P, S_l, H, D, src.element_size(),
                               _stream(stream))
    _check(st, "cpattn_head2seq")
    return out


# ------------------------------------------------------------------ windowed attention


# The current stream and device, without the wrapper objects (these calls are a few microseconds
# of host time in all, and the wrappers were four of them).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class _Entry:
    """A call that goes through cpattn_call: its number and the layout of its words (P pointer,
    q integer, d float; the stream is the last P)."""

    def __init__(self, name, code, layout):
        self.name, self.code, self.n = name, code, struct.calcsize("=" + layout.replace("P", "Q")) // 8
        self.pack = struct.Struct("=" + layout.replace("P", "Q")).pack


_WINDOW_FWD = _Entry("cpattn_window_fwd", 0, "7P9qd8qP")
_WINDOW_DECODE = _Entry("cpattn_window_decode", 1, "6P9qd4qP")
_ROPE = _Entry("cpattn_rope", 2, "4P7qd3qP")
_QK_NORM_ROPE = _Entry("cpattn_qk_norm_rope", 3, "8P8q3d5qP")
_SEQ2HEAD_QKV_NORM_ROPE = _Entry("cpattn_seq2head_qkv_norm_rope", 4, "10P7q3dP")


def _call(index, stream, entry, *args):
    """Run a library call with CUDA device ``index`` current (the library launches on the current
    device) on ``stream``, or on that device's current stream.  Pointers are addresses, 0: none."""
    if stream is None:
        raw = _raw_stream(index)
    elif stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    else:
        raw = stream.cuda_stream
    words = entry.pack(*args, raw)
    if _current_device() == index:
        st = lib().cpattn_call(entry.code, words, entry.n)
    else:
        with torch.cuda.device(index):
            st = lib().cpattn_call(entry.code, words, entry.n)
    if st != OK:
        raise CpattnError(st, entry.name)


def _same_device(first, *ts):
    """The CUDA device index that every tensor is on."""
    index = first.get_device()  # -1: not a CUDA tensor
    if index < 0:
        raise ValueError("tensors must live on a CUDA device")
    for t in ts:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors must live on one CUDA device")
    return index


def _token_stride(t, name):
    """Elements between consecutive tokens of a [..., tokens, heads, D] tensor whose heads are
    packed and whose tokens are evenly spaced through every leading axis (0: packed tokens)."""
    if t.is_contiguous():
        return 0
    shape, stride = t.shape, t.stride()
    D, H = shape[-1], shape[-2]
    if (D > 1 and stride[-1] != 1) or (H > 1 and stride[-2] != D):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    step, count = None, 1  # tokens are `step` apart; `count` of them below the axis at hand
    for n, st in zip(reversed(shape[:-2]), reversed(stride[:-2])):
        if n > 1:
            if step is None:
                step = st
            elif st != step * count:
                raise ValueError(f"{name}: tokens must be evenly spaced")
        count *= n
    if step is None:
        return 0
    if step < H * D:
        raise ValueError(f"{name}: tokens must not overlap")
    return step


def _packed(t, shape, name, dtype):
    if t.shape == shape and (dtype is None or t.dtype == dtype) and t.is_contiguous():
        return
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


def _packed_like(t, dtype, stream):
    """A new contiguous tensor of t's shape.  (A contiguous t's own layout will do, in half the time.)"""
    if stream is not None:
        return _empty(stream, t.shape, dtype, t.device)
    if t.is_contiguous():
        return torch.empty_like(t) if t.dtype == dtype else torch.empty_like(t, dtype=dtype)
    return torch.empty(t.shape, dtype=dtype, device=t.device)


def _extent(n, name):
    n = int(n)
    if not -(1 << 31) <= n < 1 << 31:
        raise ValueError(f"{name} is out of range")
    return n


_CODE = {torch.bfloat16: BF16, torch.float32: F32}


def _window_args(q, k, v, kv_len, out, lse, scale, out_dtype, want_lse, stream):
    q_shape, kv_shape, dtype = q.shape, k.shape, q.dtype
    if len(q_shape) != 4 or len(kv_shape) != 4:
        raise ValueError("q, k and v must be [B][S][H][D]")
    B, Sq, H, D = q_shape
    Bk, Skv, Hkv, Dk = kv_shape
    if Bk != B or Dk != D or v.shape != kv_shape:
        raise ValueError("k and v must be [B][Skv][Hkv][D] matching q")
    if k.dtype != dtype or v.dtype != dtype:
        raise ValueError("q, k and v must have one dtype")
    # 0: packed tokens
    qs = 0 if q.is_contiguous() else _token_stride(q, "q")
    ks = 0 if k.is_contiguous() else _token_stride(k, "k")
    vs = 0 if v.is_contiguous() else _token_stride(v, "v")
    if kv_len is not None:
        _packed(kv_len, (B,), "kv_len", torch.int32)
    if out is None:
        out = _packed_like(q, out_dtype or dtype, stream)
    else:
        _packed(out, q_shape, "out", out_dtype)
    if lse is not None:
        _packed(lse, (B, H, Sq), "lse", torch.float32)
    elif want_lse:
        if stream is None:
            lse = torch.empty_strided((B, H, Sq), (H * Sq, Sq, 1), dtype=torch.float32, device=q.device)
        else:
            lse = _empty(stream, (B, H, Sq), torch.float32, q.device)
    index = _same_device(q, k, v, kv_len, out, lse)
    codes = _CODE.get(dtype), _CODE.get(out.dtype)
    if None in codes:
        raise TypeError(f"unsupported dtype {dtype if codes[0] is None else out.dtype}")
    return (index, (B, H, Hkv, Sq, Skv, D, qs, ks, vs, 1.0 / math.sqrt(D) if scale is None else float(scale)),
            codes, out, lse)


def window_fwd(q, k, v, left=-1, right=-1, sinks=0, q_pos=0, k_pos=0, kv_len=None, out=None,
               lse=None, scale=None, out_dtype=None, want_lse=True, accumulate=False, run=None, stream=None):
    """Attention limited to a window: the query at position p = q_pos + i sees the keys at
    positions p - left .. p + right (-1: no bound on that side) and, up to p + right, those below
    ``sinks``; see cpattn_window_fwd.

    q: [B][Sq][H][D], k/v: [B][Skv][Hkv][D] with H a multiple of Hkv (bf16 -> tensor-core kernel,
    D 64 or 128; fp32 -> CUDA-core kernel, D <= 256); their heads may be slices of a wider row.
    ``kv_len``: int32 [B], keys of each sequence.  ``accumulate`` (bf16) merges into the running
    (out, lse), or merges the running (``run`` float32, lse) into a bf16 ``out``.
    Returns ``(out [B][Sq][H][D], lse [B][H][Sq] float32)``."""
    if accumulate and (lse is None or (out is None and run is None)):
        raise ValueError("accumulate needs the running out and lse")
    if run is not None:
        if not accumulate:
            raise ValueError("run is the running result of an accumulating call")
        _packed(run, q.shape, "run", torch.float32)
    index, dims, codes, out, lse = _window_args(q, k, v, kv_len, out, lse, scale, out_dtype, want_lse,
                                                stream)
    if run is not None:
        _same_device(q, run)
    _call(index, stream, _WINDOW_FWD, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
          0 if lse is None else lse.data_ptr(), 0 if kv_len is None else kv_len.data_ptr(),
          0 if run is None else run.data_ptr(), *dims, _extent(q_pos, "q_pos"), _extent(k_pos, "k_pos"),
          _extent(left, "left"), _extent(right, "right"), _extent(sinks, "sinks"), *codes,
          1 if accumulate else 0)
    return out, lse


def window_decode(q, k_cache, v_cache, kv_len=None, left=-1, sinks=0, out=None, lse=None, scale=None,
                  out_dtype=None, want_lse=True, stream=None):
    """The last Sq tokens of each sequence against its cache (causal, window and sinks as
    window_fwd): q [B][Sq][H][D], caches [B][S_max][Hkv][D], ``kv_len`` int32 [B] the tokens each
    sequence holds, the newest included (None: S_max).  See cpattn_window_decode."""
    index, dims, codes, out, lse = _window_args(q, k_cache, v_cache, kv_len, out, lse, scale, out_dtype,
                                                want_lse, stream)
    _call(index, stream, _WINDOW_DECODE, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          0 if kv_len is None else kv_len.data_ptr(), out.data_ptr(),
          0 if lse is None else lse.data_ptr(), *dims, _extent(left, "left"), _extent(sinks, "sinks"), *codes)
    return out, lse


# ------------------------------------------------------------------ rotary positions

ROPE_SCALING = {"plain": 0, "linear": 1, "ntk": 2, "by_parts": 3}


def rope_frequencies(rot, base=10000.0, scaling="plain", stretch=1.0, train_len=0.0, beta_fast=32.0,
                     beta_slow=1.0, device="cpu"):
    """``(freq float64 [rot/2], factor)``: radians per position of each rotated pair and the
    factor on the rotated part, see cpattn_rope_frequencies."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {tuple(ROPE_SCALING)}")
    rot = _extent(rot, "rot")
    freq = torch.empty(max(rot // 2, 0), dtype=torch.float64)
    factor = ctypes.c_float()
    _check(lib().cpattn_rope_frequencies(freq.data_ptr(), ctypes.addressof(factor), rot, float(base),
                                         ROPE_SCALING[scaling], float(stretch), float(train_len),
                                         float(beta_fast), float(beta_slow)),
           "cpattn_rope_frequencies")
    return freq.to(device), factor.value


def rope_axes(freqs):
    """[axes][rot/2] frequencies of a multi-axis rotation: axis a turns its own run of pairs with
    the frequencies ``freqs[a]``, the runs in order."""
    n = sum(f.numel() for f in freqs)
    out = torch.zeros(len(freqs), n, dtype=torch.float64, device=freqs[0].device)
    at = 0
    for a, f in enumerate(freqs):
        out[a, at:at + f.numel()] = f
        at += f.numel()
    return out


def _rope_args(tokens, pos, freq):
    f, p = freq.shape, pos.shape
    if freq.dtype != torch.float64 or not 1 <= len(f) <= 2 or not freq.is_contiguous():
        raise ValueError("freq must be a contiguous float64 [rot/2] or [axes][rot/2]")
    axes = 1 if len(f) == 1 else f[0]
    if pos.dtype != torch.int32 or not pos.is_contiguous():
        raise ValueError("pos must be contiguous int32")
    if axes == 0 or (len(p) > 1 and p[-1] != axes) or (len(p) < 2 and axes > 1):
        raise ValueError("pos must be [rows] or [..., rows, axes] matching freq")
    rows = pos.numel() // axes
    if tokens and (rows < 1 or tokens % rows):
        raise ValueError("the tokens must be a multiple of pos's rows")
    return rows, axes, 2 * f[-1]


def rope(x, pos, freq, interleaved=False, factor=1.0, out=None, stream=None):
    """Rotary positions of x [..., tokens, H, D] (bf16 or fp32): the first rot elements of every
    head turn by ``pos @ freq`` (pos int32 [rows] or [rows][axes], freq float64 [rot/2] or
    [axes][rot/2]); ``out=x`` rotates in place.  See cpattn_rope."""
    shape, dtype = x.shape, x.dtype
    if len(shape) < 3:
        raise ValueError("x must be [..., tokens, H, D]")
    H, D = shape[-2], shape[-1]
    tokens = shape[0] if len(shape) == 3 else shape[:-2].numel()
    rows, axes, rot = _rope_args(tokens, pos, freq)
    xs = 0 if x.is_contiguous() else _token_stride(x, "x")
    if out is None:
        out, ys = _packed_like(x, dtype, stream), 0
    else:
        if out.shape != shape or out.dtype != dtype:
            _need_shape(out, shape, "out", dtype)
        ys = xs if out is x else _token_stride(out, "out")
    index = _same_device(x, pos, freq, out)
    _call(index, stream, _ROPE, x.data_ptr(), out.data_ptr(), pos.data_ptr(), freq.data_ptr(), tokens, rows, H, D,
          rot, axes, 1 if interleaved else 0, float(factor), xs, ys, _dtype_code(dtype))
    return out


def qk_norm_rope(q, k, gamma_q, gamma_k, pos, freq, interleaved=False, factor=1.0, eps=1e-6,
                 out_scale=1.0, out=None, stream=None):
    """RMSNorm (weights float32 [D]) and rotary positions of query heads q [..., tokens, Hq, D]
    and key heads k [..., tokens, Hk, D] in one pass; ``out`` is an optional (q, k) pair, which
    may be (q, k) themselves.  See cpattn_qk_norm_rope."""
    if q.dim() < 3 or q.shape[:-2] != k.shape[:-2] or q.shape[-1] != k.shape[-1] or q.dtype != k.dtype:
        raise ValueError("q and k must be [..., tokens, H, D] of the same tokens, D and dtype")
    D = q.shape[-1]
    tokens = q.shape[:-2].numel()
    for g in (gamma_q, gamma_k):
        if g.dtype != torch.float32 or g.shape != (D,) or not g.is_contiguous():
            raise ValueError("gamma_q and gamma_k must be float32 [D]")
    rows, axes, rot = _rope_args(tokens, pos, freq)
    qs, ks = _token_stride(q, "q"), _token_stride(k, "k")
    if out is None:
        qo, ko, qos, kos = _packed_like(q, q.dtype, stream), _packed_like(k, k.dtype, stream), 0, 0
    else:
        qo, ko = out
        _need_shape(qo, q.shape, "out[0]", q.dtype)
        _need_shape(ko, k.shape, "out[1]", k.dtype)
        qos, kos = _token_stride(qo, "out[0]"), _token_stride(ko, "out[1]")
    index = _same_device(q, k, gamma_q, gamma_k, pos, freq, qo, ko)
    _call(index, stream, _QK_NORM_ROPE, q.data_ptr(), k.data_ptr(), qo.data_ptr(), ko.data_ptr(),
          gamma_q.data_ptr(), gamma_k.data_ptr(), pos.data_ptr(), freq.data_ptr(), tokens, rows, q.shape[-2],
          k.shape[-2], D, rot, axes, 1 if interleaved else 0, float(eps), float(out_scale), float(factor),
          qs, ks, qos, kos, _dtype_code(q.dtype))
    return qo, ko


def seq2head_qkv_norm_rope(q, k, v, P, gamma_q, gamma_k, pos, freq, interleaved=False, factor=1.0,
                           eps=1e-6, out_scale=1.0, out=None, stream=None):
    """seq2head of Q, K, V in one launch with Q and K head rows normalised (weights float32 [D];
    both None: not) and rotated on the way; pos [P*S_l] or [P*S_l][axes] in the order of the full
    sequence.  ``out`` is an optional (qh, kh, vh) triple.  See cpattn_seq2head_qkv_norm_rope."""
    if q.dim() != 4 or q.shape[0] != P or k.shape != q.shape or v.shape != q.shape or any(
            t.dtype != torch.bfloat16 for t in (q, k, v)):
        raise ValueError("q, k, v must be same-shaped bf16 [P][S_l][H][D] tensors")
    P, S_l, H, D = q.shape
    if (gamma_q is None) != (gamma_k is None):
        raise ValueError("gamma_q and gamma_k go together")
    for g in (gamma_q, gamma_k):
        if g is not None and (g.dtype != torch.float32 or g.shape != (D,) or not g.is_contiguous()):
            raise ValueError("gamma_q and gamma_k must be float32 [D]")
    rows, axes, rot = _rope_args(P * S_l, pos, freq)
    if rows != P * S_l:
        raise ValueError("pos must have a row for every token of the full sequence")
    grouped = (P, P * S_l, H // P, D)
    if out is None:
        out = tuple(_empty(stream, grouped, q.dtype, q.device) for _ in range(3))
    for i, t in enumerate(out):
        _packed(t, grouped, f"out[{i}]", q.dtype)
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous")
    index = _same_device(q, k, v, gamma_q, gamma_k, pos, freq, *out)
    _call(index, stream, _SEQ2HEAD_QKV_NORM_ROPE, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          *(t.data_ptr() for t in out), 0 if gamma_q is None else gamma_q.data_ptr(),
          0 if gamma_k is None else gamma_k.data_ptr(), pos.data_ptr(), freq.data_ptr(), P, S_l, H, D, rot, axes,
          1 if interleaved else 0, float(eps), float(out_scale), float(factor))
    return out


def device_error() -> int:
    """Synchronize and read/clear the device error word (OK or ERR_DEVICE_TIMEOUT)."""
    return lib().cpattn_device_error()


def selftest_wait_timeout(limit_cycles: int, stream=None):
    _check(lib().cpattn_selftest_wait_timeout(int(limit_cycles), _stream(stream)),
           "cpattn_selftest_wait_timeout")


def selftest_exp2(t, out=None, stream=None):
    """The attention kernel's FMA-pipe 2^t on a float32 CUDA tensor (test hook)."""
    if out is None:
        out = _empty(stream, t.shape, t.dtype, t.device)
    _need_cuda(t, out)
    _check(lib().cpattn_selftest_exp2(_ptr(t), _ptr(out), t.numel(), _stream(stream)),
           "cpattn_selftest_exp2")
    return out


def version() -> int:
    return lib().cpattn_version()
