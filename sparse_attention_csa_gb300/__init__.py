"""GB300 (sm_103a) forward path of DeepSeek-V4 Compressed Sparse Attention
(THD, and BSND batches), the backward of its sparse MLA attention and the
indexer's KL-loss gradient; rotary positions, and the same layers for new
tokens over paged caches.

Thin Python binding of the C ABI declared in ``include/csa.h`` (same call
names). It only marshals arguments: every step of the path runs in the CUDA
kernels of ``libcsa_gb300.so``; there is no CPU or PyTorch fallback, and a
call fails loudly when the library has not been built.

PyTorch supplies device memory and the current CUDA stream. All tensors are
CUDA tensors in THD layout, contiguous, with the dtypes ``include/csa.h``
states (bf16 activations, fp32 weights/sinks/outputs, int32 indices).

The rotation and the paged calls make results and workspaces that they are not
given from the memory of the call's ``stream``: used on another stream, such a
result needs what any tensor of that stream needs (an event, and
``record_stream`` where it may be freed early). The other calls make theirs
from the current stream's; given a ``stream`` that is not the current one, pass
them their outputs.
"""

from __future__ import annotations

import ctypes as C
import os

import torch

__all__ = [
    "CsaError", "lib", "library_path", "csa_status_string", "csa_compress_cu_seqlens",
    "csa_window_idx", "csa_indexer_topk_workspace_size", "csa_indexer_topk",
    "csa_sparse_mla_fwd", "csa_sparse_mla_bwd", "csa_device_error", "csa_indexer_topk_noalloc",
    "csa_indexer_kl_loss_grad", "csa_bsnd_mla_workspace_size", "csa_sparse_mla_fwd_bsnd",
    "csa_bsnd_indexer_workspace_size", "csa_indexer_topk_bsnd", "csa_compress_thd",
    "csa_rope_freqs", "csa_rope", "csa_cache_append", "csa_indexer_topk_paged_workspace_size",
    "csa_indexer_topk_paged", "csa_sparse_mla_paged_workspace_size", "csa_sparse_mla_paged",
    "csa_set_wait_limit_ns", "csa_set_pair_select_rows", "EXPORTED_SYMBOLS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "_build", "libcsa_gb300.so")

# Every entry point include/csa.h declares.
EXPORTED_SYMBOLS = (
    "csa_status_string", "csa_compress_cu_seqlens", "csa_window_idx",
    "csa_indexer_topk_workspace_size", "csa_indexer_topk", "csa_sparse_mla_fwd",
    "csa_sparse_mla_bwd", "csa_device_error", "csa_indexer_topk_noalloc",
    "csa_indexer_kl_loss_grad", "csa_bsnd_mla_workspace_size", "csa_sparse_mla_fwd_bsnd",
    "csa_bsnd_indexer_workspace_size", "csa_indexer_topk_bsnd", "csa_compress_thd",
    "csa_rope_freqs", "csa_rope", "csa_cache_append", "csa_indexer_topk_paged_workspace_size",
    "csa_indexer_topk_paged", "csa_sparse_mla_paged_workspace_size", "csa_sparse_mla_paged",
    "csa_set_wait_limit_ns", "csa_set_pair_select_rows",
)

_STATUS = {0: "CSA_OK", 1: "CSA_ERR_NULL", 2: "CSA_ERR_SHAPE", 3: "CSA_ERR_UNSUPPORTED",
           4: "CSA_ERR_WORKSPACE", 5: "CSA_ERR_CUDA", 6: "CSA_ERR_DEVICE_CHECK",
           7: "CSA_ERR_TIMEOUT"}


class CsaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = int(code)
        super().__init__(f"{where}: {csa_status_string(code)}")


_lib = None
_vp, _i32, _sz, _f32 = C.c_void_p, C.c_int32, C.c_size_t, C.c_float
_i64, _f64 = C.c_int64, C.c_double


def lib():
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError(
                f"{library_path} is missing: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        L = C.CDLL(library_path)
        L.csa_status_string.restype = C.c_char_p
        L.csa_status_string.argtypes = [C.c_int]
        L.csa_compress_cu_seqlens.argtypes = [_vp, _i32, _i32, _vp, _vp]
        L.csa_window_idx.argtypes = [_vp, _i32, _i32, _i32, _i32, _vp, _vp]
        L.csa_indexer_topk_workspace_size.restype = _sz
        L.csa_indexer_topk_workspace_size.argtypes = [_i32] * 5
        L.csa_indexer_topk.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _i32, _i32,
                                       _i32, _vp, _vp, _vp, _sz, _vp]
        L.csa_sparse_mla_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                         _i32, _i32, _vp, _f32, _i32, _i32, _i32, _vp, _vp, _i32,
                                         _vp]
        L.csa_sparse_mla_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                         _i32, _i32, _i32, _i32, _i32, _vp, _f32, _i32, _i32,
                                         _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
        L.csa_device_error.argtypes = [_vp, C.POINTER(_i32)]
        L.csa_indexer_topk_noalloc.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp,
                                               _i32, _i32, _i32, _vp, _vp, _vp]
        L.csa_indexer_kl_loss_grad.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                               _vp, _vp, _i32, _i32, _i32, _f32, _vp, _vp, _vp,
                                               _vp, _vp]
        L.csa_bsnd_mla_workspace_size.restype = _sz
        L.csa_bsnd_mla_workspace_size.argtypes = [_i32] * 3
        L.csa_sparse_mla_fwd_bsnd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                              _i32, _i32, _vp, _f32, _i32, _i32, _i32, _vp, _vp,
                                              _i32, _vp, _sz, _vp]
        L.csa_bsnd_indexer_workspace_size.restype = _sz
        L.csa_bsnd_indexer_workspace_size.argtypes = [_i32] * 6
        L.csa_indexer_topk_bsnd.argtypes = [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                            _i32, _i32, _vp, _vp, _vp, _sz, _vp]
        L.csa_compress_thd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                       _i32, _vp, _vp]
        L.csa_rope_freqs.argtypes = [_i32, _f64, _f64, _i32, _f64, _f64, _vp, _vp]
        L.csa_rope.argtypes = [_vp, C.c_int, _i64, _vp, _vp, _i32, _i32, _vp, _i32, _i32, _i32,
                               _i32, _i32, C.c_int, _f32, _i32, _vp, _i64, _vp]
        L.csa_cache_append.argtypes = [_vp, C.c_int, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                       _i32, _i32, _vp, _i32, _i32, C.c_int, _f32, _i32, _vp, _vp]
        L.csa_indexer_topk_paged_workspace_size.restype = _sz
        L.csa_indexer_topk_paged_workspace_size.argtypes = [_i32] * 5
        L.csa_indexer_topk_paged.argtypes = [_vp] * 6 + [_i32] * 9 + [_vp, _vp, _vp, _sz, _vp]
        L.csa_sparse_mla_paged_workspace_size.restype = _sz
        L.csa_sparse_mla_paged_workspace_size.argtypes = [_i32, _i32]
        L.csa_sparse_mla_paged.argtypes = [_vp] * 8 + [_i32] * 11 + [_vp, _f32, _i32, _i32, _i32,
                                                                     _vp, _vp, _i32, _vp, _sz, _vp]
        L.csa_set_wait_limit_ns.argtypes = [C.c_uint64]
        L.csa_set_pair_select_rows.argtypes = [_i32]
        for name in ("csa_compress_cu_seqlens", "csa_window_idx", "csa_indexer_topk",
                     "csa_sparse_mla_fwd", "csa_sparse_mla_bwd", "csa_device_error",
                     "csa_indexer_topk_noalloc", "csa_indexer_kl_loss_grad",
                     "csa_sparse_mla_fwd_bsnd", "csa_indexer_topk_bsnd", "csa_compress_thd",
                     "csa_rope_freqs", "csa_rope", "csa_cache_append", "csa_indexer_topk_paged",
                     "csa_sparse_mla_paged", "csa_set_wait_limit_ns", "csa_set_pair_select_rows"):
            getattr(L, name).restype = C.c_int
        _lib = L
    return _lib


def csa_status_string(code: int) -> str:
    try:
        return lib().csa_status_string(int(code)).decode()
    except RuntimeError:
        return _STATUS.get(int(code), "unknown")


def _ptr(t):
    return None if t is None else _vp(t.data_ptr())


def _stream(stream):
    if stream is None:  # the current device's current stream
        return _vp(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))
    return _vp(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t, name, dtype, ndim=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")


def _check(rc, where):
    if rc != 0:
        raise CsaError(rc, where)


def csa_compress_cu_seqlens(cu_seqlens, cmp_ratio: int, out=None, stream=None):
    """cu_seqlens_cmp[b+1] = cu_seqlens_cmp[b] + floor(len_b / cmp_ratio)."""
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    if out is None:
        out = torch.empty_like(cu_seqlens)
    _need(out, "out", torch.int32, 1)
    _check(lib().csa_compress_cu_seqlens(_ptr(cu_seqlens), cu_seqlens.numel() - 1, int(cmp_ratio),
                                         _ptr(out), _stream(stream)), "csa_compress_cu_seqlens")
    return out


def csa_window_idx(cu_seqlens, total_tokens: int, ori_win_left: int, ori_win_right: int = 0,
                   out=None, stream=None):
    """[T, ori_win_left+1] int32 window rows (stream-absolute, -1 padded)."""
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    if out is None:
        out = torch.empty((total_tokens, ori_win_left + 1), dtype=torch.int32,
                          device=cu_seqlens.device)
    _need(out, "out", torch.int32, 2)
    _check(lib().csa_window_idx(_ptr(cu_seqlens), cu_seqlens.numel() - 1, int(total_tokens),
                                int(ori_win_left), int(ori_win_right), _ptr(out), _stream(stream)),
           "csa_window_idx")
    return out


def csa_indexer_topk_workspace_size(total_tokens, total_cmp, index_heads, index_dim, topk) -> int:
    return int(lib().csa_indexer_topk_workspace_size(int(total_tokens), int(total_cmp),
                                                     int(index_heads), int(index_dim), int(topk)))


def csa_indexer_topk(q, k, w, cu_seqlens_q, cu_seqlens_cmp_kv, cmp_ratio: int, topk: int,
                     return_value: bool = False, workspace=None, out=None, out_val=None,
                     stream=None):
    """Top-k compressed rows per token by lightning-indexer score.

    Returns ``(topk_idx [T, topk] int32, topk_val [T, topk] fp32 or None)``."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k, "k", torch.bfloat16, 2)
    _need(w, "w", torch.float32, 2)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(cu_seqlens_cmp_kv, "cu_seqlens_cmp_kv", torch.int32, 1)
    T, Hi, Di = q.shape
    Tc = 0 if k is None else k.shape[0]
    if out is None:
        out = torch.empty((T, topk), dtype=torch.int32, device=q.device)
    if return_value and out_val is None:
        out_val = torch.empty((T, topk), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.int32, 2)
    _need(out_val, "out_val", torch.float32, 2)
    need = csa_indexer_topk_workspace_size(T, Tc, Hi, Di, topk)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().csa_indexer_topk(
        _ptr(q), _ptr(k) if Tc else None, _ptr(w), T, Tc, Hi, Di, _ptr(cu_seqlens_q),
        _ptr(cu_seqlens_cmp_kv), cu_seqlens_q.numel() - 1, int(cmp_ratio), int(topk), _ptr(out),
        _ptr(out_val) if return_value else None, _ptr(workspace), ws_bytes, _stream(stream)),
        "csa_indexer_topk")
    return out, (out_val if return_value else None)


def csa_indexer_topk_noalloc(q, k, w, cu_seqlens_q, cu_seqlens_cmp_kv, cmp_ratio: int,
                             topk: int, return_value: bool = False, out=None, out_val=None,
                             stream=None):
    """Same result as :func:`csa_indexer_topk`, for callers that cannot
    allocate device memory: no workspace, the library's own fixed 32 MiB
    scratch array instead (shared by every call; order calls on one stream)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k, "k", torch.bfloat16, 2)
    _need(w, "w", torch.float32, 2)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(cu_seqlens_cmp_kv, "cu_seqlens_cmp_kv", torch.int32, 1)
    T, Hi, Di = q.shape
    Tc = 0 if k is None else k.shape[0]
    if out is None:
        out = torch.empty((T, topk), dtype=torch.int32, device=q.device)
    if return_value and out_val is None:
        out_val = torch.empty((T, topk), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.int32, 2)
    _need(out_val, "out_val", torch.float32, 2)
    _check(lib().csa_indexer_topk_noalloc(
        _ptr(q), _ptr(k) if Tc else None, _ptr(w), T, Tc, Hi, Di, _ptr(cu_seqlens_q),
        _ptr(cu_seqlens_cmp_kv), cu_seqlens_q.numel() - 1, int(cmp_ratio), int(topk), _ptr(out),
        _ptr(out_val) if return_value else None, _stream(stream)), "csa_indexer_topk_noalloc")
    return out, (out_val if return_value else None)


def csa_sparse_mla_fwd(q, ori_kv, cmp_kv, cmp_sparse_indices, cu_seqlens_q, cu_seqlens_ori_kv,
                       cu_seqlens_cmp_kv, sinks, softmax_scale: float, cmp_ratio: int,
                       ori_win_left: int, ori_win_right: int = 0,
                       return_softmax_lse: bool = False, out=None, lse=None, stream=None):
    """Shared-KV MLA sparse attention with sinks.

    ``cmp_sparse_indices`` None attends every visible compressed row (HCA);
    ``cmp_kv`` None attends the window only. Returns ``(out, lse or None)``."""
    _need(q, "q", torch.bfloat16, 3)
    _need(ori_kv, "ori_kv", torch.bfloat16, 2)
    _need(cmp_kv, "cmp_kv", torch.bfloat16, 2)
    _need(cmp_sparse_indices, "cmp_sparse_indices", torch.int32, 2)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(cu_seqlens_ori_kv, "cu_seqlens_ori_kv", torch.int32, 1)
    _need(cu_seqlens_cmp_kv, "cu_seqlens_cmp_kv", torch.int32, 1)
    _need(sinks, "sinks", torch.float32, 1)
    T, H, D = q.shape
    Tc = 0 if cmp_kv is None else cmp_kv.shape[0]
    topk = 0 if cmp_sparse_indices is None else cmp_sparse_indices.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if return_softmax_lse and lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.bfloat16, 3)
    _need(lse, "lse", torch.float32, 2)
    _check(lib().csa_sparse_mla_fwd(
        _ptr(q), _ptr(ori_kv), _ptr(cmp_kv) if Tc else None, _ptr(cmp_sparse_indices),
        _ptr(cu_seqlens_q), _ptr(cu_seqlens_ori_kv), _ptr(cu_seqlens_cmp_kv),
        cu_seqlens_q.numel() - 1, T, Tc, H, D, topk, _ptr(sinks), float(softmax_scale),
        int(cmp_ratio), int(ori_win_left), int(ori_win_right), _ptr(out),
        _ptr(lse) if return_softmax_lse else None, 1 if return_softmax_lse else 0,
        _stream(stream)), "csa_sparse_mla_fwd")
    return out, (lse if return_softmax_lse else None)


def csa_sparse_mla_bwd(q, dout, out, lse, ori_kv, cmp_kv, cmp_sparse_indices, cu_seqlens_q,
                       cu_seqlens_ori_kv, cu_seqlens_cmp_kv, sinks, softmax_scale: float,
                       cmp_ratio: int, ori_win_left: int, ori_win_right: int = 0,
                       want_l1: bool = True, stream=None):
    """Backward of ``csa_sparse_mla_fwd`` from its ``out`` and ``lse``.

    Returns a dict of fp32 tensors: d_q [T,H,D], d_ori_kv [T,D], d_cmp_kv
    [Tc,D] (None without compressed rows), d_sinks [H] (None without sinks),
    ori_l1 [T, ori_win_left+1] and cmp_l1 [T, topk] (None without a top-k
    list, or both None when ``want_l1`` is false)."""
    for t, n, dt, nd in ((q, "q", torch.bfloat16, 3), (dout, "dout", torch.bfloat16, 3),
                         (out, "out", torch.bfloat16, 3), (lse, "lse", torch.float32, 2),
                         (ori_kv, "ori_kv", torch.bfloat16, 2), (cmp_kv, "cmp_kv", torch.bfloat16, 2),
                         (cmp_sparse_indices, "cmp_sparse_indices", torch.int32, 2),
                         (cu_seqlens_q, "cu_seqlens_q", torch.int32, 1),
                         (cu_seqlens_ori_kv, "cu_seqlens_ori_kv", torch.int32, 1),
                         (cu_seqlens_cmp_kv, "cu_seqlens_cmp_kv", torch.int32, 1),
                         (sinks, "sinks", torch.float32, 1)):
        _need(t, n, dt, nd)
    T, H, D = q.shape
    Tc = 0 if cmp_kv is None else cmp_kv.shape[0]
    topk = 0 if cmp_sparse_indices is None else cmp_sparse_indices.shape[1]
    f32 = dict(dtype=torch.float32, device=q.device)
    res = {
        "d_q": torch.empty((T, H, D), **f32),
        "d_ori_kv": torch.empty((T, D), **f32),
        "d_cmp_kv": torch.empty((Tc, D), **f32) if Tc else None,
        "d_sinks": torch.empty((H,), **f32) if sinks is not None else None,
        "ori_l1": torch.empty((T, ori_win_left + 1), **f32) if want_l1 else None,
        "cmp_l1": (torch.empty((T, topk), **f32)
                   if want_l1 and Tc and cmp_sparse_indices is not None else None),
    }
    _check(lib().csa_sparse_mla_bwd(
        _ptr(q), _ptr(dout), _ptr(out), _ptr(lse), _ptr(ori_kv), _ptr(cmp_kv) if Tc else None,
        _ptr(cmp_sparse_indices), _ptr(cu_seqlens_q), _ptr(cu_seqlens_ori_kv),
        _ptr(cu_seqlens_cmp_kv), cu_seqlens_q.numel() - 1, T, Tc, H, D, topk, _ptr(sinks),
        float(softmax_scale), int(cmp_ratio), int(ori_win_left), int(ori_win_right),
        _ptr(res["d_q"]), _ptr(res["d_ori_kv"]), _ptr(res["d_cmp_kv"]), _ptr(res["d_sinks"]),
        _ptr(res["ori_l1"]), _ptr(res["cmp_l1"]), _stream(stream)), "csa_sparse_mla_bwd")
    return res


def csa_indexer_kl_loss_grad(q, k, w, sparse_indices, attn_softmax_l1_norm, cu_seqlens_q,
                             cu_seqlens_cmp_kv, cmp_ratio: int, grad_scale: float = 1.0,
                             want_loss: bool = True, stream=None):
    """Indexer KL loss against the attention distribution, and its gradients.

    Returns a dict of fp32 tensors: d_q [T,Hi,Di], d_k [Tc,Di] (None when
    Tc == 0), d_w [T,Hi] and loss [T] (the unscaled KL per token; None unless
    ``want_loss``). The gradients are those of ``grad_scale * loss.sum()``."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k, "k", torch.bfloat16, 2)
    _need(w, "w", torch.float32, 2)
    _need(sparse_indices, "sparse_indices", torch.int32, 2)
    _need(attn_softmax_l1_norm, "attn_softmax_l1_norm", torch.float32, 2)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(cu_seqlens_cmp_kv, "cu_seqlens_cmp_kv", torch.int32, 1)
    T, Hi, Di = q.shape
    Tc = 0 if k is None else k.shape[0]
    topk = sparse_indices.shape[1]
    if tuple(attn_softmax_l1_norm.shape) != (T, topk) or sparse_indices.shape[0] != T:
        raise ValueError("sparse_indices and attn_softmax_l1_norm must both be [T, topk]")
    f32 = dict(dtype=torch.float32, device=q.device)
    res = {"d_q": torch.empty((T, Hi, Di), **f32),
           "d_k": torch.empty((Tc, Di), **f32) if Tc else None,
           "d_w": torch.empty((T, Hi), **f32),
           "loss": torch.empty((T,), **f32) if want_loss else None}
    _check(lib().csa_indexer_kl_loss_grad(
        _ptr(q), _ptr(k) if Tc else None, _ptr(w), _ptr(sparse_indices),
        _ptr(attn_softmax_l1_norm), T, Tc, Hi, Di, _ptr(cu_seqlens_q), _ptr(cu_seqlens_cmp_kv),
        cu_seqlens_q.numel() - 1, int(cmp_ratio), int(topk), float(grad_scale), _ptr(res["d_q"]),
        _ptr(res["d_k"]), _ptr(res["d_w"]), _ptr(res["loss"]), _stream(stream)),
        "csa_indexer_kl_loss_grad")
    return res


def _workspace(need, device, workspace):
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return workspace, size


def csa_sparse_mla_fwd_bsnd(q, ori_kv, cmp_kv, cmp_sparse_indices, seqused, sinks,
                            softmax_scale: float, cmp_ratio: int, ori_win_left: int,
                            ori_win_right: int = 0, return_softmax_lse: bool = False,
                            workspace=None, out=None, lse=None, stream=None):
    """Sparse MLA forward in BSND layout: q [B,S,H,D], ori_kv [B,S,D], cmp_kv
    [B,Sc,D] or None, cmp_sparse_indices [B,S,topk] batch-local or None,
    seqused [B] int32 or None. Returns ``(out [B,S,H,D], lse [B,S,H] or None)``;
    rows past seqused are unspecified."""
    _need(q, "q", torch.bfloat16, 4)
    _need(ori_kv, "ori_kv", torch.bfloat16, 3)
    _need(cmp_kv, "cmp_kv", torch.bfloat16, 3)
    _need(cmp_sparse_indices, "cmp_sparse_indices", torch.int32, 3)
    _need(seqused, "seqused", torch.int32, 1)
    _need(sinks, "sinks", torch.float32, 1)
    B, S, H, D = q.shape
    Sc = 0 if cmp_kv is None else cmp_kv.shape[1]
    topk = 0 if cmp_sparse_indices is None else cmp_sparse_indices.shape[2]
    if out is None:
        out = torch.empty_like(q)
    if return_softmax_lse and lse is None:
        lse = torch.empty((B, S, H), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.bfloat16, 4)
    _need(lse, "lse", torch.float32, 3)
    list_used = topk if Sc else 0
    need = int(lib().csa_bsnd_mla_workspace_size(B, S, list_used))
    workspace, ws_bytes = _workspace(need, q.device, workspace)
    _check(lib().csa_sparse_mla_fwd_bsnd(
        _ptr(q), _ptr(ori_kv), _ptr(cmp_kv) if Sc else None, _ptr(cmp_sparse_indices),
        _ptr(seqused), B, S, Sc, H, D, topk, _ptr(sinks), float(softmax_scale), int(cmp_ratio),
        int(ori_win_left), int(ori_win_right), _ptr(out),
        _ptr(lse) if return_softmax_lse else None, 1 if return_softmax_lse else 0,
        _ptr(workspace), ws_bytes, _stream(stream)), "csa_sparse_mla_fwd_bsnd")
    return out, (lse if return_softmax_lse else None)


def csa_indexer_topk_bsnd(q, k, w, seqused, cmp_ratio: int, topk: int,
                          return_value: bool = False, workspace=None, out=None, out_val=None,
                          stream=None):
    """Lightning-indexer top-k in BSND layout: q [B,S,Hi,Di], k [B,Sc,Di],
    w [B,S,Hi], seqused [B] int32 or None. Returns ``(topk_idx [B,S,topk]
    batch-local rows, topk_val or None)``; rows past seqused are unspecified."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k, "k", torch.bfloat16, 3)
    _need(w, "w", torch.float32, 3)
    _need(seqused, "seqused", torch.int32, 1)
    B, S, Hi, Di = q.shape
    Sc = 0 if k is None else k.shape[1]
    if out is None:
        out = torch.empty((B, S, topk), dtype=torch.int32, device=q.device)
    if return_value and out_val is None:
        out_val = torch.empty((B, S, topk), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.int32, 3)
    _need(out_val, "out_val", torch.float32, 3)
    need = int(lib().csa_bsnd_indexer_workspace_size(B, S, Sc, Hi, Di, int(topk)))
    workspace, ws_bytes = _workspace(need, q.device, workspace)
    _check(lib().csa_indexer_topk_bsnd(
        _ptr(q), _ptr(k) if Sc else None, _ptr(w), _ptr(seqused), B, S, Sc, Hi, Di,
        int(cmp_ratio), int(topk), _ptr(out), _ptr(out_val) if return_value else None,
        _ptr(workspace), ws_bytes, _stream(stream)), "csa_indexer_topk_bsnd")
    return out, (out_val if return_value else None)


def csa_compress_thd(kv, score, ape, cu_seqlens, cu_seqlens_cmp, total_cmp: int,
                     cmp_ratio: int, head_dim: int, overlap: bool = True, out=None, stream=None):
    """Compressed rows [total_cmp, head_dim] fp32 from the projections kv and
    score [T, Wd] fp32 (Wd = 2 head_dim with overlap) and ape [cmp_ratio, Wd]
    or None: per-sequence groups, overlap transform, softmax pooling over
    the slots. ``total_cmp`` is cu_seqlens_cmp's last entry (a host int)."""
    _need(kv, "kv", torch.float32, 2)
    _need(score, "score", torch.float32, 2)
    _need(ape, "ape", torch.float32, 2)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    _need(cu_seqlens_cmp, "cu_seqlens_cmp", torch.int32, 1)
    T, wd = kv.shape
    if tuple(score.shape) != (T, wd) or wd != (2 * head_dim if overlap else head_dim):
        raise ValueError("kv and score must both be [T, 2*head_dim] (overlap) or [T, head_dim]")
    if out is None:
        out = torch.empty((total_cmp, head_dim), dtype=torch.float32, device=kv.device)
    _need(out, "out", torch.float32, 2)
    _check(lib().csa_compress_thd(
        _ptr(kv), _ptr(score), _ptr(ape), _ptr(cu_seqlens), _ptr(cu_seqlens_cmp),
        cu_seqlens.numel() - 1, T, int(total_cmp), int(cmp_ratio), int(head_dim),
        1 if overlap else 0, _ptr(out), _stream(stream)), "csa_compress_thd")
    return out


_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_LAYOUTS = {"interleaved": 0, "half": 1}


def _dims(t, name, ndim):
    """The shape of a tensor argument with `ndim` axes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if len(shape) != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(shape)}")
    return shape


def _rows(t, name, ndim):
    """A bf16 or fp32 CUDA tensor whose rows (everything past the first axis)
    are contiguous; the stride between them is free. Returns the dtype code."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    if t.dim() not in ndim:
        raise ValueError(f"{name} must have {' or '.join(map(str, ndim))} dims, got {tuple(t.shape)}")
    if not t.is_contiguous() and t.numel() and not t[0].is_contiguous():
        raise ValueError(f"{name} must have contiguous rows")
    return code


def _match(dev, *specs):
    """Each (tensor or None, name, dtype, shape): on device `dev` (a CUDA one),
    contiguous, of that dtype and shape."""
    for t, name, dtype, shape in specs:
        if t is None:
            continue
        try:
            if (t.dtype is dtype and t.shape == shape and t.get_device() == dev >= 0
                    and t.is_contiguous()):
                continue
        except AttributeError:
            pass
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the call on cuda:{dev}")


def _new(shape, dtype, dev, stream):
    """A new tensor on device `dev` from the memory of the call's stream (None:
    that device's current one). Another stream's block may still be in use by
    work queued there, which the call's stream does not wait for."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _scratch(workspace, dev, stream, size, *args):
    """A call's workspace and its bytes: the caller's (its size is checked by
    the call), or a new one of `size(*args)` bytes."""
    if workspace is None:
        need = size(*args)
        if need == 0:
            return None, 0
        workspace = _new((need,), torch.uint8, dev, stream)
    elif not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev:
        raise ValueError(f"workspace must be a tensor on cuda:{dev}")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def _written(*tensors):
    """Tells autograd that the call wrote these tensors of the caller's (None:
    not given), as PyTorch's own in-place calls do: a graph that saved one of
    them then refuses its backward instead of using the new values."""
    torch._C._increment_version([t for t in tensors if t is not None])


def _addr(t):
    return None if t is None else t.data_ptr()


def _layout(layout):
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
    return _LAYOUTS[layout]


def _launch(dev, where, stream, *args):
    """Calls entry point `where` with device `dev` current, on `stream` (None:
    that device's current stream)."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    fn = getattr(_lib or lib(), where)
    if torch._C._cuda_getDevice() == dev:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc != 0:
        raise CsaError(rc, where)


def csa_rope_freqs(rope_dim: int, theta: float = 10000.0, factor: float = 1.0,
                   original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                   out=None, device=None, stream=None):
    """Rotation frequencies [rope_dim / 2] fp64 in radians per position, for
    :func:`csa_rope` and :func:`csa_cache_append`. ``factor`` > 1 stretches
    positions for longer contexts: all pairs (``original_len`` 0) or the slow
    ones, by parts."""
    rope_dim = int(rope_dim)
    half, given = max(rope_dim, 0) // 2, out
    if out is None:
        device = torch.device("cuda" if device is None else device)
        if device.type != "cuda":
            raise TypeError(f"device must be a CUDA device, got {device}")
        dev = torch.cuda.current_device() if device.index is None else device.index
        out = _new((half,), torch.float64, dev, stream)
    else:
        _dims(out, "out", 1)
        dev = out.get_device()
        _match(dev, (out, "out", torch.float64, (half,)))
    _launch(dev, "csa_rope_freqs", stream, rope_dim, theta, factor, int(original_len), beta_fast,
            beta_slow, out.data_ptr())
    _written(given)
    return out


def csa_rope(x, positions, inv_freq, rope_offset=None, layout: str = "interleaved",
             mscale: float = 1.0, inverse: bool = False, cu_seqlens=None, pos_stride: int = 1,
             out=None, stream=None):
    """Rotary positions over ``2 * inv_freq.numel()`` dims of every head of x
    [T, H, D] or [T, D] (bf16 or fp32, contiguous rows), starting at
    ``rope_offset`` (None: the head's last dims); other dims are copied.

    ``positions`` [T] int32, or None with ``cu_seqlens`` [batch+1]: the place
    in the packed sequence; both times ``pos_stride``. ``inverse`` turns back,
    which is also the backward. ``out`` may be ``x``. Returns out.

    As with every call here, nothing is recorded for autograd: the result of an
    ``x`` that requires a gradient does not require one, and the caller turns
    the gradient back with ``inverse``. Tensors of the caller's that are written
    (``out``, the caches) count as changed in place, though."""
    code = _rows(x, "x", (2, 3))
    dev, shape = x.get_device(), x.shape
    T, D = shape[0], shape[-1]
    H = shape[1] if len(shape) == 3 else 1
    if out is not None and out is not x:
        if _rows(out, "out", (2, 3)) != code:
            raise TypeError(f"out must be {x.dtype}, got {out.dtype}")
        if out.shape != shape or out.get_device() != dev:
            raise ValueError(f"out must be {list(shape)} on {x.device}, got {list(out.shape)} on "
                             f"{out.device}")
    half = 0 if inv_freq is None else _dims(inv_freq, "inv_freq", 1)[0]
    batch = 0 if cu_seqlens is None else _dims(cu_seqlens, "cu_seqlens", 1)[0] - 1
    _match(dev, (positions, "positions", torch.int32, (T,)),
           (inv_freq, "inv_freq", torch.float64, (half,)),
           (cu_seqlens, "cu_seqlens", torch.int32, (batch + 1,)))
    code_layout, given = _layout(layout), out
    if out is None:
        out = _new(shape, x.dtype, dev, stream)
    _launch(dev, "csa_rope", stream, x.data_ptr(), code, x.stride(0), _addr(positions),
            _addr(cu_seqlens), batch, pos_stride, _addr(inv_freq), T, H, D,
            D - 2 * half if rope_offset is None else rope_offset, 2 * half, code_layout, mscale,
            1 if inverse else 0, out.data_ptr(), out.stride(0))
    _written(given)
    return out


def csa_cache_append(rows, row_seq, row_pos, pages, cache, inv_freq=None, rope_offset=None,
                     layout: str = "interleaved", mscale: float = 1.0, pos_stride: int = 1,
                     stream=None):
    """Writes rows [T, width] (bf16 or fp32, contiguous rows) to the slots of
    positions ``row_pos`` [T] of sequences ``row_seq`` [T] (None: row t is
    sequence t's) in the paged ``cache`` [num_pages, page_size, width] bf16
    with table ``pages`` [batch, max_pages], rotated as :func:`csa_rope` does
    at ``row_pos * pos_stride`` when ``inv_freq`` is given. A negative
    position skips the row. Returns cache."""
    code = _rows(rows, "rows", (2,))
    dev = rows.get_device()
    T, width = rows.shape
    n_pages, page, _ = _dims(cache, "cache", 3)
    batch, max_pages = _dims(pages, "pages", 2)
    half = 0 if inv_freq is None else _dims(inv_freq, "inv_freq", 1)[0]
    _match(dev, (row_seq, "row_seq", torch.int32, (T,)), (row_pos, "row_pos", torch.int32, (T,)),
           (pages, "pages", torch.int32, (batch, max_pages)),
           (cache, "cache", torch.bfloat16, (n_pages, page, width)),
           (inv_freq, "inv_freq", torch.float64, (half,)))
    _launch(dev, "csa_cache_append", stream, rows.data_ptr(), code, rows.stride(0), _addr(row_seq),
            _addr(row_pos), pages.data_ptr(), batch, max_pages, n_pages, page, T, width,
            _addr(inv_freq), width - 2 * half if rope_offset is None else rope_offset, 2 * half,
            _layout(layout), mscale, pos_stride, cache.data_ptr())
    _written(cache)
    return cache


def csa_indexer_topk_paged_workspace_size(total_tokens, max_rows, index_heads, index_dim,
                                          topk) -> int:
    return lib().csa_indexer_topk_paged_workspace_size(int(total_tokens), int(max_rows),
                                                       int(index_heads), int(index_dim), int(topk))


def csa_indexer_topk_paged(q, k_cache, w, pages, q_seq, q_pos, cmp_ratio: int, topk: int,
                           return_value: bool = False, workspace=None, out=None, out_val=None,
                           stream=None):
    """Lightning-indexer top-k of new tokens q [T, Hi, Di], w [T, Hi] at
    positions ``q_pos`` [T] (negative: padding) of sequences ``q_seq`` [T]
    (None: token t is sequence t's) over the paged rows ``k_cache``
    [num_pages, page_size, Di] with table ``pages`` [batch, max_pages].

    Returns ``(topk_idx [T, topk] int32 rows of the sequence, -1 padded,
    topk_val [T, topk] fp32 or None)``."""
    T, Hi, Di = _dims(q, "q", 3)
    n_pages, page, _ = _dims(k_cache, "k_cache", 3)
    batch, max_pages = _dims(pages, "pages", 2)
    dev = q.get_device()
    topk = int(topk)
    shape = (T, max(topk, 0))
    if not return_value:
        out_val = None
    _match(dev, (q, "q", torch.bfloat16, (T, Hi, Di)),
           (k_cache, "k_cache", torch.bfloat16, (n_pages, page, Di)),
           (w, "w", torch.float32, (T, Hi)), (pages, "pages", torch.int32, (batch, max_pages)),
           (q_seq, "q_seq", torch.int32, (T,)), (q_pos, "q_pos", torch.int32, (T,)),
           (out, "out", torch.int32, shape), (out_val, "out_val", torch.float32, shape))
    given = out, out_val
    if out is None:
        out = _new(shape, torch.int32, dev, stream)
    if return_value and out_val is None:
        out_val = _new(shape, torch.float32, dev, stream)
    workspace, ws_bytes = _scratch(workspace, dev, stream,
                                   csa_indexer_topk_paged_workspace_size, T,
                                   min(max_pages * page, 2 ** 31 - 1), Hi, Di, topk)
    _launch(dev, "csa_indexer_topk_paged", stream, q.data_ptr(), k_cache.data_ptr(), _addr(w),
            pages.data_ptr(), _addr(q_seq), _addr(q_pos), batch, T, Hi, Di, n_pages, page, max_pages,
            cmp_ratio, topk, out.data_ptr(), _addr(out_val), _addr(workspace), ws_bytes)
    _written(*given)
    return out, out_val


def csa_sparse_mla_paged_workspace_size(total_tokens, heads) -> int:
    return lib().csa_sparse_mla_paged_workspace_size(int(total_tokens), int(heads))


def csa_sparse_mla_paged(q, ori_cache, cmp_cache, cmp_sparse_indices, ori_pages, cmp_pages, q_seq,
                         q_pos, sinks, softmax_scale: float, cmp_ratio: int, ori_win_left: int,
                         ori_win_right: int = 0, return_softmax_lse: bool = False,
                         workspace=None, out=None, lse=None, stream=None):
    """Sparse MLA attention of new tokens q [T, H, 512] at positions ``q_pos``
    [T] (negative: padding) of sequences ``q_seq`` [T] (None: token t is
    sequence t's) over the window rows of ``ori_cache`` [pages, page_size,
    512] and the rows of ``cmp_cache`` listed in ``cmp_sparse_indices`` [T,
    topk] (rows of the sequence; None: every visible row), each with its page
    table [batch, max_pages]. ``cmp_cache`` None: window only.

    Returns ``(out [T, H, 512], lse [T, H] or None)``."""
    T, H, D = _dims(q, "q", 3)
    ori_n, ori_page, _ = _dims(ori_cache, "ori_cache", 3)
    batch, ori_max = _dims(ori_pages, "ori_pages", 2)
    dev = q.get_device()
    cmp_n = cmp_page = cmp_max = topk = 0
    if cmp_cache is None:
        cmp_sparse_indices = cmp_pages = None
    else:
        cmp_n, cmp_page, _ = _dims(cmp_cache, "cmp_cache", 3)
        cmp_max = _dims(cmp_pages, "cmp_pages", 2)[1]
        if cmp_sparse_indices is not None:
            topk = _dims(cmp_sparse_indices, "cmp_sparse_indices", 2)[1]
    if not return_softmax_lse:
        lse = None
    _match(dev, (q, "q", torch.bfloat16, (T, H, D)),
           (ori_cache, "ori_cache", torch.bfloat16, (ori_n, ori_page, D)),
           (cmp_cache, "cmp_cache", torch.bfloat16, (cmp_n, cmp_page, D)),
           (cmp_sparse_indices, "cmp_sparse_indices", torch.int32, (T, topk)),
           (ori_pages, "ori_pages", torch.int32, (batch, ori_max)),
           (cmp_pages, "cmp_pages", torch.int32, (batch, cmp_max)),
           (q_seq, "q_seq", torch.int32, (T,)), (q_pos, "q_pos", torch.int32, (T,)),
           (sinks, "sinks", torch.float32, (H,)), (out, "out", torch.bfloat16, (T, H, D)),
           (lse, "lse", torch.float32, (T, H)))
    given = out, lse
    if out is None:
        out = _new((T, H, D), torch.bfloat16, dev, stream)
    if return_softmax_lse and lse is None:
        lse = _new((T, H), torch.float32, dev, stream)
    workspace, ws_bytes = _scratch(workspace, dev, stream,
                                   csa_sparse_mla_paged_workspace_size, T, H)
    _launch(dev, "csa_sparse_mla_paged", stream, q.data_ptr(), ori_cache.data_ptr(),
            _addr(cmp_cache), _addr(cmp_sparse_indices), ori_pages.data_ptr(), _addr(cmp_pages),
            _addr(q_seq), _addr(q_pos), batch, T, H, D, ori_n, ori_page, ori_max, cmp_n, cmp_page,
            cmp_max, topk, _addr(sinks), softmax_scale, cmp_ratio, ori_win_left, ori_win_right,
            out.data_ptr(), _addr(lse), 1 if return_softmax_lse else 0, _addr(workspace), ws_bytes)
    _written(*given)
    return out, lse


def csa_device_error(stream=None):
    """Synchronise the stream; return (status, raw word) of the device error word."""
    detail = _i32(0)
    rc = lib().csa_device_error(_stream(stream), C.byref(detail))
    return int(rc), int(detail.value)


def csa_set_wait_limit_ns(limit_ns: int) -> None:
    """Limit of the indexer and sparse-attention kernels' pipeline waits, in
    ns (0: the default 2 s). A wait that gives up records CSA_ERR_TIMEOUT in
    the device error word; for testing the timeout path."""
    _check(lib().csa_set_wait_limit_ns(int(limit_ns)), "csa_set_wait_limit_ns")


def csa_set_pair_select_rows(rows: int) -> None:
    """Rows above which the indexer selects a token's top-k with one warp
    instead of two (0: the default bound); for testing the one-warp path."""
    _check(lib().csa_set_pair_select_rows(int(rows)), "csa_set_pair_select_rows")
