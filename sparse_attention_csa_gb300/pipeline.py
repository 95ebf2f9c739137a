"""One CSA / HCA attention layer: its forward over packed sequences, chaining
the four C-ABI calls, and its step for new tokens over paged caches.

Order of the path (miles PR 2038 report, the attention forward excerpt:
compressed cu_seqlens, then the indexer, then sparse attention over the window
rows plus the selected compressed rows):

1. ``csa_compress_cu_seqlens``  compressed cu_seqlens of the pack;
2. ``csa_window_idx``           the window rows (returned for the caller; the
                                attention kernel derives the band itself);
3. ``csa_indexer_topk``         top-k compressed rows (INDEXER layers only);
4. ``csa_sparse_mla_fwd``       attention with sinks (COMPRESSOR_ONLY layers
                                attend every visible compressed row).

Everything runs on the current CUDA stream (the window rows optionally on a
side stream, joined before returning); nothing synchronises.

``csa_layer_decode`` continues sequences whose rows are cached: the new rows go
to their slots (rotated on the way), the indexer chooses compressed rows, the
attention reads the paged caches (compressed rows in bf16 or held in 4 bits), and
the weight that the compressed rows received is added up where the cache keeps
it. ``csa_layer_evict`` gives pages back by that weight.
"""

from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (csa_attn_mass_paged, csa_cache_append, csa_cache_evict, csa_compress_cu_seqlens,
               csa_indexer_topk, csa_indexer_topk_paged, csa_indexer_topk_workspace_size, csa_rope,
               csa_sparse_mla_fwd, csa_sparse_mla_paged, csa_sparse_mla_paged_q4, csa_window_idx)


@dataclass
class LayerOutputs:
    out: torch.Tensor                 # [T, H, 512] bf16
    lse: torch.Tensor | None          # [T, H] fp32
    topk_idx: torch.Tensor | None     # [T, topk] int32 (INDEXER layers)
    window_idx: torch.Tensor | None   # [T, W] int32
    cu_seqlens_cmp: torch.Tensor      # [batch+1] int32


def allocate_outputs(T, H, D, W, topk, batch, device, with_window=True, with_lse=True):
    """Preallocated outputs for repeated calls (benchmarks, CUDA graphs)."""
    return LayerOutputs(
        out=torch.empty((T, H, D), dtype=torch.bfloat16, device=device),
        lse=torch.empty((T, H), dtype=torch.float32, device=device) if with_lse else None,
        topk_idx=torch.empty((T, topk), dtype=torch.int32, device=device) if topk else None,
        window_idx=torch.empty((T, W), dtype=torch.int32, device=device) if with_window else None,
        cu_seqlens_cmp=torch.empty((batch + 1,), dtype=torch.int32, device=device),
    )


def csa_layer_forward(q, ori_kv, cmp_kv, cu_seqlens, sinks, softmax_scale: float, cmp_ratio: int,
                      ori_win_left: int, q_idx=None, k_idx=None, w=None, topk: int = 0,
                      return_softmax_lse: bool = True, with_window: bool = True,
                      outputs: LayerOutputs | None = None, workspace=None,
                      window_stream=None) -> LayerOutputs:
    """Forward of one layer. ``q_idx``/``k_idx``/``w``/``topk`` given -> INDEXER
    layer (CSA); omitted -> COMPRESSOR_ONLY layer (HCA, every visible block).
    ``cmp_kv`` must hold exactly the pack's compressed row count.
    ``window_stream`` (a CUDA stream): the window rows, which nothing else of
    the layer reads, are computed there, beside the indexer, and the current
    stream waits for them before returning."""
    T, H, D = q.shape
    batch = cu_seqlens.numel() - 1
    indexer = q_idx is not None
    if outputs is None:
        outputs = allocate_outputs(T, H, D, ori_win_left + 1, topk if indexer else 0, batch,
                                   q.device, with_window, return_softmax_lse)
    csa_compress_cu_seqlens(cu_seqlens, cmp_ratio, out=outputs.cu_seqlens_cmp)
    main = torch.cuda.current_stream()
    win_done = None
    if with_window:
        if window_stream is None:
            csa_window_idx(cu_seqlens, T, ori_win_left, 0, out=outputs.window_idx)
        else:
            window_stream.wait_stream(main)
            csa_window_idx(cu_seqlens, T, ori_win_left, 0, out=outputs.window_idx,
                           stream=window_stream)
            win_done = torch.cuda.Event()
            win_done.record(window_stream)
    idx = None
    if indexer:
        if workspace is None:
            need = csa_indexer_topk_workspace_size(T, k_idx.shape[0], q_idx.shape[1],
                                                   q_idx.shape[2], topk)
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
        idx, _ = csa_indexer_topk(q_idx, k_idx, w, cu_seqlens, outputs.cu_seqlens_cmp, cmp_ratio,
                                  topk, workspace=workspace, out=outputs.topk_idx)
    csa_sparse_mla_fwd(q, ori_kv, cmp_kv, idx, cu_seqlens, cu_seqlens, outputs.cu_seqlens_cmp,
                       sinks, softmax_scale, cmp_ratio, ori_win_left, 0, return_softmax_lse,
                       out=outputs.out, lse=outputs.lse)
    if win_done is not None:
        main.wait_event(win_done)
    return outputs


@dataclass
class PagedLayerCache:
    """One layer's paged caches. Original and compressed rows have tables of
    their own; the indexer's rows share the compressed rows' table."""
    ori: torch.Tensor                    # [pages, page_size, 512] bf16
    ori_pages: torch.Tensor              # [batch, max_pages] int32
    cmp: torch.Tensor | None = None      # [pages, page_size, 512] bf16, or [.., 384] uint8 (4 bits)
    cmp_pages: torch.Tensor | None = None
    k_idx: torch.Tensor | None = None    # [pages, page_size, Di] bf16 (INDEXER layers)
    # attention weight that the compressed rows received so far, where it is
    # wanted: [batch, max_pages * page_size] fp32, zero for a new sequence
    mass: torch.Tensor | None = None


@dataclass
class DecodeOutputs:
    out: torch.Tensor                 # [T, H, 512] bf16
    lse: torch.Tensor | None          # [T, H] fp32
    topk_idx: torch.Tensor | None     # [T, topk] int32 rows of the sequence (INDEXER layers)


def csa_layer_decode(q, kv, cache: PagedLayerCache, q_seq, q_pos, sinks, softmax_scale: float,
                     cmp_ratio: int, ori_win_left: int, inv_freq=None, rope_layout="interleaved",
                     turn_back: bool = False, q_idx=None, w=None, topk: int = 0,
                     return_softmax_lse: bool = False, indexer_workspace=None,
                     attention_workspace=None, mass_workspace=None) -> DecodeOutputs:
    """New tokens of one layer: q [T, H, 512] and their rows kv [T, 512] at
    positions ``q_pos`` [T] (negative: padding) of sequences ``q_seq`` [T]
    (None: token t is sequence t's).

    ``kv`` is appended to ``cache.ori`` (None: the rows are there already).
    With ``inv_freq`` the last ``2 * inv_freq.numel()`` dims of q and kv are
    rotated at their positions first (q into a new tensor), and with
    ``turn_back`` those of the output are turned back at the token's own
    position. ``q_idx``/``w``/``topk`` given -> INDEXER layer; omitted ->
    every visible compressed row, or none without ``cache.cmp``.

    Left to the caller: compressed rows that these tokens complete, appended
    before the call (``csa_cache_append`` with the group's number as position
    and ``pos_stride=cmp_ratio``), and with them the raw projections of the
    unfinished group, and of the one before it for overlapping layers, that
    ``csa_compress_thd`` makes a row from (``csa_cache_append_q4`` where
    ``cache.cmp`` holds rows in 4 bits); the rotation of the indexer's
    queries and rows (``q_idx`` comes as the indexer takes it); an ``mscale``
    other than 1 (rotate by ``csa_rope`` and ``csa_cache_append``, and leave
    ``inv_freq`` and ``kv`` out)."""
    if kv is not None:
        csa_cache_append(kv, q_seq, q_pos, cache.ori_pages, cache.ori, inv_freq=inv_freq,
                         layout=rope_layout)
    if inv_freq is not None:
        q = csa_rope(q, q_pos, inv_freq, layout=rope_layout)
    idx = None
    if q_idx is not None:
        idx, _ = csa_indexer_topk_paged(q_idx, cache.k_idx, w, cache.cmp_pages, q_seq, q_pos,
                                        cmp_ratio, topk, workspace=indexer_workspace)
    weigh = cache.mass is not None and cache.cmp is not None
    attend = (csa_sparse_mla_paged_q4 if cache.cmp is not None and cache.cmp.dtype is torch.uint8
              else csa_sparse_mla_paged)
    out, lse = attend(q, cache.ori, cache.cmp, idx, cache.ori_pages, cache.cmp_pages, q_seq, q_pos,
                      sinks, softmax_scale, cmp_ratio, ori_win_left,
                      return_softmax_lse=return_softmax_lse or weigh,
                      workspace=attention_workspace)
    if weigh:
        csa_attn_mass_paged(q, lse, cache.cmp, idx, cache.cmp_pages, q_seq, q_pos, cache.mass,
                            softmax_scale, cmp_ratio, out=cache.mass, workspace=mass_workspace)
    if inv_freq is not None and turn_back:
        csa_rope(out, q_pos, inv_freq, layout=rope_layout, inverse=True, out=out)
    return DecodeOutputs(out, lse if return_softmax_lse else None, idx)


def csa_layer_evict(cache: PagedLayerCache, rows, keep_pages: int, keep_first: int = 0,
                    keep_last: int = 0):
    """Gives back pages of compressed rows (and with them the indexer's) of every
    sequence that holds more than ``keep_pages``: those whose rows received the
    least attention weight by ``cache.mass``; ``rows`` [batch] int32 compressed
    rows are in use (negative: leave the sequence alone). ``cache.cmp_pages`` is
    changed in place. Returns ``(freed [batch, max_pages] pool pages, -1 padded,
    n_freed [batch])``."""
    _, freed, n_freed = csa_cache_evict(cache.mass, cache.cmp_pages, rows, keep_pages,
                                        keep_first=keep_first, keep_last=keep_last,
                                        out=cache.cmp_pages)
    return freed, n_freed
