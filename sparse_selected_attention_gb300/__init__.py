"""GB300-native QSA (sparse selected attention) hot path.

Python binding of the C ABI in include/qsa.h: each function marshals torch
CUDA tensors into the argument struct and calls the library on the current
CUDA stream.  All computation runs in libqsa.so's kernels; tensors on the CPU
are rejected rather than computed elsewhere.

    qsa_prep   query RMS-norm + RoPE, K/V int8 quantisation into the cache
    qsa_score  head-reduced fp32 scores of every causal cache cell
    qsa_select per-token selected cell ids from the scores
    qsa_attn   chunked attention over per-token selected cell ids
    qsa_fill_ids_decode / qsa_fill_ids_even  the workloads' id lists, on the device

A paged cache shared by many sequences (kq, vq [layers, pages, page, Hkv, D],
ksc, vsc [layers, pages, page, Hkv, 4], page_table [rows, max_pages], seq_lens
[rows]; one layer is a qsa_attn cache of pages * page cells):

    qsa_page_update  the batch's next page table: fork, reorder, free, extend
    qsa_paged_prep   norms, rotation and quantised K/V rows of new tokens
    qsa_paged_attn   attention of one new token per row over its whole length
    qsa_paged_gather cached rows as fp16, bf16 or fp32 values
    qsa_page_compact held pages moved to the lowest numbers
"""
from __future__ import annotations

import ctypes
import math

from . import _abi
from ._abi import (QSA_DEVERR_BAD_ID, QSA_DEVERR_NO_PAGES, QSA_DEVERR_TIMEOUT,  # noqa: F401
                   QSA_SCORE_NOALLOC_MAX_TOKENS, QSA_SELECT_MAX_CELLS, QSAError, lib)

__all__ = ["qsa_prep", "qsa_score", "qsa_score_noalloc", "qsa_select", "qsa_attn", "qsa_score_workspace_bytes",
           "qsa_fill_ids_decode", "qsa_fill_ids_even", "qsa_abi_version",
           "qsa_paged_prep", "qsa_paged_gather", "qsa_paged_attn", "qsa_paged_attn_workspace_bytes",
           "qsa_page_update", "qsa_page_compact", "qsa_pages_workspace_bytes",
           "QSAError", "QSA_DEVERR_BAD_ID", "QSA_DEVERR_TIMEOUT", "QSA_DEVERR_NO_PAGES", "QSA_SCORE_NOALLOC_MAX_TOKENS",
           "QSA_SELECT_MAX_CELLS", "lib"]


def _ptr(t, name, dtype=None, optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the QSA path runs only on the GPU)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def qsa_abi_version() -> int:
    return lib().qsa_abi_version()


def qsa_score_workspace_bytes(ntok: int, head_dim: int = 128) -> int:
    return int(lib().qsa_score_workspace_bytes(ntok, head_dim))


def qsa_prep(q_in, k_in, v_in, norm_w, pos0, kq, vq, ksc, vsc, q_out, q_out_f32=None,
             eps=1e-6, rope_theta=10000.0, rope_dims=64, rope_k=False, qbar_out=None, stream=None):
    """Normalise + rotate q_in into q_out (fp16) / q_out_f32 and quantise k_in,
    v_in into cache rows pos0 .. pos0+ntok-1 (with rope_k, the key rows are
    rotated first).  Shapes: q_in [T, Hq, D] fp32, k_in / v_in [T, 1, D]
    fp32, norm_w [D], kq / vq [C, D] int8, ksc / vsc [C, D/32] fp16.
    qbar_out, if given, is a qsa_score workspace (qsa_score_workspace_bytes(T)
    bytes) that receives the score's head sum, for a qsa_score call with
    workspace_holds_qbar=True."""
    import torch
    T, H, D = q_in.shape
    a = _abi.PrepArgs(ntok=T, pos0=int(pos0), n_q_heads=H, n_kv_heads=k_in.shape[1], head_dim=D, group=32,
                      rope_dims=int(rope_dims), cache_cells=kq.shape[0], eps=float(eps),
                      rope_theta=float(rope_theta),
                      q_in=_ptr(q_in, "q_in", torch.float32), k_in=_ptr(k_in, "k_in", torch.float32),
                      v_in=_ptr(v_in, "v_in", torch.float32), norm_w=_ptr(norm_w, "norm_w", torch.float32),
                      q_out=_ptr(q_out, "q_out", torch.float16),
                      q_out_f32=_ptr(q_out_f32, "q_out_f32", torch.float32, optional=True),
                      kq=_ptr(kq, "kq", torch.int8), vq=_ptr(vq, "vq", torch.int8),
                      ksc=_ptr(ksc, "ksc", torch.float16), vsc=_ptr(vsc, "vsc", torch.float16),
                      rope_k=1 if rope_k else 0, qbar_out=_ptr(qbar_out, "qbar_out", optional=True))
    _abi.check(lib().qsa_prep(ctypes.byref(a), _stream(stream)))


def qsa_score(q, kq, ksc, pos0, scores, workspace, err=None, stream=None, workspace_holds_qbar=False,
              n_q_heads=12, max_ctas=0):
    """scores[t, c] for c <= pos0 + t (others untouched).  q [T, Hq, D] fp32 or
    fp16; scores [T, ld] fp32 with ld >= pos0 + T; workspace a uint8 CUDA
    tensor of at least qsa_score_workspace_bytes(T) bytes.  With
    workspace_holds_qbar=True the workspace was filled by qsa_prep(qbar_out=)
    for these tokens and q may be None (T is then scores.shape[0]).
    max_ctas > 0 caps the persistent CTAs (one per SM when 0), leaving the
    other SMs to kernels on other streams."""
    import torch
    if q is None:
        if not workspace_holds_qbar:
            raise ValueError("q is required unless the workspace holds the head sum")
        T, H, D = scores.shape[0], int(n_q_heads), 128
        qp, qdt = None, _abi.QSA_F32
    else:
        T, H, D = q.shape
        if q.dtype not in (torch.float32, torch.float16):
            raise ValueError("q must be float32 or float16")
        qp, qdt = _ptr(q, "q"), (_abi.QSA_F16 if q.dtype == torch.float16 else _abi.QSA_F32)
    if scores.dim() != 2 or scores.shape[0] < T:
        raise ValueError("scores must be [T, ld]")
    a = _abi.ScoreArgs(ntok=T, pos0=int(pos0), n_q_heads=H, head_dim=D, group=32, cache_cells=kq.shape[0],
                       q=qp, q_dtype=qdt, workspace_holds_qbar=1 if workspace_holds_qbar else 0,
                       kq=_ptr(kq, "kq", torch.int8), ksc=_ptr(ksc, "ksc", torch.float16),
                       scores=_ptr(scores, "scores", torch.float32), ld=scores.shape[1],
                       workspace=_ptr(workspace, "workspace"),
                       workspace_bytes=workspace.numel() * workspace.element_size(),
                       err=_ptr(err, "err", torch.int32, optional=True), max_ctas=int(max_ctas))
    _abi.check(lib().qsa_score(ctypes.byref(a), _stream(stream)))


def qsa_score_noalloc(q, kq, ksc, pos0, scores, err=None, stream=None, max_ctas=0):
    """qsa_score without a caller workspace, for callers that cannot allocate
    device memory when they score.  It uses the library's built-in scratch
    (at most 8192 tokens), so calls must not overlap on the GPU."""
    import torch
    T, H, D = q.shape
    if q.dtype not in (torch.float32, torch.float16):
        raise ValueError("q must be float32 or float16")
    if scores.dim() != 2 or scores.shape[0] < T:
        raise ValueError("scores must be [T, ld]")
    a = _abi.ScoreArgs(ntok=T, pos0=int(pos0), n_q_heads=H, head_dim=D, group=32, cache_cells=kq.shape[0],
                       q=_ptr(q, "q"), q_dtype=_abi.QSA_F16 if q.dtype == torch.float16 else _abi.QSA_F32,
                       kq=_ptr(kq, "kq", torch.int8), ksc=_ptr(ksc, "ksc", torch.float16),
                       scores=_ptr(scores, "scores", torch.float32), ld=scores.shape[1],
                       workspace=None, workspace_bytes=0, err=_ptr(err, "err", torch.int32, optional=True),
                       max_ctas=int(max_ctas))
    _abi.check(lib().qsa_score_noalloc(ctypes.byref(a), _stream(stream)))


def qsa_select(scores, pos0, ids, budget=2048, sink=64, local=256, stream=None):
    """ids [T, W] int32 <- the forced decode window plus the top-scoring causal
    cells of each row of scores [T, ld] fp32 (ties to the lower id), ascending,
    -1 padded."""
    import torch
    T = ids.shape[0]
    if scores.dim() != 2 or scores.shape[0] < T:
        raise ValueError("scores must be [T, ld]")
    a = _abi.SelectArgs(ntok=T, pos0=int(pos0), width=ids.shape[1], budget=int(budget), sink=int(sink),
                        local=int(local), scores=_ptr(scores, "scores", torch.float32), ld=scores.shape[1],
                        ids=_ptr(ids, "ids", torch.int32))
    _abi.check(lib().qsa_select(ctypes.byref(a), _stream(stream)))


def qsa_fill_ids_decode(ids, pos0, sink=64, local=256, stream=None):
    """ids [T, W] int32 <- each token's decode window (sink cells, the
    previous `local` cells, its own cell p = pos0 + t), ascending, -1 padded."""
    import torch
    T, W = ids.shape
    _abi.check(lib().qsa_fill_ids_decode(T, int(pos0), W, int(sink), int(local),
                                         _ptr(ids, "ids", torch.int32), _stream(stream)))


def qsa_fill_ids_even(ids, pos0, select=2048, stream=None):
    """ids [T, W] int32 <- up to `select` evenly spaced causal cells of each
    token (always 0 and p = pos0 + t), ascending, -1 padded."""
    import torch
    T, W = ids.shape
    _abi.check(lib().qsa_fill_ids_even(T, int(pos0), W, int(select), _ptr(ids, "ids", torch.int32),
                                       _stream(stream)))


def qsa_attn(q, kq, vq, ksc, vsc, ids, out, softmax_scale=None, part=None, err=None, gate=None, stream=None):
    """Chunked attention of q [T, Hq, D] fp16 over ids [T, W] int32 (-1 =
    padding, W a multiple of 64) into out [T, Hq, D] fp16.  kq/vq are
    [cells, D] (one KV head) or [cells, Hkv, D] int8, scales [cells, (Hkv,)
    4] fp16; D is 128 (32-dim groups) or 256 (64-dim groups).  gate, if
    given, is [T, Hq, D] fp32 logits: out = fp16(O * sigmoid(gate)).  part,
    if given, is [T, W/64, Hq, D+2] fp32 and selects the split per-chunk +
    merge path."""
    import torch
    T, H, D = q.shape
    hkv = 1 if kq.dim() == 2 else kq.shape[1]
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    a = _abi.AttnArgs(ntok=T, n_q_heads=H, n_kv_heads=hkv, head_dim=D, group=D // 4, cache_cells=kq.shape[0],
                      width=ids.shape[1], q=_ptr(q, "q", torch.float16), kq=_ptr(kq, "kq", torch.int8),
                      vq=_ptr(vq, "vq", torch.int8), ksc=_ptr(ksc, "ksc", torch.float16),
                      vsc=_ptr(vsc, "vsc", torch.float16), ids=_ptr(ids, "ids", torch.int32),
                      softmax_scale=float(softmax_scale), out=_ptr(out, "out", torch.float16),
                      part=_ptr(part, "part", torch.float32, optional=True),
                      err=_ptr(err, "err", torch.int32, optional=True),
                      gate=_ptr(gate, "gate", torch.float32, optional=True))
    _abi.check(lib().qsa_attn(ctypes.byref(a), _stream(stream)))


def _dtype_code(t, name, float32):
    import torch
    code = {torch.float16: _abi.QSA_F16, torch.bfloat16: _abi.QSA_BF16}.get(t.dtype)
    if code is None and float32 and t.dtype == torch.float32:
        code = _abi.QSA_F32
    if code is None:
        raise ValueError(f"{name} must be float16{', bfloat16 or float32' if float32 else ' or bfloat16'}, got {t.dtype}")
    return code


def _shape(t, name, shape):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


def _launch(fn, args, tensors, stream):
    """Calls fn(args, stream) with the tensors' device current; they must all
    be on one, and a given stream must belong to it."""
    import torch
    dev = tensors[0].device
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"all tensors must be on one device, got {dev} and {t.device}")
    if stream is not None and stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {dev}")
    with torch.cuda.device(dev):
        raw = torch.cuda.current_stream(dev).cuda_stream if stream is None else stream.cuda_stream
        _abi.check(fn(ctypes.byref(args), raw))


def _layer_shape(kq, vq, ksc, vsc, what):
    """(cells, KV heads, head dim) of one layer's cache: kq, vq [..., Hkv, D],
    scales [..., Hkv, 4] with the same leading dims."""
    if kq.dim() < 3:
        raise ValueError(f"{what}: kq must be [cells, Hkv, D] or [pages, page, Hkv, D]")
    _shape(vq, "vq", kq.shape)
    for t, name in ((ksc, "ksc"), (vsc, "vsc")):
        _shape(t, name, (*kq.shape[:-1], 4))
    hkv, d = kq.shape[-2:]
    return (kq.numel() // (hkv * d) if hkv * d else 0), hkv, d


def _token_rows(t, name, tokens, heads, d):
    """Token stride of a [T, H, D] input whose heads are contiguous."""
    if t is None or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the QSA path runs only on the GPU)")
    _shape(t, name, (tokens, heads, d))
    if t.numel() and (t.stride(2) != 1 or (heads > 1 and t.stride(1) != d)):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return t.stride(0)


def qsa_paged_prep(q_in, k_in, v_in, positions, slots, kq, vq, ksc, vsc, q_out, q_norm_w=None, k_norm_w=None,
                   inv_freq=None, interleaved=False, eps=1e-6, rope_mscale=1.0, err=None, stream=None):
    """New tokens of any sequences: q_out [T, Hq, D] (fp16 or bf16) <- the
    query heads normed (with q_norm_w [D] fp32) and rotated; pool cell slots[t]
    of kq / vq / ksc / vsc (one layer, [..., Hkv, D] and [..., Hkv, 4]) <- the
    key heads normed (k_norm_w) and rotated and the value heads, quantised.
    q_in [T, Hq, D], k_in / v_in [T, Hkv, D] are fp32, fp16 or bf16, alike;
    tokens may be strided (views of one projection).  inv_freq fp32
    [rope_dims/2] holds the rotation's frequencies (None: no rotation), paired
    in halves or interleaved; positions, slots int32 [T], a slot of -1 marks a
    padding token."""
    import torch
    T, H, D = q_in.shape
    cells, hkv, d = _layer_shape(kq, vq, ksc, vsc, "qsa_paged_prep")
    if d != D:
        raise ValueError(f"q_in has head dim {D}, the cache {d}")
    code = _dtype_code(q_in, "q_in", True)
    if k_in.dtype != q_in.dtype or v_in.dtype != q_in.dtype:
        raise ValueError("q_in, k_in and v_in must have one dtype")
    qs, ks, vs = (_token_rows(t, n, T, h, D) for t, n, h in ((q_in, "q_in", H), (k_in, "k_in", hkv), (v_in, "v_in", hkv)))
    _shape(positions, "positions", (T,))
    _shape(slots, "slots", (T,))
    _shape(q_out, "q_out", (T, H, D))
    _shape(q_norm_w, "q_norm_w", (D,))
    _shape(k_norm_w, "k_norm_w", (D,))
    if inv_freq is not None and inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [rope_dims/2]")
    f32, i32 = torch.float32, torch.int32
    a = _abi.PagedPrepArgs(
        T, H, hkv, D, D // 4, 0 if inv_freq is None else 2 * inv_freq.shape[0], 1 if interleaved else 0, cells, code,
        _dtype_code(q_out, "q_out", False), float(eps), float(rope_mscale), q_in.data_ptr(), k_in.data_ptr(),
        v_in.data_ptr(), qs, ks, vs, _ptr(q_norm_w, "q_norm_w", f32, True), _ptr(k_norm_w, "k_norm_w", f32, True),
        _ptr(inv_freq, "inv_freq", f32, True), _ptr(positions, "positions", i32), _ptr(slots, "slots", i32),
        _ptr(q_out, "q_out"), _ptr(kq, "kq", torch.int8), _ptr(vq, "vq", torch.int8), _ptr(ksc, "ksc", torch.float16),
        _ptr(vsc, "vsc", torch.float16), _ptr(err, "err", i32, True))
    _launch(lib().qsa_paged_prep, a, (q_in, k_in, v_in, positions, slots, kq, vq, ksc, vsc, q_out, q_norm_w, k_norm_w,
                                      inv_freq, err), stream)


def qsa_paged_gather(kq, vq, ksc, vsc, ids, k_out, v_out, rows=None, page_table=None, err=None, stream=None):
    """k_out, v_out [N, Hkv, D] (fp16, bf16 or fp32) <- the cached rows of
    cells ids [N] int32 as the values they stand for; -1 gives zeros.  With
    page_table [R, max_pages] int32 and rows [N] int32, ids[i] is a cell of
    sequence rows[i] and kq [pages, page, Hkv, D]; without, a pool cell."""
    import torch
    cells, hkv, d = _layer_shape(kq, vq, ksc, vsc, "qsa_paged_gather")
    if (rows is None) != (page_table is None):
        raise ValueError("rows and page_table go together")
    n = ids.numel()
    _shape(ids, "ids", (n,))
    _shape(rows, "rows", (n,))
    _shape(k_out, "k_out", (n, hkv, d))
    _shape(v_out, "v_out", (n, hkv, d))
    page = n_rows = wide = 0
    if page_table is not None:
        if kq.dim() != 4 or page_table.dim() != 2:
            raise ValueError("with a page table, kq must be [pages, page, Hkv, D] and page_table [R, max_pages]")
        page, (n_rows, wide) = kq.shape[1], page_table.shape
    code = _dtype_code(k_out, "k_out", True)
    if v_out.dtype != k_out.dtype:
        raise ValueError("k_out and v_out must have one dtype")
    i32 = torch.int32
    a = _abi.PagedGatherArgs(
        n, hkv, d, d // 4, cells, page, n_rows, wide, code, _ptr(kq, "kq", torch.int8), _ptr(vq, "vq", torch.int8),
        _ptr(ksc, "ksc", torch.float16), _ptr(vsc, "vsc", torch.float16), _ptr(ids, "ids", i32),
        _ptr(rows, "rows", i32, True), _ptr(page_table, "page_table", i32, True), _ptr(k_out, "k_out"),
        _ptr(v_out, "v_out"), _ptr(err, "err", i32, True))
    _launch(lib().qsa_paged_gather, a, (kq, vq, ksc, vsc, ids, k_out, v_out, rows, page_table, err), stream)


def qsa_paged_attn_workspace_bytes(n_q_heads: int, n_kv_heads: int, head_dim: int = 128) -> int:
    return int(lib().qsa_paged_attn_workspace_bytes(n_q_heads, n_kv_heads, head_dim))


def qsa_paged_attn(q, kq, vq, ksc, vsc, page_table, seq_lens, out, workspace, rows=None, softmax_scale=None, gate=None,
                   lse=None, err=None, stream=None):
    """Attention of one new token per row: out [T, Hq, D] <- q [T, Hq, D] (both
    fp16 or both bf16) over cells 0 .. seq_lens[t]-1 of sequence rows[t] (t
    itself when rows is None) of one layer of the pool (kq / vq [pages, page,
    Hkv, D], ksc / vsc [pages, page, Hkv, 4]) through page_table [R, max_pages]
    int32.  gate, if given, is fp32 [T, Hq, D] logits: out = O * sigmoid(gate);
    lse, if given, fp32 [T, Hq] receives the log of the softmax denominator.
    workspace is a uint8 CUDA tensor of at least
    qsa_paged_attn_workspace_bytes(Hq, Hkv, D) bytes."""
    import torch
    T, H, D = q.shape
    cells, hkv, d = _layer_shape(kq, vq, ksc, vsc, "qsa_paged_attn")
    if kq.dim() != 4 or d != D:
        raise ValueError(f"kq must be [pages, page, Hkv, {D}], got {tuple(kq.shape)}")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [R, max_pages]")
    code = _dtype_code(q, "q", False)
    _shape(seq_lens, "seq_lens", (T,))
    _shape(rows, "rows", (T,))
    _shape(out, "out", (T, H, D))
    _shape(gate, "gate", (T, H, D))
    _shape(lse, "lse", (T, H))
    f32, i32 = torch.float32, torch.int32
    a = _abi.PagedAttnArgs(
        T, H, hkv, D, D // 4, kq.shape[1], kq.shape[0], page_table.shape[0], page_table.shape[1], code, _ptr(q, "q"),
        _ptr(kq, "kq", torch.int8), _ptr(vq, "vq", torch.int8), _ptr(ksc, "ksc", torch.float16),
        _ptr(vsc, "vsc", torch.float16), _ptr(page_table, "page_table", i32), _ptr(seq_lens, "seq_lens", i32),
        _ptr(rows, "rows", i32, True), 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale),
        _ptr(gate, "gate", f32, True), _ptr(out, "out", q.dtype), _ptr(lse, "lse", f32, True),
        _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(), _ptr(err, "err", i32, True))
    _launch(lib().qsa_paged_attn, a, (q, kq, vq, ksc, vsc, page_table, seq_lens, out, workspace, rows, gate, lse, err),
            stream)


def qsa_pages_workspace_bytes(n_rows: int, n_pages: int) -> int:
    """Workspace of qsa_page_update and qsa_page_compact."""
    return int(lib().qsa_pages_workspace_bytes(n_rows, n_pages))


def _pool_shape(kq, vq, ksc, vsc, what):
    """(layers, pages, page, Hkv, D) of a pool, or of one layer of it."""
    if kq.dim() not in (4, 5):
        raise ValueError(f"{what}: kq must be [layers, pages, page, Hkv, D] or [pages, page, Hkv, D]")
    _layer_shape(kq, vq, ksc, vsc, what)
    return (kq.shape[0] if kq.dim() == 5 else 1, *kq.shape[-4:])


def qsa_page_update(page_table, seq_lens, src, n_new, kq, vq, ksc, vsc, page_table_out, seq_lens_out, refs, slots,
                    positions, workspace, err=None, stream=None):
    """The batch's next page table: row r of page_table_out [R, max_pages] and
    seq_lens_out [R] <- the pages and length of old row src[r] (src None: r
    itself; -1: none), grown by n_new[r] tokens with pages from the lowest
    free ones; a partly filled last page that is held more than once is copied
    (all layers) before it grows.  refs [pages] <- how often each page is held;
    slots, positions [N] <- pool cell and position of the packed new tokens, -1
    past them and for a row that could not grow (QSA_DEVERR_NO_PAGES in err).
    All int32.  With src None the outputs may be the inputs.  workspace: uint8,
    qsa_pages_workspace_bytes(R, pages) bytes."""
    import torch
    layers, pages, page, hkv, d = _pool_shape(kq, vq, ksc, vsc, "qsa_page_update")
    if page_table.dim() != 2 or page_table_out.dim() != 2 or page_table.shape[1] != page_table_out.shape[1]:
        raise ValueError("page_table and page_table_out must be [rows, max_pages] of one width")
    r_in, wide = page_table.shape
    r_out = page_table_out.shape[0]
    _shape(seq_lens, "seq_lens", (r_in,))
    _shape(src, "src", (r_out,))
    _shape(n_new, "n_new", (r_out,))
    _shape(seq_lens_out, "seq_lens_out", (r_out,))
    _shape(refs, "refs", (pages,))
    _shape(slots, "slots", (slots.numel(),))
    _shape(positions, "positions", slots.shape)
    i32 = torch.int32
    a = _abi.PageUpdateArgs(
        r_in, r_out, wide, layers, pages, page, hkv, d, d // 4, slots.numel(), _ptr(page_table, "page_table", i32),
        _ptr(seq_lens, "seq_lens", i32), _ptr(src, "src", i32, True), _ptr(n_new, "n_new", i32),
        _ptr(kq, "kq", torch.int8), _ptr(vq, "vq", torch.int8), _ptr(ksc, "ksc", torch.float16),
        _ptr(vsc, "vsc", torch.float16), _ptr(page_table_out, "page_table_out", i32),
        _ptr(seq_lens_out, "seq_lens_out", i32), _ptr(refs, "refs", i32), _ptr(slots, "slots", i32),
        _ptr(positions, "positions", i32), _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _ptr(err, "err", i32, True))
    _launch(lib().qsa_page_update, a, (page_table, seq_lens, src, n_new, kq, vq, ksc, vsc, page_table_out, seq_lens_out,
                                       refs, slots, positions, workspace, err), stream)


def qsa_page_compact(page_table, seq_lens, kq, vq, ksc, vsc, page_table_out, refs, page_map, n_live, workspace, err=None,
                     stream=None):
    """Moves the pages that rows of page_table [R, max_pages] hold (by
    seq_lens [R]) to the lowest page numbers: n_live [1] <- how many there are,
    page_map [pages] <- each page's new number (-1: free), page_table_out and
    refs [pages] by the new numbers, and the moved pages' contents in all
    layers.  All int32; page_table_out may be page_table.  workspace: uint8,
    qsa_pages_workspace_bytes(R, pages) bytes."""
    import torch
    layers, pages, page, hkv, d = _pool_shape(kq, vq, ksc, vsc, "qsa_page_compact")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [rows, max_pages]")
    rows, wide = page_table.shape
    _shape(seq_lens, "seq_lens", (rows,))
    _shape(page_table_out, "page_table_out", (rows, wide))
    _shape(refs, "refs", (pages,))
    _shape(page_map, "page_map", (pages,))
    _shape(n_live, "n_live", (1,))
    i32 = torch.int32
    a = _abi.PageCompactArgs(
        rows, wide, layers, pages, page, hkv, d, d // 4, _ptr(page_table, "page_table", i32),
        _ptr(seq_lens, "seq_lens", i32), _ptr(kq, "kq", torch.int8), _ptr(vq, "vq", torch.int8),
        _ptr(ksc, "ksc", torch.float16), _ptr(vsc, "vsc", torch.float16), _ptr(page_table_out, "page_table_out", i32),
        _ptr(refs, "refs", i32), _ptr(page_map, "page_map", i32), _ptr(n_live, "n_live", i32),
        _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(), _ptr(err, "err", i32, True))
    _launch(lib().qsa_page_compact, a, (page_table, seq_lens, kq, vq, ksc, vsc, page_table_out, refs, page_map, n_live,
                                        workspace, err), stream)
