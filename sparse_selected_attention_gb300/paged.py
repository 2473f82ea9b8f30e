"""Python binding of the paged cache's calls (include/qsa.h, "The paged cache").

A decode step makes three of these calls and its kernels take some
microseconds each, so the host's share is kept small: _paged_binding
(csrc/paged_binding.cpp) checks and reads the tensors on torch's C++ side and
makes the call.  Where it finds anything amiss it says so, and the functions
below called _checked_* look again: they hold the checks with their words, and
make the calls that need another device current.  The checks are the C ABI's
and the ones only Python can make (device, dtype, shape, contiguity):
everything the kernels index by is a shape that was checked here.
"""
from __future__ import annotations

import struct
import sysconfig

import torch

from . import _abi


def binding_of_this_torch():
    """The compiled binding, if it was built for the torch and interpreter that run."""
    how = "build it with `python -m sparse_selected_attention_gb300.build --all`"
    try:
        from . import _paged_binding as native
    except ImportError as e:
        raise RuntimeError(f"_paged_binding.so is missing or of another torch: {how}") from e
    made_for = (getattr(native, "torch_version", None), getattr(native, "abi_tag", None))
    here = (torch.__version__, sysconfig.get_config_var("SOABI"))
    if made_for != here:
        raise RuntimeError(f"_paged_binding.so is for torch {made_for[0]} ({made_for[1]}), this is {here[0]} ({here[1]}): {how}")
    return native


class _NoBinding:
    """In the binding's place where there is none: each paged call says why."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise RuntimeError(self._why)


try:
    _native = binding_of_this_torch()
except RuntimeError as e:
    _native = _NoBinding(str(e))
F32, F16, BF16, I32, I8 = torch.float32, torch.float16, torch.bfloat16, torch.int32, torch.int8
_CODE = {F32: _abi.QSA_F32, F16: _abi.QSA_F16, BF16: _abi.QSA_BF16}
# The raw handle of the current stream and the current device's number: what
# torch.cuda.current_stream() and current_device() wrap, without their objects.
_raw_stream, _current_device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))


def _formats():
    """struct formats of the argument structs, from their ctypes mirrors."""
    letter = {_abi._c_int: "i", _abi._c_float: "f", _abi._vp: "P", _abi.ctypes.c_int64: "q", _abi.ctypes.c_size_t: "N"}
    return {cls: struct.Struct("@" + "".join(letter[t] for _, t in cls._fields_))
            for cls in (_abi.PagedPrepArgs, _abi.PagedGatherArgs, _abi.PagedAttnArgs, _abi.PageUpdateArgs, _abi.PageCompactArgs,
                        _abi.PageBoundsArgs, _abi.PageScoreArgs, _abi.PageSelectArgs, _abi.PagedSparseAttnArgs,
                        _abi.PagedTreeAttnArgs)}


_FORMAT = _formats()
_PREP, _GATHER, _ATTN, _UPDATE, _COMPACT, _BOUNDS, _SCORE, _SELECT, _SPARSE, _TREE = (_FORMAT[c].pack for c in _FORMAT)


def _bad(t, name, dtype, shape, dev):
    """Says what is wrong with a tensor that failed _in()'s checks."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the QSA path runs only on the GPU)")
    if t.get_device() != dev:
        raise ValueError(f"all tensors must be on one device: {name} is on {t.device}, the first on cuda:{dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _in(t, name, dtype, shape, dev):
    """Address of a contiguous tensor of this dtype, shape and device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _bad(t, name, dtype, shape, dev)
    return t.data_ptr()


def _opt(t, name, dtype, shape, dev):
    return 0 if t is None else _in(t, name, dtype, shape, dev)


def _err(t, dev):
    """Address of the device error word, a one-element int32 tensor."""
    if t is None:
        return 0
    if t.dtype is not I32 or t.get_device() != dev or t.numel() < 1:
        raise ValueError("err must be an int32 CUDA tensor on the other tensors' device")
    return t.data_ptr()


def _scratch(t, dev):
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the other tensors' device")
    return t.data_ptr(), t.numel() * t.element_size()


def _cache(kq, vq, ksc, vsc, dev):
    """Addresses of a cache: codes [..., Hkv, D], scales [..., Hkv, 4]."""
    shape = kq.shape
    scales = (*shape[:-1], 4)
    return (_in(kq, "kq", I8, shape, dev), _in(vq, "vq", I8, shape, dev), _in(ksc, "ksc", F16, scales, dev),
            _in(vsc, "vsc", F16, scales, dev))


def _call(name, packed, dev, stream):
    """Runs a library call with the tensors' device current."""
    if stream is None:
        raw = _raw_stream(dev)
    elif stream.device_index != dev:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors are on cuda:{dev}")
    else:
        raw = stream.cuda_stream
    fn = _abi.packed(name)
    if _current_device() == dev:
        status = fn(packed, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(packed, raw)
    if status:
        _abi.check(status)


def _again(status, checked, *args):
    """After a call that did not go through: the library's status, or -1."""
    if status > 0:
        _abi.check(status)
    checked(*args)


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
    status = _native.prep(_abi.entry("qsa_paged_prep"), q_in, k_in, v_in, positions, slots, kq, vq, ksc, vsc, q_out,
                          q_norm_w, k_norm_w, inv_freq, interleaved, eps, rope_mscale, err, stream)
    if status:
        _again(status, _checked_prep, q_in, k_in, v_in, positions, slots, kq, vq, ksc, vsc, q_out, q_norm_w, k_norm_w, inv_freq,
               interleaved, eps, rope_mscale, err, stream)


def _checked_prep(q_in, k_in, v_in, positions, slots, kq, vq, ksc, vsc, q_out, q_norm_w, k_norm_w, inv_freq,
                  interleaved, eps, rope_mscale, err, stream):
    T, H, D = q_in.shape
    dev, itype = q_in.get_device(), q_in.dtype
    hkv, d = kq.shape[-2:]
    cells = kq.numel() // max(hkv * d, 1)
    if dev < 0:
        raise ValueError("q_in must be a CUDA tensor (the QSA path runs only on the GPU)")
    if itype not in _CODE or q_out.dtype not in (F16, BF16):
        raise ValueError(f"q_in must be float16, bfloat16 or float32 and q_out float16 or bfloat16, got {itype}, {q_out.dtype}")
    if kq.dim() < 3 or d != D:
        raise ValueError(f"kq must be [cells, Hkv, {D}] or [pages, page, Hkv, {D}], got {tuple(kq.shape)}")
    strides = []
    for t, name, h in ((q_in, "q_in", H), (k_in, "k_in", hkv), (v_in, "v_in", hkv)):
        if t.dtype is not itype or t.get_device() != dev or t.shape != (T, h, D):
            raise ValueError(f"{name} must be {itype} {(T, h, D)} on cuda:{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
        st, sh, sd = t.stride()
        if t.numel() and (sd != 1 or (h > 1 and sh != D)):
            raise ValueError(f"{name}: a token's heads must be contiguous")
        strides.append(st)
    rope = 0
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [rope_dims/2]")
        rope = 2 * inv_freq.shape[0]
    kv = _cache(kq, vq, ksc, vsc, dev)
    _call("qsa_paged_prep", _PREP(
        T, H, hkv, D, D // 4, rope, 1 if interleaved else 0, cells, _CODE[itype], _CODE[q_out.dtype], eps, rope_mscale,
        q_in.data_ptr(), k_in.data_ptr(), v_in.data_ptr(), *strides, _opt(q_norm_w, "q_norm_w", F32, (D,), dev),
        _opt(k_norm_w, "k_norm_w", F32, (D,), dev), _opt(inv_freq, "inv_freq", F32, (rope // 2,), dev),
        _in(positions, "positions", I32, (T,), dev), _in(slots, "slots", I32, (T,), dev),
        _in(q_out, "q_out", q_out.dtype, (T, H, D), dev), *kv, _err(err, dev)), dev, stream)


def qsa_paged_gather(kq, vq, ksc, vsc, ids, k_out, v_out, rows=None, page_table=None, err=None, stream=None):
    """k_out, v_out [N, Hkv, D] (fp16, bf16 or fp32) <- the cached rows of
    cells ids [N] int32 as the values they stand for; -1 gives zeros.  With
    page_table [R, max_pages] int32 and rows [N] int32, ids[i] is a cell of
    sequence rows[i] and kq [pages, page, Hkv, D]; without, a pool cell."""
    status = _native.gather(_abi.entry("qsa_paged_gather"), kq, vq, ksc, vsc, ids, k_out, v_out, rows, page_table,
                            err, stream)
    if status:
        _again(status, _checked_gather, kq, vq, ksc, vsc, ids, k_out, v_out, rows, page_table, err, stream)


def _checked_gather(kq, vq, ksc, vsc, ids, k_out, v_out, rows, page_table, err, stream):
    hkv, d = kq.shape[-2:]
    dev, otype = kq.get_device(), k_out.dtype
    cells = kq.numel() // max(hkv * d, 1)
    if dev < 0:
        raise ValueError("kq must be a CUDA tensor (the QSA path runs only on the GPU)")
    if otype not in _CODE:
        raise ValueError(f"k_out must be float16, bfloat16 or float32, got {otype}")
    if (rows is None) != (page_table is None):
        raise ValueError("rows and page_table go together")
    n = ids.numel()
    page = n_rows = wide = 0
    if page_table is not None:
        if kq.dim() != 4 or page_table.dim() != 2:
            raise ValueError("with a page table, kq must be [pages, page, Hkv, D] and page_table [R, max_pages]")
        page, (n_rows, wide) = kq.shape[1], page_table.shape
    elif kq.dim() < 3:
        raise ValueError("kq must be [cells, Hkv, D] or [pages, page, Hkv, D]")
    kv = _cache(kq, vq, ksc, vsc, dev)
    _call("qsa_paged_gather", _GATHER(
        n, hkv, d, d // 4, cells, page, n_rows, wide, _CODE[otype], *kv, _in(ids, "ids", I32, (n,), dev),
        _opt(rows, "rows", I32, (n,), dev), _opt(page_table, "page_table", I32, (n_rows, wide), dev),
        _in(k_out, "k_out", otype, (n, hkv, d), dev), _in(v_out, "v_out", otype, (n, hkv, d), dev), _err(err, dev)),
          dev, stream)


def qsa_paged_attn_workspace_bytes(n_q_heads: int, n_kv_heads: int, head_dim: int = 128) -> int:
    return int(_abi.lib().qsa_paged_attn_workspace_bytes(n_q_heads, n_kv_heads, head_dim))


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
    status = _native.attn(_abi.entry("qsa_paged_attn"), q, kq, vq, ksc, vsc, page_table, seq_lens, out, workspace,
                          rows, softmax_scale, gate, lse, err, stream)
    if status:
        _again(status, _checked_attn, q, kq, vq, ksc, vsc, page_table, seq_lens, out, workspace, rows, softmax_scale, gate, lse, err,
               stream)


def _checked_attn(q, kq, vq, ksc, vsc, page_table, seq_lens, out, workspace, rows, softmax_scale, gate, lse, err,
                  stream):
    T, H, D = q.shape
    dev, dtype = q.get_device(), q.dtype
    if dev < 0:
        raise ValueError("q must be a CUDA tensor (the QSA path runs only on the GPU)")
    if dtype is not F16 and dtype is not BF16:
        raise ValueError(f"q must be float16 or bfloat16, got {dtype}")
    if kq.dim() != 4 or kq.shape[3] != D:
        raise ValueError(f"kq must be [pages, page, Hkv, {D}], got {tuple(kq.shape)}")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [R, max_pages]")
    pages, page, hkv, _ = kq.shape
    table = page_table.shape
    heads = (T, H, D)
    k, v, ks, vs = _cache(kq, vq, ksc, vsc, dev)
    ws, ws_bytes = _scratch(workspace, dev)
    _call("qsa_paged_attn", _ATTN(
        T, H, hkv, D, D // 4, page, pages, table[0], table[1], _CODE[dtype], _in(q, "q", dtype, heads, dev), k, v, ks, vs,
        _in(page_table, "page_table", I32, table, dev), _in(seq_lens, "seq_lens", I32, (T,), dev),
        _opt(rows, "rows", I32, (T,), dev), D ** -0.5 if softmax_scale is None else softmax_scale,
        _opt(gate, "gate", F32, heads, dev), _in(out, "out", dtype, heads, dev), _opt(lse, "lse", F32, (T, H), dev), ws, ws_bytes,
        _err(err, dev)), dev, stream)


def qsa_pages_workspace_bytes(n_rows: int, n_pages: int) -> int:
    """Workspace of qsa_page_update and qsa_page_compact."""
    return int(_abi.lib().qsa_pages_workspace_bytes(n_rows, n_pages))


def _pool(kq, page_table):
    """Device and (layers, pages, page, Hkv, D) of a pool, or of one layer of it."""
    dev = kq.get_device()
    if dev < 0:
        raise ValueError("kq must be a CUDA tensor (the QSA path runs only on the GPU)")
    if kq.dim() not in (4, 5):
        raise ValueError(f"kq must be [layers, pages, page, Hkv, D] or [pages, page, Hkv, D], got {tuple(kq.shape)}")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [rows, max_pages]")
    s = kq.shape
    return dev, (s if len(s) == 5 else (1, *s))


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
    status = _native.update(_abi.entry("qsa_page_update"), page_table, seq_lens, src, n_new, kq, vq, ksc, vsc,
                            page_table_out, seq_lens_out, refs, slots, positions, workspace, err, stream)
    if status:
        _again(status, _checked_update, page_table, seq_lens, src, n_new, kq, vq, ksc, vsc, page_table_out, seq_lens_out, refs, slots,
               positions, workspace, err, stream)


def _checked_update(page_table, seq_lens, src, n_new, kq, vq, ksc, vsc, page_table_out, seq_lens_out, refs, slots,
                    positions, workspace, err, stream):
    dev, (layers, pages, page, hkv, d) = _pool(kq, page_table)
    r_in, wide = page_table.shape
    r_out = n_new.numel()
    n = slots.numel()
    kv = _cache(kq, vq, ksc, vsc, dev)
    ws, ws_bytes = _scratch(workspace, dev)
    _call("qsa_page_update", _UPDATE(
        r_in, r_out, wide, layers, pages, page, hkv, d, d // 4, n, _in(page_table, "page_table", I32, (r_in, wide), dev),
        _in(seq_lens, "seq_lens", I32, (r_in,), dev), _opt(src, "src", I32, (r_out,), dev),
        _in(n_new, "n_new", I32, (r_out,), dev), *kv, _in(page_table_out, "page_table_out", I32, (r_out, wide), dev),
        _in(seq_lens_out, "seq_lens_out", I32, (r_out,), dev), _in(refs, "refs", I32, (pages,), dev),
        _in(slots, "slots", I32, (n,), dev), _in(positions, "positions", I32, (n,), dev), ws, ws_bytes, _err(err, dev)),
          dev, stream)


def qsa_page_compact(page_table, seq_lens, kq, vq, ksc, vsc, page_table_out, refs, page_map, n_live, workspace, err=None,
                     stream=None):
    """Moves the pages that rows of page_table [R, max_pages] hold (by
    seq_lens [R]) to the lowest page numbers: n_live [1] <- how many there are,
    page_map [pages] <- each page's new number (-1: free), page_table_out and
    refs [pages] by the new numbers, and the moved pages' contents in all
    layers.  All int32; page_table_out may be page_table.  workspace: uint8,
    qsa_pages_workspace_bytes(R, pages) bytes."""
    status = _native.compact(_abi.entry("qsa_page_compact"), page_table, seq_lens, kq, vq, ksc, vsc, page_table_out,
                             refs, page_map, n_live, workspace, err, stream)
    if status:
        _again(status, _checked_compact, page_table, seq_lens, kq, vq, ksc, vsc, page_table_out, refs, page_map, n_live, workspace, err,
               stream)


def _checked_compact(page_table, seq_lens, kq, vq, ksc, vsc, page_table_out, refs, page_map, n_live, workspace, err,
                     stream):
    dev, (layers, pages, page, hkv, d) = _pool(kq, page_table)
    rows, wide = table = page_table.shape
    kv = _cache(kq, vq, ksc, vsc, dev)
    ws, ws_bytes = _scratch(workspace, dev)
    _call("qsa_page_compact", _COMPACT(
        rows, wide, layers, pages, page, hkv, d, d // 4, _in(page_table, "page_table", I32, table, dev),
        _in(seq_lens, "seq_lens", I32, (rows,), dev), *kv, _in(page_table_out, "page_table_out", I32, table, dev),
        _in(refs, "refs", I32, (pages,), dev), _in(page_map, "page_map", I32, (pages,), dev),
        _in(n_live, "n_live", I32, (1,), dev), ws, ws_bytes, _err(err, dev)), dev, stream)


def qsa_page_bounds(page_table, seq_lens, kq, ksc, hi_q, lo_q, hi_sc, lo_sc, n_new=None, err=None, stream=None):
    """Bounds of the keys in each page that rows' new tokens are in: hi_q, lo_q
    [pages, Hkv, D] int8 and hi_sc, lo_sc [pages, Hkv, 4] fp16 <- the largest and
    smallest key per dim of the page's filled cells, rounded outwards, by kq
    [pages, page, Hkv, D] and ksc [pages, page, Hkv, 4] (one layer of the pool).
    seq_lens [R] int32 are the rows' lengths with the new tokens, n_new [R] int32
    how many of them are new (None: all).  A cache of one cell per page, which
    qsa_paged_gather reads back."""
    status = _native.bounds(_abi.entry("qsa_page_bounds"), page_table, seq_lens, kq, ksc, hi_q, lo_q, hi_sc, lo_sc, n_new, err,
                            stream)
    if status:
        _again(status, _checked_bounds, page_table, seq_lens, kq, ksc, hi_q, lo_q, hi_sc, lo_sc, n_new, err, stream)


def _page_bounds(hi_q, lo_q, hi_sc, lo_sc, shape, dev):
    scales = (*shape[:-1], 4)
    return (_in(hi_q, "hi_q", I8, shape, dev), _in(lo_q, "lo_q", I8, shape, dev), _in(hi_sc, "hi_sc", F16, scales, dev),
            _in(lo_sc, "lo_sc", F16, scales, dev))


def _checked_bounds(page_table, seq_lens, kq, ksc, hi_q, lo_q, hi_sc, lo_sc, n_new, err, stream):
    dev = kq.get_device()
    if dev < 0:
        raise ValueError("kq must be a CUDA tensor (the QSA path runs only on the GPU)")
    if kq.dim() != 4 or page_table.dim() != 2:
        raise ValueError(f"kq must be [pages, page, Hkv, D] and page_table [R, max_pages], got {tuple(kq.shape)}, {tuple(page_table.shape)}")
    pages, page, hkv, d = kq.shape
    rows, wide = table = page_table.shape
    _call("qsa_page_bounds", _BOUNDS(
        rows, wide, pages, page, hkv, d, d // 4, _in(page_table, "page_table", I32, table, dev),
        _in(seq_lens, "seq_lens", I32, (rows,), dev), _opt(n_new, "n_new", I32, (rows,), dev), _in(kq, "kq", I8, kq.shape, dev),
        _in(ksc, "ksc", F16, (pages, page, hkv, 4), dev), *_page_bounds(hi_q, lo_q, hi_sc, lo_sc, (pages, hkv, d), dev),
        _err(err, dev)), dev, stream)


def qsa_page_score(q, hi_q, lo_q, hi_sc, lo_sc, page_table, seq_lens, scores, page_size, rows=None, err=None, stream=None):
    """scores [T, Hkv, ld] fp32 (ld >= the table's columns): element [t, h, j] <-
    the most that the products of q [T, Hq, D]'s query heads of KV head h (fp16 or
    bf16) with a key of page j can add up to, by the bounds of qsa_page_bounds,
    for each page j of the sequence rows[t] (t itself when rows is None) with
    seq_lens[t] cells; the others are left untouched."""
    status = _native.score(_abi.entry("qsa_page_score"), q, hi_q, lo_q, hi_sc, lo_sc, page_table, seq_lens, scores, page_size, rows,
                           err, stream)
    if status:
        _again(status, _checked_score, q, hi_q, lo_q, hi_sc, lo_sc, page_table, seq_lens, scores, page_size, rows, err, stream)


def _tokens(q, page_table):
    """T, H, D, device and type of the queries of a call on a paged cache."""
    if q.dim() != 3:
        raise ValueError(f"q must be [T, Hq, D], got {tuple(q.shape)}")
    dev, dtype = q.get_device(), q.dtype
    if dev < 0:
        raise ValueError("q must be a CUDA tensor (the QSA path runs only on the GPU)")
    if dtype is not F16 and dtype is not BF16:
        raise ValueError(f"q must be float16 or bfloat16, got {dtype}")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [R, max_pages]")
    return *q.shape, dev, dtype


def _checked_score(q, hi_q, lo_q, hi_sc, lo_sc, page_table, seq_lens, scores, page_size, rows, err, stream):
    T, H, D, dev, dtype = _tokens(q, page_table)
    if hi_q.dim() != 3 or hi_q.shape[2] != D:
        raise ValueError(f"hi_q must be [pages, Hkv, {D}], got {tuple(hi_q.shape)}")
    pages, hkv, _ = hi_q.shape
    if scores.dim() != 3:
        raise ValueError(f"scores must be [{T}, {hkv}, ld], got {tuple(scores.shape)}")
    table, ld = page_table.shape, scores.shape[2]
    _call("qsa_page_score", _SCORE(
        T, H, hkv, D, D // 4, page_size, pages, table[0], table[1], _CODE[dtype], _in(q, "q", dtype, (T, H, D), dev),
        *_page_bounds(hi_q, lo_q, hi_sc, lo_sc, hi_q.shape, dev), _in(page_table, "page_table", I32, table, dev),
        _in(seq_lens, "seq_lens", I32, (T,), dev), _opt(rows, "rows", I32, (T,), dev), _in(scores, "scores", F32, (T, hkv, ld), dev), ld,
        _err(err, dev)), dev, stream)


def qsa_page_select(scores, seq_lens, pages, counts, page_size, budget, sink=1, local=1, err=None, stream=None):
    """pages [T, Hkv, W] int32 <- the first `sink` pages of a sequence of
    seq_lens[t] cells, its last `local` and the best of the others by scores [T,
    Hkv, ld] fp32 (ties to the lower page), `budget` in all, ascending, -1 padded;
    counts [T, Hkv] int32 <- how many."""
    status = _native.select(_abi.entry("qsa_page_select"), scores, seq_lens, pages, counts, page_size, budget, sink, local, err,
                            stream)
    if status:
        _again(status, _checked_select, scores, seq_lens, pages, counts, page_size, budget, sink, local, err, stream)


def _checked_select(scores, seq_lens, pages, counts, page_size, budget, sink, local, err, stream):
    dev = scores.get_device()
    if dev < 0:
        raise ValueError("scores must be a CUDA tensor (the QSA path runs only on the GPU)")
    if scores.dim() != 3 or pages.dim() != 3:
        raise ValueError(f"scores must be [T, Hkv, ld] and pages [T, Hkv, W], got {tuple(scores.shape)}, {tuple(pages.shape)}")
    T, hkv, ld = scores.shape
    w = pages.shape[2]
    _call("qsa_page_select", _SELECT(
        T, hkv, page_size, w, budget, sink, local, _in(scores, "scores", F32, (T, hkv, ld), dev), ld,
        _in(seq_lens, "seq_lens", I32, (T,), dev), _in(pages, "pages", I32, (T, hkv, w), dev), _in(counts, "counts", I32, (T, hkv), dev),
        _err(err, dev)), dev, stream)


def qsa_paged_sparse_attn_workspace_bytes(n_q_heads: int, n_kv_heads: int, head_dim: int = 128) -> int:
    return int(_abi.lib().qsa_paged_sparse_attn_workspace_bytes(n_q_heads, n_kv_heads, head_dim))


def qsa_paged_sparse_attn(q, kq, vq, ksc, vsc, page_table, seq_lens, pages, counts, out, workspace, rows=None, softmax_scale=None,
                          gate=None, lse=None, err=None, stream=None):
    """qsa_paged_attn over listed pages: KV head h of row t attends to the cells
    below seq_lens[t] of the first counts[t, h] pages of pages [T, Hkv, W] int32
    (page numbers of the sequence, -1 is padding), as qsa_page_select writes them.
    workspace is a uint8 CUDA tensor of at least
    qsa_paged_sparse_attn_workspace_bytes(Hq, Hkv, D) bytes."""
    status = _native.sparse_attn(_abi.entry("qsa_paged_sparse_attn"), q, kq, vq, ksc, vsc, page_table, seq_lens, pages, counts, out,
                                 workspace, rows, softmax_scale, gate, lse, err, stream)
    if status:
        _again(status, _checked_sparse, q, kq, vq, ksc, vsc, page_table, seq_lens, pages, counts, out, workspace, rows, softmax_scale,
               gate, lse, err, stream)


def _attn_parts(T, H, D, dev, dtype, q, kq, vq, ksc, vsc, page_table, out, gate, lse, rows):
    """What the two calls below check alike: the sizes, and addresses by name."""
    if kq.dim() != 4 or kq.shape[3] != D:
        raise ValueError(f"kq must be [pages, page, Hkv, {D}], got {tuple(kq.shape)}")
    pages, page, hkv, _ = kq.shape
    table, heads = page_table.shape, (T, H, D)
    kv = _cache(kq, vq, ksc, vsc, dev)
    return ((T, H, hkv, D, D // 4, page, pages, table[0], table[1]), (_in(q, "q", dtype, heads, dev), *kv,
            _in(page_table, "page_table", I32, table, dev)), _opt(rows, "rows", I32, (T,), dev),
            (_opt(gate, "gate", F32, heads, dev), _in(out, "out", dtype, heads, dev), _opt(lse, "lse", F32, (T, H), dev)))


def _checked_sparse(q, kq, vq, ksc, vsc, page_table, seq_lens, pages, counts, out, workspace, rows, softmax_scale, gate, lse, err,
                    stream):
    T, H, D, dev, dtype = _tokens(q, page_table)
    sizes, first, rows, last = _attn_parts(T, H, D, dev, dtype, q, kq, vq, ksc, vsc, page_table, out, gate, lse, rows)
    hkv = sizes[2]
    if pages.dim() != 3:
        raise ValueError(f"pages must be [{T}, {hkv}, W], got {tuple(pages.shape)}")
    w = pages.shape[2]
    ws, ws_bytes = _scratch(workspace, dev)
    _call("qsa_paged_sparse_attn", _SPARSE(
        *sizes, w, _CODE[dtype], *first, _in(seq_lens, "seq_lens", I32, (T,), dev), rows, _in(pages, "pages", I32, (T, hkv, w), dev),
        _in(counts, "counts", I32, (T, hkv), dev), D ** -0.5 if softmax_scale is None else softmax_scale, *last, ws, ws_bytes,
        _err(err, dev)), dev, stream)


def qsa_paged_tree_attn_workspace_bytes(n_q_heads: int, n_kv_heads: int, head_dim: int = 128) -> int:
    return int(_abi.lib().qsa_paged_tree_attn_workspace_bytes(n_q_heads, n_kv_heads, head_dim))


def qsa_paged_tree_attn(q, kq, vq, ksc, vsc, page_table, prefix_lens, mask, out, workspace, rows=None, softmax_scale=None, gate=None,
                        lse=None, err=None, stream=None):
    """qsa_paged_attn for drafted tokens that branch: row t attends to cells 0 ..
    prefix_lens[t]-1 of its sequence and to cell prefix_lens[t] + b for each bit b
    of mask [T, words] int32 (bit b % 32 of word b / 32; up to QSA_TREE_MAX_WORDS
    words): of a tree whose node i is cached in cell prefix + i, the node itself
    and those that lead to it.  workspace is a uint8 CUDA tensor of at least
    qsa_paged_tree_attn_workspace_bytes(Hq, Hkv, D) bytes."""
    status = _native.tree_attn(_abi.entry("qsa_paged_tree_attn"), q, kq, vq, ksc, vsc, page_table, prefix_lens, mask, out, workspace,
                               rows, softmax_scale, gate, lse, err, stream)
    if status:
        _again(status, _checked_tree, q, kq, vq, ksc, vsc, page_table, prefix_lens, mask, out, workspace, rows, softmax_scale, gate, lse,
               err, stream)


def _checked_tree(q, kq, vq, ksc, vsc, page_table, prefix_lens, mask, out, workspace, rows, softmax_scale, gate, lse, err, stream):
    T, H, D, dev, dtype = _tokens(q, page_table)
    sizes, first, rows, last = _attn_parts(T, H, D, dev, dtype, q, kq, vq, ksc, vsc, page_table, out, gate, lse, rows)
    if mask.dim() != 2:
        raise ValueError(f"mask must be [{T}, words], got {tuple(mask.shape)}")
    words = mask.shape[1]
    ws, ws_bytes = _scratch(workspace, dev)
    _call("qsa_paged_tree_attn", _TREE(
        *sizes, words, _CODE[dtype], *first, _in(prefix_lens, "prefix_lens", I32, (T,), dev), rows, _in(mask, "mask", I32, (T, words), dev),
        D ** -0.5 if softmax_scale is None else softmax_scale, *last, ws, ws_bytes, _err(err, dev)), dev, stream)
