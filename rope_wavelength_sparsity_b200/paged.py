"""Binding of the paged-cache operators: what a serving step does around ``decode_paged``.

A cache is a pair of page pools k_pages, v_pages [num_pages, page_size, Hkv, D] (bf16 CUDA; one
pair per layer), a block table [rows, max_pages] (int32 CUDA, -1 = no page), refs [num_pages]
(int32 CUDA, how many table entries name each page) and the sequences' lengths, which the host
keeps.  A step: ``pages_extend`` for the pages that the new tokens need, ``append_paged`` to
rotate and store them, then ``prefill_paged`` (or ``decode_paged``) to attend; ``pages_fork``,
``pages_free``, ``pages_copy`` and ``pages_compact`` tend the pages between steps.

Calls run on torch's current stream of the tensors' device, or on ``stream``: what a call
allocates then belongs to that stream.  Lengths and row numbers are host ints.
"""
from __future__ import annotations

import contextlib
import ctypes
from array import array

import torch

from . import Window, _check, lib

_NOTHING = contextlib.nullcontext()


def _on(t, stream):
    """Context in which a call on tensor t allocates and launches."""
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
        return torch.cuda.stream(stream)
    return _NOTHING if t.device.index == torch.cuda.current_device() else torch.cuda.device(t.device)


def _stream(t):
    """torch's current stream of t's device, as the library takes it."""
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _ints(values, n=None, what="lengths"):
    """Host ints as an array of int32; pass ``.buffer_info()[0]`` on."""
    try:
        a = array("i", values)
    except OverflowError as e:
        raise ValueError(f"{what}: {e}") from None
    if n is not None and len(a) != n:
        raise ValueError(f"{what} has {len(a)} entries, expected {n}")
    return a


def _at(a):
    return a.buffer_info()[0]


def _tensor(t, name, dtype, like=None, shape=None):
    """Check a contiguous CUDA tensor; its device pointer."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if like is not None and t.device != like.device:
        raise TypeError(f"{name} must be on {like.device}")
    return t.data_ptr()


def _tokens(t, name, like=None):
    """Check [T, H, D] bf16 whose tokens may be strided; (pointer, elements between tokens)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    if t.dtype != torch.bfloat16 or t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise TypeError(f"{name} must be bf16 with each token's heads contiguous")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if like is not None and t.device != like.device:
        raise TypeError(f"{name} must be on {like.device}")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def _pages(k_pages, v_pages, like=None):
    """Check a pair of page pools; (k pointer, v pointer, (num_pages, page_size, Hkv, D))."""
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must be [num_pages, page_size, Hkv, D]")
    return (_tensor(k_pages, "k_pages", torch.bfloat16, like),
            _tensor(v_pages, "v_pages", torch.bfloat16, k_pages, k_pages.shape), k_pages.shape)


def _table(block_table, like, rows=None):
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [rows, max_pages]")
    if rows is not None and block_table.shape[0] != rows:
        raise ValueError(f"block_table has {block_table.shape[0]} rows for {rows} sequences")
    return _tensor(block_table, "block_table", torch.int32, like)


def prefill_paged_workspace_size(w: Window, q_len, kv_len, Hq: int, Hkv: int) -> int:
    """Workspace bytes of ``prefill_paged`` on the current device."""
    B = len(q_len)
    ql, kl = _ints(q_len), _ints(kv_len, B)
    return int(lib().wpattn_prefill_paged_workspace_size(ctypes.byref(w._c()), _at(ql), _at(kl), B, Hq, Hkv))


def prefill_paged(q, k_pages, v_pages, block_table, q_len, kv_len, w: Window, *, scale: float | None = None,
                  out=None, lse=None, want_lse: bool = True, workspace=None, stream=None):
    """Windowed attention of a ragged batch of chunks over a paged cache.

    q [T, Hq, D]: the new tokens of each sequence one after another, q_len[b] of them; kv_len[b]
    counts the sequence's cached keys, the new tokens' among them.  Rows of q behind the last
    sequence are not read, those of out and lse left as they are.  Returns (out [T, Hq, D] bf16,
    lse [T, Hq] fp32 or None).
    """
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [tokens, Hq, D]")
    T, Hq, D = q.shape
    B = len(q_len)
    if D != w.head_dim:
        raise ValueError(f"q has head dim {D}, the window {w.head_dim}")
    ql, kl = _ints(q_len, B, "q_len"), _ints(kv_len, B, "kv_len")
    if sum(ql) > T:
        raise ValueError(f"q has {T} rows for {sum(ql)} new tokens")
    qp = _tensor(q, "q", torch.bfloat16)
    kp, vp, (num_pages, page_size, Hkv, Dk) = _pages(k_pages, v_pages, q)
    if Dk != D:
        raise ValueError(f"k_pages has head dim {Dk}, q {D}")
    tp = _table(block_table, q, B)
    if out is not None:
        _tensor(out, "out", torch.bfloat16, q, q.shape)
    if lse is not None:
        _tensor(lse, "lse", torch.float32, q, (T, Hq))
    if workspace is not None:
        _tensor(workspace, "workspace", torch.uint8, q)
    L, cw = lib(), ctypes.byref(w._c())
    with _on(q, stream):
        if workspace is None:
            need = L.wpattn_prefill_paged_workspace_size(cw, _at(ql), _at(kl), B, Hq, Hkv)
            if need:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        if out is None:
            out = torch.empty_like(q)
        if lse is None and want_lse:
            lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
        rc = L.wpattn_prefill_paged(cw, qp, kp, vp, num_pages, page_size, tp, block_table.shape[1], _at(ql), _at(kl), B,
                                    Hq, Hkv, float(scale) if scale else 0.0, out.data_ptr(),
                                    lse.data_ptr() if lse is not None else None,
                                    workspace.data_ptr() if workspace is not None else None,
                                    workspace.numel() if workspace is not None else 0, _stream(q))
    _check(rc, "wpattn_prefill_paged")
    return out, lse


def _positions(positions, tokens, like):
    """Check positions [tokens] or [axes, tokens]; (pointer, stride, axes)."""
    if not isinstance(positions, torch.Tensor) or positions.dim() not in (1, 2):
        raise ValueError("positions must be [tokens] or [axes, tokens]")
    if positions.shape[-1] < tokens:
        raise ValueError(f"positions has {positions.shape[-1]} entries for {tokens} tokens")
    return (_tensor(positions, "positions", torch.int32, like), positions.shape[-1],
            positions.shape[0] if positions.dim() == 2 else 1)


def _pair_axes(pair_axes, D, axes):
    if pair_axes is None:
        return None
    pair_axes = bytes(pair_axes)               # refuses what is not in 0 .. 255
    if len(pair_axes) != D // 2 or max(pair_axes) >= axes:
        raise ValueError(f"pair_axes must name one of {axes} axes for each of {D // 2} pairs")
    return pair_axes


def rope_axes(q, k, positions, pair_axes=None, *, base: float, inverse: bool = False, q_out=None, k_out=None,
              stream=None):
    """RoPE with positions along several axes: pair p of token t turns by
    positions[pair_axes[p], t] * base^(-2p/D), or by minus that (``inverse``: the rotation's
    transpose and gradient).  q [T, Hq, D] and k [T, Hkv, D] (or None) may be slices of one
    projection; positions int32 CUDA [axes, T] (1 to 4 axes) or [T]; pair_axes: the axis of each
    of the D/2 pairs (None: all 0).  Returns (q_out, k_out)."""
    qp, qs = _tokens(q, "q")
    T, Hq, D = q.shape
    kp, ks, Hkv = None, 0, 0
    if k is not None:
        kp, ks = _tokens(k, "k", q)
        Hkv = k.shape[1]
        if k.shape[0] != T or k.shape[2] != D:
            raise ValueError(f"k has shape {tuple(k.shape)}, expected [{T}, Hkv, {D}]")
    elif k_out is not None:
        raise ValueError("k_out without k")
    pp, pstride, axes = _positions(positions, T, q)
    pa = _pair_axes(pair_axes, D, axes)
    for t, o, name in ((q, q_out, "q_out"), (k, k_out, "k_out")):
        if o is not None:
            _tensor(o, name, torch.bfloat16, q, t.shape)
    with _on(q, stream):
        if q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
        if k is not None and k_out is None:
            k_out = torch.empty((T, Hkv, D), dtype=q.dtype, device=q.device)
        rc = lib().wpattn_rope_axes(qp, qs, q_out.data_ptr(), kp, ks, k_out.data_ptr() if k is not None else None, T,
                                    Hq, Hkv, D, pp, pstride, axes, pa, float(base), int(bool(inverse)), _stream(q))
    _check(rc, "wpattn_rope_axes")
    return q_out, k_out


def append_paged(k, v, k_pages, v_pages, block_table, new_len, kv_len, *, q=None, q_out=None,
                 base: float | None = None, positions=None, pair_axes=None, stream=None):
    """New tokens into a paged cache: k, v [T, Hkv, D] of new_len[b] tokens of each sequence, one
    after another, become rows kv_len[b] - new_len[b] .. kv_len[b] - 1 (kv_len counts them).

    With ``base`` k is rotated on the way, and q [T, Hq, D] beside it (returned), as in
    ``rope_axes`` by ``positions`` and ``pair_axes`` (None: by each token's cache row).  k, v and q
    may be slices of one projection.  Rows behind the last sequence are neither read nor written.
    """
    kp, ks = _tokens(k, "k")
    vp, vs = _tokens(v, "v", k)
    T, Hkv, D = k.shape
    if tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"v has shape {tuple(v.shape)}, expected {tuple(k.shape)}")
    B = len(new_len)
    nl, kl = _ints(new_len, B, "new_len"), _ints(kv_len, B, "kv_len")
    tokens = sum(nl)
    if tokens > T:
        raise ValueError(f"k has {T} rows for {tokens} new tokens")
    kpp, vpp, (num_pages, page_size, Hp, Dp) = _pages(k_pages, v_pages, k)
    if (Hp, Dp) != (Hkv, D):
        raise ValueError(f"the pages hold {Hp} heads of {Dp}, k {Hkv} of {D}")
    tp = _table(block_table, k, B)
    if base is None and (q is not None or positions is not None or pair_axes is not None):
        raise ValueError("q, positions and pair_axes need base")
    qp, qs, Hq = None, 0, 0
    if q is not None:
        qp, qs = _tokens(q, "q", k)
        Hq = q.shape[1]
        if q.shape[0] != T or q.shape[2] != D:
            raise ValueError(f"q has shape {tuple(q.shape)}, expected [{T}, Hq, {D}]")
        if q_out is not None:
            _tensor(q_out, "q_out", torch.bfloat16, k, q.shape)
    elif q_out is not None:
        raise ValueError("q_out without q")
    pp, pstride, axes = (None, 0, 1) if positions is None else _positions(positions, tokens, k)
    pa = _pair_axes(pair_axes, D, axes)
    with _on(k, stream):
        if q is not None and q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
        rc = lib().wpattn_append_paged(kp, ks, vp, vs, qp, qs, q_out.data_ptr() if q is not None else None, kpp, vpp,
                                       num_pages, page_size, tp, block_table.shape[1], _at(nl), _at(kl), B, Hq, Hkv, D, pp,
                                       pstride, axes, pa, 0.0 if base is None else float(base), _stream(k))
    _check(rc, "wpattn_append_paged")
    return q_out


def _pools(pools, refs, pages_known=True):
    """Check page pools of one cache; (array of pointers, count, bytes of a page)."""
    pools = list(pools)
    for i, t in enumerate(pools):
        _tensor(t, f"pools[{i}]", torch.bfloat16, refs)
        if t.dim() != 4 or t.shape != pools[0].shape:
            raise ValueError("the pools must be [num_pages, page_size, Hkv, D], all of one shape")
        if pages_known and t.shape[0] != refs.shape[0]:
            raise ValueError(f"pools[{i}] has {t.shape[0]} pages, refs {refs.shape[0]}")
    array = (ctypes.c_void_p * max(1, len(pools)))(*[t.data_ptr() for t in pools])
    return array, len(pools), pools[0][0].numel() * 2 if pools and pools[0].shape[0] else 16


def _refs(refs):
    if not isinstance(refs, torch.Tensor) or refs.dim() != 1:
        raise ValueError("refs must be [num_pages]")
    return _tensor(refs, "refs", torch.int32)


def _pages_workspace(workspace, refs):
    if workspace is None:
        return torch.empty(lib().wpattn_pages_workspace_size(refs.shape[0]), dtype=torch.uint8, device=refs.device)
    _tensor(workspace, "workspace", torch.uint8, refs)
    return workspace


def pages_copy(pools, src, dst, *, stream=None):
    """Page src[i] onto page dst[i] in every pool (src, dst int32 CUDA [n])."""
    pools = list(pools)
    if not pools:
        return
    if not isinstance(src, torch.Tensor) or src.dim() != 1:
        raise ValueError("src must be [n]")
    sp, dp = _tensor(src, "src", torch.int32), _tensor(dst, "dst", torch.int32, src, src.shape)
    array, n, page_bytes = _pools(pools, src, pages_known=False)
    with _on(src, stream):
        rc = lib().wpattn_pages_copy(array, n, pools[0].shape[0], page_bytes, sp, dp, src.shape[0], _stream(src))
    _check(rc, "wpattn_pages_copy")


def pages_fork(pools, block_table, refs, src_rows, dst_rows, lens, *, workspace=None, stream=None):
    """Table rows dst_rows[i] become copies of rows src_rows[i] holding lens[i] keys: full pages
    shared, the begun page's keys copied in every pool into a page of its own."""
    rp, tp = _refs(refs), _table(block_table, refs)
    pools = list(pools)
    array, n_pools, page_bytes = _pools(pools, refs)
    if not pools:
        raise ValueError("pages_fork needs the cache's pools")
    page_size = pools[0].shape[1]
    src = _ints(src_rows, None, "src_rows")
    n = len(src)
    dst, ln = _ints(dst_rows, n, "dst_rows"), _ints(lens, n, "lens")
    with _on(refs, stream):
        workspace = _pages_workspace(workspace, refs)
        rc = lib().wpattn_pages_fork(array, n_pools, refs.shape[0], page_size, page_bytes // page_size, tp,
                                     block_table.shape[0], block_table.shape[1], rp, _at(src), _at(dst), _at(ln), n,
                                     workspace.data_ptr(), workspace.numel(), _stream(refs))
    _check(rc, "wpattn_pages_fork")


def pages_free(block_table, refs, rows, lens, page_size: int, *, stream=None):
    """The pages of rows holding lens[i] keys lose a reference each; their entries become -1."""
    rp, tp = _refs(refs), _table(block_table, refs)
    r = _ints(rows, None, "rows")
    ln = _ints(lens, len(r), "lens")
    with _on(refs, stream):
        rc = lib().wpattn_pages_free(refs.shape[0], page_size, tp, block_table.shape[0], block_table.shape[1], rp, _at(r),
                                     _at(ln), len(r), _stream(refs))
    _check(rc, "wpattn_pages_free")


def pages_extend(block_table, refs, rows, lens, new_lens, page_size: int, *, stream=None):
    """Rows growing from lens[i] to new_lens[i] keys get the pages they lack, lowest free first."""
    rp, tp = _refs(refs), _table(block_table, refs)
    r = _ints(rows, None, "rows")
    a, b = _ints(lens, len(r), "lens"), _ints(new_lens, len(r), "new_lens")
    with _on(refs, stream):
        rc = lib().wpattn_pages_extend(refs.shape[0], page_size, tp, block_table.shape[0], block_table.shape[1], rp, _at(r),
                                       _at(a), _at(b), len(r), _stream(refs))
    _check(rc, "wpattn_pages_extend")


def pages_compact(pools, block_table, refs, *, workspace=None, stream=None):
    """The pages in use move into the first slots of every pool; the table and refs follow.
    Returns how many there are (int32 CUDA [1])."""
    rp, tp = _refs(refs), _table(block_table, refs)
    array, n_pools, page_bytes = _pools(pools, refs)
    with _on(refs, stream):
        workspace = _pages_workspace(workspace, refs)
        live = torch.empty(1, dtype=torch.int32, device=refs.device)
        rc = lib().wpattn_pages_compact(array, n_pools, refs.shape[0], page_bytes, tp, block_table.numel(), rp,
                                        live.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream(refs))
    _check(rc, "wpattn_pages_compact")
    return live
