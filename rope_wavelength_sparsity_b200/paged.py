"""Binding of the paged-cache operators: what a serving step does around ``decode_paged``.

A cache is a pair of page pools k_pages, v_pages [num_pages, page_size, Hkv, D] (bf16 CUDA; one
pair per layer), a block table [rows, max_pages] (int32 CUDA, -1 = no page, all of it -1 to begin
with), refs [num_pages] (int32 CUDA, how many table entries name each page) and the sequences'
lengths, which the host keeps.  A step: ``pages_extend`` for the pages that the new tokens need,
``append_paged`` to rotate and store them, then ``prefill_paged`` (or ``decode_paged``) to attend;
``pages_fork``, ``pages_free``, ``pages_copy`` and ``pages_compact`` tend the pages between steps.

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
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _on(dev, stream):
    """Context in which a call on tensors of device index dev allocates and launches."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
        return torch.cuda.stream(stream)
    return _NOTHING if dev == torch.cuda.current_device() else torch.cuda.device(dev)


def _stream(dev):
    """torch's current stream of device index dev, as the library takes it."""
    return torch._C._cuda_getCurrentRawStream(dev)


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


def _device(t, name):
    """Device index of a CUDA tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    dev = t.get_device()
    if dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    return dev


def _tensor(t, name, dtype, dev, shape=None):
    """Check a contiguous tensor on device index dev; its device pointer."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor")
    if t.get_device() != dev:
        raise TypeError(f"{name} must be a CUDA tensor on cuda:{dev}, not on {t.device}")
    return t.data_ptr()


def _tokens(t, name, dev):
    """Check [T, H, D] bf16 whose tokens may be strided; (pointer, elements between tokens, shape)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    if t.dtype is not _BF16 or stride[2] != 1 or (shape[1] > 1 and stride[1] != shape[2]):
        raise TypeError(f"{name} must be bf16 with each token's heads contiguous")
    if t.get_device() != dev:
        raise TypeError(f"{name} must be a CUDA tensor on cuda:{dev}, not on {t.device}")
    return t.data_ptr(), stride[0] if shape[0] > 1 else shape[1] * shape[2], shape


def _pages(k_pages, v_pages, dev):
    """Check a pair of page pools; (k pointer, v pointer, (num_pages, page_size, Hkv, D))."""
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must be [num_pages, page_size, Hkv, D]")
    shape = k_pages.shape
    return _tensor(k_pages, "k_pages", _BF16, dev), _tensor(v_pages, "v_pages", _BF16, dev, shape), shape


def _table(block_table, dev, rows=None):
    """Check a block table; (pointer, rows, entries of a row)."""
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [rows, max_pages]")
    n, width = block_table.shape
    if rows is not None and n != rows:
        raise ValueError(f"block_table has {n} rows for {rows} sequences")
    return _tensor(block_table, "block_table", _I32, dev), n, width


def prefill_paged_workspace_size(w: Window, q_len, kv_len, Hq: int, Hkv: int) -> int:
    """Workspace bytes of ``prefill_paged`` on the current device."""
    B = len(q_len)
    ql, kl = _ints(q_len), _ints(kv_len, B)
    return int(lib().wpattn_prefill_paged_workspace_size(ctypes.byref(w._c()), _at(ql), _at(kl), B, Hq, Hkv))


def prefill_paged(q, k_pages, v_pages, block_table, q_len, kv_len, w: Window, *, scale: float | None = None,
                  out=None, lse=None, want_lse: bool = True, workspace=None, stream=None):
    """Windowed attention of a ragged batch of chunks over a paged cache.

    q [T, Hq, D]: the new tokens of each sequence one after another, q_len[b] of them; kv_len[b]
    counts the sequence's cached keys, the new tokens' among them.  The window goes by the distance
    of cache rows, also where ``append_paged`` was given other positions (``decode_paged`` takes
    those; with alpha = inf no distance matters).  Rows of q behind the last sequence are not read,
    those of out and lse left as they are.  Returns (out [T, Hq, D] bf16, lse [T, Hq] fp32 or None).
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
    kp, vp, pools = _pages(k_pages, v_pages, q.get_device())
    num_pages, page_size, Hkv, Dk = pools
    if Dk != D:
        raise ValueError(f"k_pages has head dim {Dk}, q {D}")
    dev = _device(q, "q")
    qp = _tensor(q, "q", _BF16, dev)
    tp, _, width = _table(block_table, dev, B)
    if out is not None:
        _tensor(out, "out", _BF16, dev, q.shape)
    if lse is not None:
        _tensor(lse, "lse", _F32, dev, (T, Hq))
    if workspace is not None:
        _tensor(workspace, "workspace", _U8, dev)
    L, cw = lib(), ctypes.byref(w._c())
    with _on(dev, stream):
        if workspace is None:
            need = L.wpattn_prefill_paged_workspace_size(cw, _at(ql), _at(kl), B, Hq, Hkv)
            if need:
                workspace = torch.empty(need, dtype=_U8, device=q.device)
        if out is None:
            out = torch.empty_like(q)
        if lse is None and want_lse:
            lse = torch.empty((T, Hq), dtype=_F32, device=q.device)
        rc = L.wpattn_prefill_paged(cw, qp, kp, vp, num_pages, page_size, tp, width, _at(ql), _at(kl), B, Hq, Hkv,
                                    float(scale) if scale else 0.0, out.data_ptr(),
                                    None if lse is None else lse.data_ptr(),
                                    None if workspace is None else workspace.data_ptr(),
                                    0 if workspace is None else workspace.numel(), _stream(dev))
    _check(rc, "wpattn_prefill_paged")
    return out, lse


def _positions(positions, tokens, dev):
    """Check positions [tokens] or [axes, tokens]; (pointer, stride, axes)."""
    shape = positions.shape if isinstance(positions, torch.Tensor) else ()
    if len(shape) not in (1, 2):
        raise ValueError("positions must be [tokens] or [axes, tokens]")
    if shape[-1] < tokens:
        raise ValueError(f"positions has {shape[-1]} entries for {tokens} tokens")
    return _tensor(positions, "positions", _I32, dev), shape[-1], shape[0] if len(shape) == 2 else 1


def _pair_axes(pair_axes, D, axes):
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
    dev = q.get_device() if isinstance(q, torch.Tensor) else -1
    qp, qs, (T, Hq, D) = _tokens(q, "q", dev)
    kp, ks, Hkv = None, 0, 0
    if k is not None:
        kp, ks, (Tk, Hkv, Dk) = _tokens(k, "k", dev)
        if Tk != T or Dk != D:
            raise ValueError(f"k has shape {tuple(k.shape)}, expected [{T}, Hkv, {D}]")
    elif k_out is not None:
        raise ValueError("k_out without k")
    pp, pstride, axes = _positions(positions, T, dev)
    pa = None if pair_axes is None else _pair_axes(pair_axes, D, axes)
    dev = _device(q, "q")
    if q_out is not None:
        _tensor(q_out, "q_out", _BF16, dev, q.shape)
    if k_out is not None:
        _tensor(k_out, "k_out", _BF16, dev, k.shape)
    with _on(dev, stream):
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        if k is not None and k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        rc = lib().wpattn_rope_axes(qp, qs, q_out.data_ptr(), kp, ks, None if k is None else k_out.data_ptr(), T, Hq,
                                    Hkv, D, pp, pstride, axes, pa, float(base), 1 if inverse else 0, _stream(dev))
    _check(rc, "wpattn_rope_axes")
    return q_out, k_out


def append_paged(k, v, k_pages, v_pages, block_table, new_len, kv_len, *, q=None, q_out=None,
                 base: float | None = None, positions=None, pair_axes=None, stream=None):
    """New tokens into a paged cache: k, v [T, Hkv, D] of new_len[b] tokens of each sequence, one
    after another, become rows kv_len[b] - new_len[b] .. kv_len[b] - 1 (kv_len counts them).

    With ``base`` k is rotated on the way, and q [T, Hq, D] beside it (returned), as in
    ``rope_axes`` by ``positions`` and ``pair_axes`` (None: by each token's cache row).  Positions
    are not kept with the cache: ``prefill_paged`` prunes by the distance of rows whatever they
    were.  k, v and q may be slices of one projection.  Rows behind the last sequence are neither
    read nor written.
    """
    dev = k.get_device() if isinstance(k, torch.Tensor) else -1
    kp, ks, shape = _tokens(k, "k", dev)
    vp, vs, vshape = _tokens(v, "v", dev)
    T, Hkv, D = shape
    if vshape != shape:
        raise ValueError(f"v has shape {tuple(vshape)}, expected {tuple(shape)}")
    B = len(new_len)
    nl, kl = _ints(new_len, B, "new_len"), _ints(kv_len, B, "kv_len")
    tokens = sum(nl)
    if tokens > T:
        raise ValueError(f"k has {T} rows for {tokens} new tokens")
    kpp, vpp, (num_pages, page_size, Hp, Dp) = _pages(k_pages, v_pages, dev)
    if Hp != Hkv or Dp != D:
        raise ValueError(f"the pages hold {Hp} heads of {Dp}, k {Hkv} of {D}")
    tp, _, width = _table(block_table, dev, B)
    if base is None and (q is not None or positions is not None or pair_axes is not None):
        raise ValueError("q, positions and pair_axes need base")
    qp, qs, Hq = None, 0, 0
    if q is not None:
        qp, qs, (Tq, Hq, Dq) = _tokens(q, "q", dev)
        if Tq != T or Dq != D:
            raise ValueError(f"q has shape {tuple(q.shape)}, expected [{T}, Hq, {D}]")
        if q_out is not None:
            _tensor(q_out, "q_out", _BF16, dev, q.shape)
    elif q_out is not None:
        raise ValueError("q_out without q")
    pp, pstride, axes = (None, 0, 1) if positions is None else _positions(positions, tokens, dev)
    pa = None if pair_axes is None else _pair_axes(pair_axes, D, axes)
    dev = _device(k, "k")
    with _on(dev, stream):
        if q is not None and q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        rc = lib().wpattn_append_paged(kp, ks, vp, vs, qp, qs, None if q is None else q_out.data_ptr(), kpp, vpp,
                                       num_pages, page_size, tp, width, _at(nl), _at(kl), B, Hq, Hkv, D, pp, pstride,
                                       axes, pa, 0.0 if base is None else float(base), _stream(dev))
    _check(rc, "wpattn_append_paged")
    return q_out


def _pools(pools, dev, num_pages=None):
    """Check page pools of one cache; (array of pointers, their shape, bytes of a page)."""
    if not pools:
        raise ValueError("the cache's pools are missing")
    shape = pools[0].shape if isinstance(pools[0], torch.Tensor) else ()
    if len(shape) != 4:
        raise ValueError("the pools must be [num_pages, page_size, Hkv, D], all of one shape")
    if num_pages is not None and shape[0] != num_pages:
        raise ValueError(f"the pools have {shape[0]} pages, refs {num_pages}")
    array_of = (ctypes.c_void_p * len(pools))(*[_tensor(t, f"pools[{i}]", _BF16, dev, shape)
                                               for i, t in enumerate(pools)])
    return array_of, shape, shape[1] * shape[2] * shape[3] * 2


def _refs(refs, block_table):
    """Check a cache's refs and table; (device index, refs pointer, num_pages, table pointer, rows, width)."""
    if not isinstance(refs, torch.Tensor) or refs.dim() != 1:
        raise ValueError("refs must be [num_pages]")
    dev = refs.get_device()
    rp = _tensor(refs, "refs", _I32, dev)
    return (dev, rp, refs.shape[0], *_table(block_table, dev))


def _pages_workspace(workspace, num_pages, dev):
    if workspace is None:
        return torch.empty(lib().wpattn_pages_workspace_size(num_pages), dtype=_U8, device=f"cuda:{dev}")
    _tensor(workspace, "workspace", _U8, dev)
    return workspace


def pages_copy(pools, src, dst, *, stream=None):
    """Page src[i] onto page dst[i] in every pool (src, dst int32 CUDA [n])."""
    if not isinstance(src, torch.Tensor) or src.dim() != 1:
        raise ValueError("src must be [n]")
    dev = src.get_device()
    sp, dp = _tensor(src, "src", _I32, dev), _tensor(dst, "dst", _I32, dev, src.shape)
    pools = list(pools)
    array_of, shape, page_bytes = _pools(pools, dev)
    dev = _device(src, "src")
    with _on(dev, stream):
        rc = lib().wpattn_pages_copy(array_of, len(pools), shape[0], page_bytes, sp, dp, src.shape[0], _stream(dev))
    _check(rc, "wpattn_pages_copy")


def pages_fork(pools, block_table, refs, src_rows, dst_rows, lens, *, workspace=None, stream=None):
    """Table rows dst_rows[i] become copies of rows src_rows[i] holding lens[i] keys: full pages
    shared, the begun page's keys copied in every pool into a page of its own."""
    dev, rp, num_pages, tp, rows, width = _refs(refs, block_table)
    pools = list(pools)
    array_of, shape, page_bytes = _pools(pools, dev, num_pages)
    src = _ints(src_rows, None, "src_rows")
    n = len(src)
    dst, ln = _ints(dst_rows, n, "dst_rows"), _ints(lens, n, "lens")
    dev = _device(refs, "refs")
    with _on(dev, stream):
        workspace = _pages_workspace(workspace, num_pages, dev)
        rc = lib().wpattn_pages_fork(array_of, len(pools), num_pages, shape[1], page_bytes // max(shape[1], 1), tp, rows,
                                     width, rp, _at(src), _at(dst), _at(ln), n, workspace.data_ptr(),
                                     workspace.numel(), _stream(dev))
    _check(rc, "wpattn_pages_fork")


def pages_free(block_table, refs, rows, lens, page_size: int, *, stream=None):
    """The pages of rows holding lens[i] keys lose a reference each, and those that a row holds behind
    them (of drafts that were not kept); the entries become -1.  Rows of no keys are left as they are."""
    dev, rp, num_pages, tp, num_rows, width = _refs(refs, block_table)
    r = _ints(rows, None, "rows")
    ln = _ints(lens, len(r), "lens")
    dev = _device(refs, "refs")
    with _on(dev, stream):
        rc = lib().wpattn_pages_free(num_pages, page_size, tp, num_rows, width, rp, _at(r), _at(ln), len(r),
                                     _stream(dev))
    _check(rc, "wpattn_pages_free")


def pages_extend(block_table, refs, rows, lens, new_lens, page_size: int, *, stream=None):
    """Rows growing from lens[i] to new_lens[i] keys get the pages they lack, lowest free first; pages
    that a row holds behind lens[i] (of drafts that were not kept) it grows into."""
    dev, rp, num_pages, tp, num_rows, width = _refs(refs, block_table)
    r = _ints(rows, None, "rows")
    a, b = _ints(lens, len(r), "lens"), _ints(new_lens, len(r), "new_lens")
    dev = _device(refs, "refs")
    with _on(dev, stream):
        rc = lib().wpattn_pages_extend(num_pages, page_size, tp, num_rows, width, rp, _at(r), _at(a), _at(b), len(r),
                                       _stream(dev))
    _check(rc, "wpattn_pages_extend")


def pages_compact(pools, block_table, refs, *, workspace=None, stream=None):
    """The pages in use move into the first slots of every pool; the table and refs follow.
    Returns how many there are (int32 CUDA [1])."""
    dev, rp, num_pages, tp, rows, width = _refs(refs, block_table)
    pools = list(pools)
    array_of, _, page_bytes = _pools(pools, dev, num_pages)
    dev = _device(refs, "refs")
    with _on(dev, stream):
        workspace = _pages_workspace(workspace, num_pages, dev)
        live = refs.new_empty(1)
        rc = lib().wpattn_pages_compact(array_of, len(pools), num_pages, page_bytes, tp, rows * width, rp,
                                        live.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream(dev))
    _check(rc, "wpattn_pages_compact")
    return live
