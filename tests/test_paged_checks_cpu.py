"""Refusals of the paged-cache operators, by the library and by the binding (no kernel runs)."""
import ctypes

import pytest
import torch

import rope_wavelength_sparsity_b200 as wp

V = ctypes.c_void_p(256)                        # an aligned address that nothing reads
ODD = ctypes.c_void_p(258)
W = wp.Window(64, 1e4, 1.0, 1)


def _i(*x):
    return (ctypes.c_int32 * len(x))(*x)


def _p(*x):
    return (ctypes.c_void_p * len(x))(*x)


def _prefill(**kw):
    a = dict(w=W, q=V, k=V, v=V, num_pages=8, page=16, table=V, max_pages=4, q_len=_i(3, 1), kv_len=_i(3, 64), B=2,
             Hq=4, Hkv=2, scale=0.0, out=V, lse=None, ws=None, n=0)
    a.update(kw)
    return wp.lib().wpattn_prefill_paged(ctypes.byref(a["w"]._c()), a["q"], a["k"], a["v"], a["num_pages"], a["page"],
                                         a["table"], a["max_pages"], a["q_len"], a["kv_len"], a["B"], a["Hq"], a["Hkv"],
                                         a["scale"], a["out"], a["lse"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(Hq=3), "EINVAL"), (dict(B=-1), "EINVAL"), (dict(num_pages=0), "EINVAL"), (dict(max_pages=0), "EINVAL"),
    (dict(q_len=_i(3, -1)), "EINVAL"), (dict(kv_len=_i(3, 65)), "EINVAL"), (dict(kv_len=_i(-1, 6)), "EINVAL"),
    (dict(q_len=_i(2**31 - 1, 1)), "EINVAL"), (dict(scale=float("nan")), "EINVAL"), (dict(q=None), "EINVAL"),
    (dict(k=ODD), "EINVAL"), (dict(table=ODD), "EINVAL"), (dict(out=ODD), "EINVAL"), (dict(q_len=None), "EINVAL"),
    (dict(page=24), "EUNSUPPORTED"), (dict(page=4), "EUNSUPPORTED"), (dict(Hq=258, Hkv=2), "EUNSUPPORTED"),
    (dict(w=wp.Window(96, 1e4, 1.0, 1)), "EUNSUPPORTED"), (dict(B=1025), "EUNSUPPORTED"),
    (dict(num_pages=1 << 28), "EUNSUPPORTED"), (dict(w=wp.Window(64, 1e4, -1.0, 1)), "EINVAL"),
    (dict(B=0), "OK"), (dict(q_len=_i(0, 0)), "OK"),
])
def test_prefill_paged_refusals(kw, code):
    assert _prefill(**kw) == getattr(wp, code)


def _rope(**kw):
    a = dict(q=V, qs=256, qo=V, k=V, ks=128, ko=V, T=3, Hq=4, Hkv=2, D=64, pos=V, stride=3, axes=2, pa=None, base=1e4,
             inv=0)
    a.update(kw)
    return wp.lib().wpattn_rope_axes(a["q"], a["qs"], a["qo"], a["k"], a["ks"], a["ko"], a["T"], a["Hq"], a["Hkv"],
                                     a["D"], a["pos"], a["stride"], a["axes"], a["pa"], a["base"], a["inv"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), "EINVAL"), (dict(Hq=0), "EINVAL"), (dict(D=96), "EUNSUPPORTED"), (dict(pos=None), "EINVAL"),
    (dict(axes=0), "EINVAL"), (dict(axes=5), "EINVAL"), (dict(stride=2), "EINVAL"), (dict(base=1.0), "EINVAL"),
    (dict(base=float("inf")), "EINVAL"), (dict(base=float("nan")), "EINVAL"), (dict(qs=255), "EINVAL"),
    (dict(qs=252), "EINVAL"), (dict(ks=120), "EINVAL"), (dict(q=ODD), "EINVAL"), (dict(ko=None), "EINVAL"),
    (dict(pa=(ctypes.c_uint8 * 32)(*([2] * 32))), "EINVAL"), (dict(inv=2), "EINVAL"), (dict(pos=ODD), "EINVAL"),
    (dict(T=0), "OK"),
])
def test_rope_axes_refusals(kw, code):
    assert _rope(**kw) == getattr(wp, code)


def _append(**kw):
    a = dict(k=V, ks=128, v=V, vs=128, q=V, qs=256, qo=V, kp=V, vp=V, num_pages=8, page=16, table=V, max_pages=4,
             new=_i(3, 1), kv=_i(3, 64), B=2, Hq=4, Hkv=2, D=64, pos=None, stride=0, axes=1, pa=None, base=1e4)
    a.update(kw)
    return wp.lib().wpattn_append_paged(*[a[n] for n in "k ks v vs q qs qo kp vp num_pages page table max_pages new kv "
                                          "B Hq Hkv D pos stride axes pa base".split()], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), "EINVAL"), (dict(Hkv=0), "EINVAL"), (dict(qo=None), "EINVAL"), (dict(D=32), "EUNSUPPORTED"),
    (dict(base=0.0), "EINVAL"), (dict(base=0.5), "EINVAL"), (dict(page=12), "EUNSUPPORTED"), (dict(B=1025), "EUNSUPPORTED"),
    (dict(new=_i(4, 1)), "EINVAL"), (dict(new=_i(-1, 1)), "EINVAL"), (dict(kv=_i(3, 65)), "EINVAL"),
    (dict(kp=None), "EINVAL"), (dict(vp=ODD), "EINVAL"), (dict(ks=100), "EINVAL"), (dict(vs=132), "EINVAL"),
    (dict(qs=8), "EINVAL"), (dict(axes=2), "EINVAL"), (dict(pos=V, axes=2, stride=3), "EINVAL"), (dict(num_pages=0), "EINVAL"),
    (dict(B=0), "OK"), (dict(new=_i(0, 0)), "OK"),
])
def test_append_paged_refusals(kw, code):
    assert _append(**kw) == getattr(wp, code)


def test_positions_of_no_token_may_be_null():
    """What an empty [axes, 0] tensor passes."""
    assert _rope(T=0, q=None, qo=None, k=None, ko=None, pos=None, stride=0, axes=3) == wp.OK
    assert _append(new=_i(0, 0), pos=None, axes=3) == wp.OK
    assert _append(new=_i(0, 1), pos=None, axes=3) == wp.EINVAL


def test_page_operator_sizes():
    """At most 2^30 pages and 2^30 keys a row: no index of the kernels passes 32 bits."""
    L, big = wp.lib(), 2**31 - 1

    def calls(num_pages, page, width, length):
        n = L.wpattn_pages_workspace_size(num_pages)
        yield L.wpattn_pages_fork(_p(256), 1, num_pages, page, 32, V, 6, width, V, _i(0), _i(1), _i(length), 1, V, n, None)
        yield L.wpattn_pages_free(num_pages, page, V, 6, width, V, _i(0), _i(length), 1, None)
        yield L.wpattn_pages_extend(num_pages, page, V, 6, width, V, _i(0), _i(0), _i(length), 1, None)

    for args in [(big, 16, 3, 40), (8, 16, big, big), (8, 16, 1 << 27, 40), (8, big, 1, big), (8, big, 2, 7)]:
        assert set(calls(*args)) == {wp.EUNSUPPORTED}, args
    n = L.wpattn_pages_workspace_size(big)
    assert L.wpattn_pages_compact(_p(256), 1, big, 32, V, 12, V, V, V, n, None) == wp.EUNSUPPORTED
    assert L.wpattn_pages_copy(_p(256), 1, 8, 32, V, V, big, None) == wp.EUNSUPPORTED


def test_page_operator_refusals():
    L = wp.lib()
    ok = wp.EINVAL, wp.EUNSUPPORTED
    # copy
    assert L.wpattn_pages_copy(_p(256), 1, 8, 24, V, V, 2, None) == ok[0]       # not a multiple of 16 bytes
    assert L.wpattn_pages_copy(_p(258), 1, 8, 32, V, V, 2, None) == ok[0]
    assert L.wpattn_pages_copy(_p(256), 1, 0, 32, V, V, 2, None) == ok[0]
    assert L.wpattn_pages_copy(_p(256), 1, 8, 32, None, V, 2, None) == ok[0]
    assert L.wpattn_pages_copy(_p(*[256] * 257), 257, 8, 32, V, V, 2, None) == ok[1]
    assert L.wpattn_pages_copy(_p(256), 1, 8, 32, None, None, 0, None) == wp.OK
    # fork

    def fork(src, dst, ln, rows=6, max_pages=3, row_bytes=32, ws=V, size=1 << 20, n=None):
        return L.wpattn_pages_fork(_p(256), 1, 8, 16, row_bytes, V, rows, max_pages, V, _i(*src), _i(*dst), _i(*ln),
                                   len(src) if n is None else n, ws, size, None)

    assert fork([0, 0], [1, 1], [5, 5]) == ok[0]                                # one row twice
    assert fork([0, 1], [1, 2], [5, 5]) == ok[0]                                # a source that is written
    assert fork([0], [6], [5]) == ok[0] and fork([0], [-1], [5]) == ok[0] and fork([6], [1], [5]) == ok[0]
    assert fork([0], [1], [49]) == ok[0] and fork([0], [1], [-1]) == ok[0]
    assert fork([0], [1], [5], row_bytes=8) == ok[0]
    assert fork([0], [1], [5], ws=None) == wp.EWORKSPACE and fork([0], [1], [5], size=100) == wp.EWORKSPACE
    assert fork([0], [1], [5], n=1025) == ok[1] and fork([], [], []) == wp.OK
    # free and extend
    assert L.wpattn_pages_free(8, 16, V, 6, 3, V, _i(1, 1), _i(5, 5), 2, None) == ok[0]
    assert L.wpattn_pages_free(8, 16, V, 6, 3, V, _i(1), _i(49), 1, None) == ok[0]
    assert L.wpattn_pages_free(8, 16, V, 6, 3, None, _i(1), _i(4), 1, None) == ok[0]
    assert L.wpattn_pages_free(8, 16, V, 6, 3, V, _i(1), _i(0), 1, None) == wp.OK
    assert L.wpattn_pages_extend(8, 16, V, 6, 3, V, _i(1), _i(9), _i(8), 1, None) == ok[0]   # it shrinks
    assert L.wpattn_pages_extend(8, 16, V, 6, 3, V, _i(2, 2), _i(1, 1), _i(40, 40), 2, None) == ok[0]
    assert L.wpattn_pages_extend(8, 16, V, 6, 3, V, _i(2), _i(1), _i(49), 1, None) == ok[0]
    assert L.wpattn_pages_extend(8, 16, V, 6, 3, V, _i(2), _i(1), _i(16), 1, None) == wp.OK  # no page needed
    # compact
    assert L.wpattn_pages_compact(_p(256), 1, 8, 32, V, 12, V, V, None, 0, None) == wp.EWORKSPACE
    assert L.wpattn_pages_compact(_p(256), 1, 8, 32, None, 12, V, V, V, 1 << 20, None) == ok[0]
    assert L.wpattn_pages_compact(_p(256), 1, 8, 32, V, 12, V, ODD, V, 1 << 20, None) == ok[0]
    assert L.wpattn_pages_workspace_size(0) == 0 and L.wpattn_pages_workspace_size(8) >= 72
    assert L.wpattn_strerror(wp.EPAGES).decode() != "unknown status code"


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _int(*shape):
    return torch.zeros(shape, dtype=torch.int32)


KP, VP, T2 = _bf(8, 16, 2, 64), _bf(8, 16, 2, 64), _int(2, 4)


@pytest.mark.parametrize("call", [
    lambda: wp.prefill_paged(_bf(4, 4, 32), KP, VP, T2, [3, 1], [3, 9], W),          # head dim
    lambda: wp.prefill_paged(_bf(3, 4, 64), KP, VP, T2, [3, 1], [3, 9], W),          # too few rows
    lambda: wp.prefill_paged(_bf(4, 4, 64), KP, VP, T2, [3, 1], [3], W),
    lambda: wp.prefill_paged(_bf(4, 4, 64), KP, VP, T2, [3], [3], W, out=_bf(4, 4, 64)),
    lambda: wp.prefill_paged(_bf(4, 4, 64), KP, _bf(7, 16, 2, 64), T2, [3, 1], [3, 9], W),
    lambda: wp.prefill_paged(_bf(4, 4, 64), KP, VP, T2, [3, 1], [3, 2**40], W),
    lambda: wp.rope_axes(_bf(4, 4, 64), _bf(3, 2, 64), _int(4), base=1e4),
    lambda: wp.rope_axes(_bf(4, 4, 64), None, _int(2, 3), base=1e4),
    lambda: wp.append_paged(_bf(4, 2, 64), _bf(4, 1, 64), KP, VP, T2, [3, 1], [3, 9]),
    lambda: wp.append_paged(_bf(4, 2, 64), _bf(4, 2, 64), KP, VP, T2, [3, 2], [3, 9]),
    lambda: wp.append_paged(_bf(4, 2, 64), _bf(4, 2, 64), KP, VP, T2, [3, 1], [3, 9], q=_bf(4, 2, 64)),
    lambda: wp.pages_fork([KP, VP], T2, _int(7), [0], [1], [4]),
    lambda: wp.pages_free(T2, _int(8, 1), [0], [4], 16),
    lambda: wp.pages_extend(T2, _int(8), [0, 1], [4], [5, 5], 16),
    lambda: wp.pages_copy([KP], _int(3, 1), _int(3)),
])
def test_binding_refusals(call):
    with pytest.raises((ValueError, TypeError)):
        call()


def test_binding_checks_types_and_layout():
    with pytest.raises(TypeError):
        wp.prefill_paged(_bf(4, 4, 64).float(), KP, VP, T2, [3, 1], [3, 9], W)
    with pytest.raises(TypeError):
        wp.prefill_paged(_bf(4, 8, 64)[:, ::2], KP, VP, T2, [3, 1], [3, 9], W)
    with pytest.raises(TypeError):
        wp.append_paged(_bf(4, 2, 128)[..., ::2], _bf(4, 2, 64), KP, VP, T2, [3, 1], [3, 9])
    with pytest.raises(TypeError, match="CUDA"):
        wp.rope_axes(_bf(4, 4, 64), None, _int(4), base=1e4)
    with pytest.raises(AttributeError):
        wp.no_such_operator
