"""Largest counts of the paged-cache operators: what 32-bit indexes of the kernels and plans cannot hold is refused
(no kernel runs)."""
import ctypes

import pytest

import rope_wavelength_sparsity_b200 as wp

V = ctypes.c_void_p(256)                        # an aligned address that nothing reads
TOP = 1 << 30


def _i(*x):
    return (ctypes.c_int32 * len(x))(*x)


@pytest.mark.parametrize("page,old,new", [
    (1, [0, 0], [TOP, TOP - 1]),                # 2^31 - 1 pages: the last loop's index would pass 2^31
    (1, [0, 0], [TOP, TOP - 1024]),
    (1, [0, 0], [TOP, TOP]),
    (1, [0, 0], [TOP, 1]),                      # one more than there may be pages
    (8, [0] * 9, [TOP] * 9),
])
def test_extend_by_more_pages_than_a_pool_may_have(page, old, new):
    n = len(old)
    rc = wp.lib().wpattn_pages_extend(1 << 30, page, V, n, TOP // page, V, _i(*range(n)), _i(*old), _i(*new), n, None)
    assert rc == wp.EUNSUPPORTED


@pytest.mark.parametrize("G", [1, 3, 128])
@pytest.mark.parametrize("q_len", [[2**31 - 1], [2**31 - 127], [5, 2**31 - 100]])
def test_prefill_of_more_tokens_than_tiles_can_count(q_len, G):
    """Lengths that, rounded up to whole row tiles, pass 32 bits."""
    w, n = wp.Window(64, 1e4, 1.0, 1), len(q_len)
    ql, kl = _i(*q_len), _i(*[64] * n)
    rc = wp.lib().wpattn_prefill_paged(ctypes.byref(w._c()), V, V, V, 8, 16, V, 4, ql, kl, n, G, 1, 0.0, V, None, V,
                                       1 << 40, None)
    assert rc == wp.EUNSUPPORTED
    assert wp.lib().wpattn_prefill_paged_workspace_size(ctypes.byref(w._c()), ql, kl, n, G, 1) == 0
