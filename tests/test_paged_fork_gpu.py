"""Forks of rows whose pages no count holds."""
import pytest

import rope_wavelength_sparsity_b200 as wp

from test_paged_cache_gpu import _cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("begun", [7, 32])
@pytest.mark.parametrize("length", [32, 20, 3])
def test_fork_from_a_free_page_is_reported(cuda_dev, length, begun):
    """Also where the same call hands that page out for a begun one."""
    for _ in range(5):
        made, table, refs, _ = _cache(16, 1, 64, 2, 8, 6, 2)
        wp.pages_extend(table, refs, [0, 1], [0, 0], [32, 32], 16)
        refs[table[0].long()] = 0                # as if row 0 had been freed with its entries left behind
        wp.pages_fork(made, table, refs, [1, 0, 1], [2, 3, 4], [begun, length, begun])
        assert wp.device_status() == wp.EINDEX
    refs[table[0].long()] = 1
    wp.pages_fork(made, table, refs, [1, 0], [2, 3], [32, 32])
    assert wp.device_status() == wp.OK


def test_every_fork_of_a_thousand_is_looked_at(cuda_dev):
    page, n = 8, 1024
    made, table, refs, host = _cache(page, 1, 64, 1, 4000, n + 2, 4)
    wp.pages_extend(table, refs, [0, 1], [0, 0], [9, 9], page)
    host.extend([0, 1], [0, 0], [9, 9])
    src, dst, lens = [0] * n, list(range(2, n + 2)), [9] * n
    wp.pages_fork(made, table, refs, src, dst, lens)
    host.fork(src, dst, lens)
    assert wp.device_status() == wp.OK
    host.check(made, table, refs)
    wp.pages_free(table, refs, dst, lens, page)
    refs[table[1, 1].long()] = 0                 # the begun page of the last fork's source
    wp.pages_fork(made, table, refs, src[:-1] + [1], dst, lens)
    assert wp.device_status() == wp.EINDEX
