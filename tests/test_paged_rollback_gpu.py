"""Rows whose length goes back (drafts that were not kept): the pages taken for them stay the row's, are used when
it grows again."""
import random

import pytest
import torch

import rope_wavelength_sparsity_b200 as wp

from _paged import pages_of
from test_paged_cache_gpu import Host, _cache

pytestmark = pytest.mark.gpu


class Rows(Host):
    """The rules for rows that hold more pages than their length needs."""

    def extend(self, rows, lens, new):
        slots = [(r, j) for r, a, b in zip(rows, lens, new) for j in range(pages_of(a, self.page), pages_of(b, self.page))]
        slots = [(r, j) for r, j in slots if self.table[r, j] < 0]          # an entry that names a page keeps it
        free = self.free_pages(len(slots))
        for (r, j), pg in zip(slots, free + [-1] * len(slots)):
            self.table[r, j] = pg
            if pg >= 0:
                self.refs[pg] = 1


@pytest.mark.parametrize("page", [1, 8, 16])
def test_draft_reject_grow_free(cuda_dev, page):
    """One sequence: full pages, drafts into the next one, none kept, one token, gone."""
    made, table, refs, _ = _cache(16, 1, 64, 1, 40, 3, 12)
    host = Rows(made, table, refs, page)

    def extend(a, b):
        wp.pages_extend(table, refs, [1], [a], [b], page)
        host.extend([1], [a], [b])
        assert wp.device_status() == wp.OK
        host.check(made, table, refs)

    extend(0, page)
    extend(page, 3 * page - page // 2)
    held = table[1].clone()
    extend(page, page + 1)                       # every draft was rejected
    assert torch.equal(table[1], held)
    extend(page + 1, 5 * page)                   # behind the pages it held
    assert torch.equal(table[1, :3], held[:3])
    assert int(refs.sum()) == 5 and int((table >= 0).sum()) == 5
    wp.pages_free(table, refs, [1], [5 * page], page)
    assert wp.device_status() == wp.OK and not refs.any() and (table == -1).all()


@pytest.mark.parametrize("rows,width,num_pages", [(5, 9, 60), (300, 30, 12000), (1024, 7, 5000)])
def test_lengths_go_back_and_forth(cuda_dev, rows, width, num_pages):
    """Random drafts, cuts and ends of up to 1024 rows, several thousand entries a call, some calls with too few pages."""
    page = 8
    rng = random.Random(rows)
    made, table, refs, _ = _cache(page, 1, 64, 1, num_pages, rows, width)
    host = Rows(made, table, refs, page)
    length = [0] * rows
    for step in range(8):
        some = rng.sample(range(rows), rng.randint(1, rows))
        a = [length[r] for r in some]
        b = [rng.randint(n, min(width * page, n + 12 * page)) for n in a]
        wp.pages_extend(table, refs, some, a, b, page)
        host.extend(some, a, b)
        short = bool((host.table[some] < 0).any(1).any()) and any(
            (host.table[r, :pages_of(n, page)] < 0).any() for r, n in zip(some, b))
        assert wp.device_status() == (wp.EPAGES if short else wp.OK)
        host.check(made, table, refs)
        for r, x, y in zip(some, a, b):
            had = int((host.table[r] >= 0).sum()) * page
            length[r] = rng.randint(x, min(y, max(x, had)))     # what was kept
        gone = rng.sample(range(rows), rows // 4)
        ln = [int((host.table[r] >= 0).sum()) * page for r in gone]
        wp.pages_free(table, refs, gone, ln, page)
        host.free(gone, ln)
        assert wp.device_status() == wp.OK
        host.check(made, table, refs)
        for r in gone:
            length[r] = 0
    assert int(refs.sum()) == int((table >= 0).sum())


def test_extend_over_an_entry_of_a_free_page_is_reported(cuda_dev):
    made, table, refs, _ = _cache(8, 1, 64, 1, 6, 2, 3)
    table[0, 1] = 4                              # names a page that no count holds
    wp.pages_extend(table, refs, [0], [0], [20], 8)
    assert wp.device_status() == wp.EINDEX
    assert table[0].tolist() == [0, 1, 2] and refs.tolist() == [1, 1, 1, 0, 0, 0]


def test_serving_with_rejected_drafts(cuda_dev):
    """Drafts attended, cut back and replaced by other tokens: the pages' rows and counts stay right."""
    page, D, Hkv = 16, 64, 2
    made, table, refs, _ = _cache(page, Hkv, D, 2, 40, 2, 20)
    kp, vp = made
    gen = torch.Generator().manual_seed(1)
    kept = [torch.zeros((0, Hkv, D), dtype=torch.bfloat16) for _ in range(2)]
    rng = random.Random(3)
    for _ in range(20):
        n = [len(x) for x in kept]
        new = [rng.randint(1, 9), rng.randint(1, 30)]
        kv = [min(a + b, 20 * page) for a, b in zip(n, new)]
        new = [b - a for a, b in zip(n, kv)]
        wp.pages_extend(table, refs, [0, 1], n, kv, page)
        k = torch.randn((sum(new), Hkv, D), generator=gen).to(torch.bfloat16)
        wp.append_paged(k.cuda(), k.cuda(), kp, vp, table, new, kv)
        at = 0
        for r, m in enumerate(new):
            kept[r] = torch.cat([kept[r], k[at:at + rng.randint(0, m)]])   # the drafts that stay
            at += m
    assert wp.device_status() == wp.OK
    for r, x in enumerate(kept):
        rows = kp[table[r, :pages_of(len(x), page)].long()].view(-1, Hkv, D)[:len(x)]
        assert torch.equal(rows.cpu(), x)
    used = table[table >= 0]
    assert len(used.unique()) == len(used) and int(refs.sum()) == len(used)


class Ending(Rows):
    """Rows that end with their kept length."""

    def free(self, rows, lens):
        for r, n in zip(rows, lens):
            j, width = 0, self.table.shape[1]
            while n > 0 and j < width and (j < pages_of(n, self.page) or self.table[r, j] >= 0):
                self.refs[self.table[r, j]] -= 1
                self.table[r, j] = -1
                j += 1


@pytest.mark.parametrize("kept", [1, 17, 16, 32, 33])
def test_free_with_the_kept_length(cuda_dev, kept):
    """A sequence that ends right after its drafts were rejected gives back their pages too."""
    page = 16
    made, table, refs, _ = _cache(page, 1, 64, 1, 700, 3, 600)
    host = Ending(made, table, refs, page)
    for rows, a, b in (([0, 2], [0, 0], [kept, 20]), ([0], [kept], [kept + 9000])):   # more pages than a block has threads
        wp.pages_extend(table, refs, rows, a, b, page)
        host.extend(rows, a, b)
    assert wp.device_status() == wp.OK
    host.check(made, table, refs)
    wp.pages_free(table, refs, [0], [kept], page)
    host.free([0], [kept])
    assert wp.device_status() == wp.OK
    host.check(made, table, refs)
    assert int(refs.sum()) == 2 and (table[0] == -1).all()


def test_free_up_to_the_last_column(cuda_dev):
    made, table, refs, _ = _cache(8, 1, 64, 1, 9, 2, 3)
    wp.pages_extend(table, refs, [0, 1], [0, 0], [24, 24], 8)
    wp.pages_free(table, refs, [0], [3], 8)      # all three columns; the next row's stay
    assert wp.device_status() == wp.OK
    assert table.tolist() == [[-1] * 3, [3, 4, 5]] and refs.tolist() == [0, 0, 0, 1, 1, 1, 0, 0, 0]
    wp.pages_free(table, refs, [0, 1], [0, 8], 8)   # a row of no keys is left as it is
    assert wp.device_status() == wp.OK and not refs.any()


@pytest.mark.parametrize("rows,width,num_pages", [(5, 9, 60), (300, 30, 12000), (1024, 7, 5000)])
def test_rows_end_with_their_kept_lengths(cuda_dev, rows, width, num_pages):
    page = 8
    rng = random.Random(rows + 1)
    made, table, refs, _ = _cache(page, 1, 64, 1, num_pages, rows, width)
    host = Ending(made, table, refs, page)
    for _ in range(4):
        new = [rng.randint(0, width * page) for _ in range(rows)]
        wp.pages_extend(table, refs, range(rows), [0] * rows, new, page)
        host.extend(range(rows), [0] * rows, new)
        wp.device_status()                        # some calls run out of pages: then rows hold fewer
        kept = [rng.randint(0, int((host.table[r] >= 0).sum()) * page) for r in range(rows)]
        kept = [max(n, 1) if host.table[r, 0] >= 0 else 0 for r, n in enumerate(kept)]
        wp.pages_free(table, refs, range(rows), kept, page)
        host.free(range(rows), kept)
        assert wp.device_status() == wp.OK
        host.check(made, table, refs)
        assert not refs.any() and (table == -1).all()


def test_growing_over_a_shared_page_is_reported(cuda_dev):
    """A row cut back below a length it was forked at: its tokens would go into pages that the fork reads."""
    made, table, refs, _ = _cache(8, 1, 64, 1, 9, 3, 4)
    wp.pages_extend(table, refs, [0], [0], [24], 8)
    wp.pages_fork(made, table, refs, [0], [1], [24])
    wp.pages_extend(table, refs, [0], [24], [25], 8)           # both go on from there
    assert wp.device_status() == wp.OK
    wp.pages_extend(table, refs, [0], [24], [30], 8)           # a page of its own
    assert wp.device_status() == wp.OK
    wp.pages_extend(table, refs, [0], [16], [20], 8)
    assert wp.device_status() == wp.EINDEX
    assert table[0].tolist() == [0, 1, 2, 3] and refs.tolist() == [2, 2, 2, 1, 0, 0, 0, 0, 0]


def test_entries_of_free_pages_in_a_large_call(cuda_dev):
    """Several thousand entries: the first rows are given the pages that the last row's entries name."""
    made, table, refs, _ = _cache(8, 1, 64, 1, 9000, 3, 6000)
    refs[5] = 1                                  # in use elsewhere
    table[2, :3] = torch.tensor([7, 8999, 3], dtype=torch.int32)
    wp.pages_extend(table, refs, [0, 1, 2], [0, 0, 0], [8 * 5000, 8 * 100, 8 * 3], 8)
    assert wp.device_status() == wp.EINDEX
    used = table[table >= 0]
    assert len(used) == 5103 and len(used.unique()) == 5103
    assert refs.tolist() == [1] * 5104 + [0] * (9000 - 5104)
    assert table[2, :3].tolist() == [5101, 5102, 5103]
