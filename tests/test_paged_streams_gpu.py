"""Every paged-cache operator on streams of its own: two caches served at once, with inputs made beforehand and no
wait between the calls, must end with the bits that each gets alone."""
import pytest
import torch

import rope_wavelength_sparsity_b200 as wp

from _paged import make_cache
from test_prefill_paged_gpu import CASES

pytestmark = pytest.mark.gpu


class Cache:
    """One cache with its inputs; serve(stream) makes a round of calls and returns what they gave."""

    def __init__(self, seed, D, g, page, prompt):
        gen = torch.Generator().manual_seed(seed)
        Hq, Hkv, rows, width, pages = 6, 2, 8, 40, 200
        self.win, self.D, self.page, self.prompt = wp.Window(D, 1e4, 1.0, g), D, page, prompt
        self.pools = [torch.randn((pages, page, Hkv, D), generator=gen).to(torch.bfloat16).cuda() for _ in range(4)]
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        T = 2 * prompt + 4
        qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=gen).to(torch.bfloat16).cuda()
        self.q, self.k, self.v = (t.view(T, -1, D) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
        self.pos = torch.randint(0, 5000, (3, T), generator=gen, dtype=torch.int32).cuda()
        self.pair_axes = [p % 3 for p in range(D // 2)]
        self.pos_new = self.pos[:, 2 * prompt:].contiguous()
        self.start = [t.clone() for t in [self.table, self.refs] + self.pools]
        self.move = torch.arange(4, dtype=torch.int32, device="cuda"), torch.arange(196, 200, dtype=torch.int32, device="cuda")

    def reset(self):
        for a, b in zip([self.table, self.refs] + self.pools, self.start):
            a.copy_(b)

    def calls(self, stream):
        """The round's calls, one at a time; what they returned is left in self.got."""
        n, page, kp, vp, table, refs = self.prompt, self.page, self.pools[0], self.pools[1], self.table, self.refs
        on = dict(stream=stream)
        self.got = got = []
        wp.pages_extend(table, refs, [0, 1], [0, 0], [n, n], page, **on)
        yield
        two = table[:2]
        q = wp.append_paged(self.k[:2 * n], self.v[:2 * n], kp, vp, two, [n, n], [n, n], q=self.q[:2 * n], base=1e4, **on)
        yield
        got += [q, *wp.prefill_paged(q, kp, vp, two, [n, n], [n, n], self.win, **on)]
        yield
        wp.pages_fork(self.pools, table, refs, [0, 1, 1], [4, 5, 7], [n, n, n - 3], **on)
        yield
        wp.pages_extend(table, refs, [4, 5], [n, n], [n + 1, n + 3], page, **on)
        yield
        at, mine = slice(2 * n, 2 * n + 4), table[4:6]
        q = wp.append_paged(self.k[at], self.v[at], kp, vp, mine, [1, 3], [n + 1, n + 3], q=self.q[at], base=1e4,
                            positions=self.pos_new, pair_axes=self.pair_axes, **on)
        yield
        got += [q, *wp.prefill_paged(q, kp, vp, mine, [1, 3], [n + 1, n + 3], self.win, **on)]
        yield
        wp.pages_free(table, refs, [0, 5], [n, n + 3], page, **on)
        yield
        got.append(wp.pages_compact(self.pools, table, refs, **on))
        yield
        wp.pages_copy(self.pools, *self.move, **on)
        yield
        got += wp.rope_axes(self.q, self.k, self.pos, self.pair_axes, base=1e4, inverse=True, **on)
        yield

    def state(self):
        return [t.clone() for t in self.got + [self.table, self.refs] + self.pools]


def test_two_caches_on_two_streams(cuda_dev):
    caches = [Cache(1, 64, 8, 16, 500), Cache(2, 128, 1, 32, 700)]
    want = []
    for c in caches:
        for _ in c.calls(None):
            torch.cuda.synchronize()
        want.append(c.state())
    assert wp.device_status() == wp.OK
    streams = [torch.cuda.Stream() for _ in caches]
    for _ in range(4):
        for c in caches:
            c.reset()
        torch.cuda.synchronize()
        for _ in zip(*(c.calls(s) for c, s in zip(caches, streams))):   # a call of one, a call of the other
            pass
        torch.cuda.synchronize()
        for c, w in zip(caches, want):
            assert all(torch.equal(a, b) for a, b in zip(c.state(), w))
    assert wp.device_status() == wp.OK


def test_prefills_side_by_side(cuda_dev):
    """Split key ranges on three streams at once, several calls each, all queued before the first is waited for."""
    cases = [CASES[n] for n in ("mixed_batch", "long_context_chunk", "long_context")]
    jobs = []
    for i, (D, g, alpha, base, Hq, Hkv, page, q_len, kv_len) in enumerate(cases):
        kp, vp, table, _, _ = make_cache(kv_len, page, Hkv, D, i)
        q = torch.randn((sum(q_len), Hq, D), generator=torch.Generator().manual_seed(9 + i)).to(torch.bfloat16).cuda()
        jobs.append((q, kp, vp, table, q_len, kv_len, wp.Window(D, base, alpha, g)))
    want = [wp.prefill_paged(*j) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = [[wp.prefill_paged(*j, stream=s) for j, s in zip(jobs, streams)] for _ in range(12)]
    torch.cuda.synchronize()
    assert wp.device_status() == wp.OK
    for turn in got:
        for (a, b), (x, y) in zip(want, turn):
            assert torch.equal(a, x) and torch.equal(b, y)
