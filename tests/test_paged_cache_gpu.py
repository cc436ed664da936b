"""RoPE along several axes, the append to a paged cache and page maintenance; then all of them
together as serving steps."""
import math

import numpy as np
import pytest
import torch

import oracle
import rope_wavelength_sparsity_b200 as wp
from rope_wavelength_sparsity_b200 import inputs

from _paged import BF16, F32, attention64, check_attention, make_cache, pages_of

pytestmark = pytest.mark.gpu


def _rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def _turned64(x, pos, axes, base, sign=1.0):
    """x [T, H, D] turned in 64 bits by pos [axes, T]."""
    D = x.shape[-1]
    P = D // 2
    theta = torch.tensor([base ** (-2 * p / D) for p in range(P)], dtype=torch.float64, device=x.device)
    at = pos.double()[torch.tensor(axes, device=x.device)].T * theta * sign
    c, s = at.cos()[:, None], at.sin()[:, None]
    lo, hi = x[..., :P].double(), x[..., P:].double()
    return torch.cat([lo * c - hi * s, lo * s + hi * c], -1)


def _check_turn(got, x, pos, axes, base, sign=1.0):
    """One rounding to bf16 of a value off by the float rotation: the reduced angle, its cosine
    and sine and two products are each within a few F32 of the pair's size."""
    P = x.shape[-1] // 2
    want = _turned64(x, pos, axes, base, sign)
    size = x[..., :P].double().abs() + x[..., P:].double().abs()
    tol = BF16 * want.abs() + 8 * F32 * (1 + BF16) * torch.cat([size, size], -1) + 1e-38
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("D,T,Hq,Hkv,axes", [(64, 1, 1, 1, 1), (128, 3, 5, 1, 2), (128, 700, 28, 4, 3), (64, 333, 14, 2, 4),
                                             (128, 40000, 2, 1, 3)])
def test_rope_axes(cuda_dev, D, T, Hq, Hkv, axes, inverse):
    q, k = _rand((T, Hq, D), 1), _rand((T, Hkv, D), 2)
    gen = torch.Generator().manual_seed(3)
    pos = torch.randint(0, 1 << 20, (axes, T), generator=gen, dtype=torch.int32)
    pos[0, 0], pos[-1, -1] = 0, 2**31 - 1
    pos = pos.cuda()
    pair_axes = torch.randint(0, axes, (D // 2,), generator=gen).tolist()
    qo, ko = wp.rope_axes(q, k, pos, pair_axes, base=1e6, inverse=inverse)
    for got, x in ((qo, q), (ko, k)):
        _check_turn(got, x, pos, pair_axes, 1e6, -1.0 if inverse else 1.0)


def test_rope_axes_one_axis_is_rope(cuda_dev):
    q, k = _rand((90, 6, 128), 1), _rand((90, 2, 128), 2)
    pos = torch.randint(0, 100000, (1, 90), dtype=torch.int32).cuda()
    qo, ko = wp.rope_axes(q, k, pos, base=5e5)
    assert torch.equal(qo, wp.rope(q[None], base=5e5, positions=pos)[0])
    assert torch.equal(ko, wp.rope(k[None], base=5e5, positions=pos)[0])
    same = wp.rope_axes(q, k, pos.repeat(3, 1), [p % 3 for p in range(64)], base=5e5)
    assert torch.equal(qo, same[0]) and torch.equal(ko, same[1])
    only, none = wp.rope_axes(q, None, pos[0], base=5e5)
    assert none is None and torch.equal(only, qo)


def test_rope_axes_strided_in_place_and_empty(cuda_dev):
    D, Hq, Hkv, T = 64, 4, 2, 77
    qkv = _rand((T, (Hq + 2 * Hkv) * D), 5)
    q, k = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    pos = torch.arange(2 * T, dtype=torch.int32, device="cuda").view(2, T)
    axes = [p % 2 for p in range(32)]
    want = wp.rope_axes(q.contiguous(), k.contiguous(), pos, axes, base=1e4)
    got = wp.rope_axes(q, k, pos, axes, base=1e4)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a, b = q.contiguous(), k.contiguous()
    wp.rope_axes(a, b, pos, axes, base=1e4, q_out=a, k_out=b)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    e = wp.rope_axes(q[:0], k[:0], pos, axes, base=1e4)
    assert e[0].shape == (0, Hq, D) and e[1].shape == (0, Hkv, D)


def test_rope_axes_inverse_is_the_gradient(cuda_dev):
    """<g, R x> = <R^T g, x>, and against differences: R is linear, so a difference in any direction
    is R of that direction."""
    T, H, D = 50, 3, 64
    x, g = _rand((T, H, D), 1), _rand((T, H, D), 2)
    pos = torch.randint(0, 5000, (3, T), dtype=torch.int32).cuda()
    axes = [p % 3 for p in range(32)]
    y = wp.rope_axes(x, None, pos, axes, base=1e4)[0].double()
    gx = wp.rope_axes(g, None, pos, axes, base=1e4, inverse=True)[0].double()
    left, right = (g.double() * y).sum((1, 2)), (gx * x.double()).sum((1, 2))
    tol = 2 * (BF16 + 8 * F32) * 2 * (g.double().square().sum((1, 2)) * x.double().square().sum((1, 2))).sqrt()
    assert ((left - right).abs() <= tol).all()
    step = 0.5                                   # exact in bf16 on unit directions
    for e in (0, 5, 31, 32, 63):
        d = torch.zeros_like(x)
        d[..., e] = step
        col = _turned64(d, pos, axes, 1e4) / step
        want = (col * g.double()).sum(-1)
        P, p = D // 2, e % (D // 2)
        size = g[..., p].double().abs() + g[..., p + P].double().abs()
        assert ((gx[..., e] - want).abs() <= BF16 * want.abs() + 8 * F32 * size + 1e-38).all()


APPEND = {
    # D, Hq, Hkv, page, new_len, kv_len, axes
    "one_token": (64, 2, 1, 8, [1], [1], 1),
    "single_tokens": (128, 24, 8, 16, [1] * 5, [1, 16, 17, 500, 333], 1),
    "chunks": (128, 28, 4, 64, [300, 0, 7, 64], [300, 90, 100, 128], 3),
    "odd_pages": (64, 14, 2, 96, [95, 97, 1], [95, 200, 97], 2),
    "many": (64, 3, 3, 16, [1 + i % 3 for i in range(200)], [5 + 7 * i for i in range(200)], 1),
}


@pytest.mark.parametrize("rotated", [True, False])
@pytest.mark.parametrize("name", APPEND)
def test_append(cuda_dev, name, rotated):
    D, Hq, Hkv, page, new, kv, axes = APPEND[name]
    kp, vp, table, _, _ = make_cache(kv, page, Hkv, D, 1, fill=3.0)
    k0, v0 = kp.clone(), vp.clone()
    T = sum(new)
    qkv = _rand((T + 2, (Hq + 2 * Hkv) * D), 2)   # two rows behind the last sequence
    q, k, v = (t.view(T + 2, -1, D) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    row = torch.tensor([m - n + t for n, m in zip(new, kv) for t in range(n)], dtype=torch.int32).cuda()
    if not rotated:
        assert wp.append_paged(k, v, kp, vp, table, new, kv) is None
    elif axes == 1:
        pos, pa = row[None], [0] * (D // 2)
        qo = wp.append_paged(k, v, kp, vp, table, new, kv, q=q, base=5e5)
    else:
        pos = torch.randint(0, 9999, (axes, T), dtype=torch.int32).cuda()
        pa = [p % axes for p in range(D // 2)]
        out = torch.full((T + 2, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
        qo = wp.append_paged(k, v, kp, vp, table, new, kv, q=q, base=5e5, positions=pos, pair_axes=pa, q_out=out)
        assert qo is out and (out[T:] == 5).all()
    assert wp.device_status() == wp.OK
    seq = torch.tensor([b for b, n in enumerate(new) for _ in range(n)]).cuda()
    slot = table[seq, (row // page).long()].long() * page + row % page
    want_k = k[:T]
    if rotated:
        _check_turn(qo[:T], q[:T], pos, pa, 5e5)
        _check_turn(kp.view(-1, Hkv, D)[slot], k[:T], pos, pa, 5e5)
        want_k = kp.view(-1, Hkv, D)[slot]
    k0.view(-1, Hkv, D)[slot], v0.view(-1, Hkv, D)[slot] = want_k, v[:T]
    assert torch.equal(kp, k0) and torch.equal(vp, v0)   # and nothing else


def test_append_bad_page(cuda_dev):
    kp = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.tensor([[2, -1], [1, 4]], dtype=torch.int32, device="cuda")
    k, v = _rand((6, 2, 64), 1), _rand((6, 2, 64), 2)
    wp.append_paged(k, v, kp, vp, table, [3, 3], [18, 18])
    assert wp.device_status() == wp.EINDEX
    assert torch.equal(kp[2, 15], k[0]) and torch.equal(vp[1, 15], v[3])
    kp[2, 15], kp[1, 15], vp[2, 15], vp[1, 15] = 0, 0, 0, 0
    assert not kp.any() and not vp.any()


# ------------------------------------------------------------------ pages, against the same on the host
class Host:
    """Pages, table and refs on the host, with the rules written out."""

    def __init__(self, pools, table, refs, page):
        self.pools, self.page = [p.cpu().clone() for p in pools], page
        self.table, self.refs = table.cpu().clone(), refs.cpu().clone()

    def free_pages(self, n):
        return (self.refs == 0).nonzero()[:n, 0].tolist()

    def fork(self, src, dst, lens):
        begun = [i for i, n in enumerate(lens) if n % self.page]
        fresh = dict(zip(begun, self.free_pages(len(begun))))
        for i, (s, d, n) in enumerate(zip(src, dst, lens)):
            full = n // self.page
            self.table[d] = -1
            self.table[d, :full] = self.table[s, :full]
            for e in self.table[d, :full].tolist():
                self.refs[e] += 1
            if n % self.page and i in fresh:
                self.table[d, full] = fresh[i]
                self.refs[fresh[i]] = 1
                for p in self.pools:
                    p[fresh[i], :n % self.page] = p[self.table[s, full], :n % self.page]

    def free(self, rows, lens):
        for r, n in zip(rows, lens):
            for j in range(pages_of(n, self.page)):
                self.refs[self.table[r, j]] -= 1
                self.table[r, j] = -1

    def extend(self, rows, lens, new):
        want = [(r, j) for r, a, b in zip(rows, lens, new) for j in range(pages_of(a, self.page), pages_of(b, self.page))]
        free = self.free_pages(len(want))
        for (r, j), pg in zip(want, free + [-1] * len(want)):
            self.table[r, j] = pg
            if pg >= 0:
                self.refs[pg] = 1

    def compact(self):
        live = int((self.refs > 0).sum())
        holes = [i for i in range(live) if self.refs[i] == 0]
        late = [i for i in range(live, len(self.refs)) if self.refs[i] > 0]
        to = dict(zip(late, holes))
        for a, b in to.items():
            for p in self.pools:
                p[b] = p[a]
            self.refs[b], self.refs[a] = self.refs[a].item(), 0
        self.table = torch.tensor([[to.get(e, e) for e in r] for r in self.table.tolist()], dtype=torch.int32)
        return live

    def check(self, pools, table, refs):
        assert torch.equal(table.cpu(), self.table) and torch.equal(refs.cpu(), self.refs)
        for a, b in zip(pools, self.pools):
            assert torch.equal(a.cpu(), b)


def _cache(page, Hkv, D, pools, num_pages, rows, max_pages, seed=0):
    made = [_rand((num_pages, page, Hkv, D), seed + i) for i in range(pools)]
    table = torch.full((rows, max_pages), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    return made, table, refs, Host(made, table, refs, page)


@pytest.mark.parametrize("page,Hkv,D,pools,num_pages", [(8, 1, 64, 1, 70), (16, 8, 128, 2, 400), (96, 3, 64, 6, 2500)])
def test_page_life(cuda_dev, page, Hkv, D, pools, num_pages):
    made, table, refs, host = _cache(page, Hkv, D, pools, num_pages, 12, 16)
    lens = [page * 3 + 1, 5, 0, page * 2, page]

    def same():
        assert wp.device_status() == wp.OK
        host.check(made, table, refs)

    rows = [0, 2, 4, 6, 8]
    wp.pages_extend(table, refs, rows, [0] * 5, lens, page)
    host.extend(rows, [0] * 5, lens)
    same()
    src, dst = [0, 0, 2, 6, 4, 8], [1, 11, 3, 7, 5, 9]
    ln = [lens[0], lens[0] - 2, 5, page * 2, 0, page]
    wp.pages_fork(made, table, refs, src, dst, ln)
    host.fork(src, dst, ln)
    same()
    gone, glen = [0, 2, 8, 4], [lens[0], 5, page, 0]
    wp.pages_free(table, refs, gone, glen, page)
    host.free(gone, glen)
    same()
    wp.pages_extend(table, refs, [1, 3, 6], [lens[0], 5, page * 2], [lens[0] + 2 * page, 5 + page, page * 2 + 1], page)
    host.extend([1, 3, 6], [lens[0], 5, page * 2], [lens[0] + 2 * page, 5 + page, page * 2 + 1])
    same()
    live = wp.pages_compact(made, table, refs)
    assert int(live) == host.compact()
    same()
    assert int(wp.pages_compact(made, table, refs)) == int(live)   # nothing left to move
    same()


@pytest.mark.parametrize("num_pages", [1, 31, 1024, 1025, 5000])
@pytest.mark.parametrize("used", [0.0, 0.3, 0.97, 1.0])
def test_compact_any_pool(cuda_dev, num_pages, used):
    made, table, refs, _ = _cache(8, 1, 64, 2, num_pages, 7, -(-num_pages // 7) + 1, seed=num_pages)
    gen = torch.Generator().manual_seed(num_pages)
    ids = torch.randperm(num_pages, generator=gen)[:int(round(used * num_pages))].to(torch.int32)
    table.view(-1)[:len(ids)] = ids.cuda()
    refs[ids.long().cuda()] = 1
    if len(ids) > 2:                              # a shared page
        table[6, -1] = int(ids[1])
        refs[int(ids[1])] += 1
    host = Host(made, table, refs, 8)
    assert int(wp.pages_compact(made, table, refs)) == host.compact()
    host.check(made, table, refs)
    assert wp.device_status() == wp.OK


def test_a_thousand_rows(cuda_dev):
    """As many rows as a call takes: grown, forked (many from one source), freed again."""
    page, rows = 8, 1034
    made, table, refs, host = _cache(page, 1, 64, 2, 3000, rows, 4)
    src_len = [1 + 3 * i for i in range(10)]
    wp.pages_extend(table, refs, range(10), [0] * 10, src_len, page)
    host.extend(range(10), [0] * 10, src_len)
    dst = list(range(10, rows))
    src = [i * i % 10 for i in range(1024)]
    ln = [src_len[r] - i % 2 for i, r in enumerate(src)]
    wp.pages_fork(made, table, refs, src, dst, ln)
    host.fork(src, dst, ln)
    host.check(made, table, refs)
    new = [n + i % 5 for i, n in enumerate(ln)]
    wp.pages_extend(table, refs, dst, ln, new, page)
    host.extend(dst, ln, new)
    host.check(made, table, refs)
    wp.pages_free(table, refs, dst, new, page)
    host.free(dst, new)
    host.check(made, table, refs)
    assert wp.device_status() == wp.OK and int(refs.sum()) == sum(pages_of(n, page) for n in src_len)


def test_too_few_pages(cuda_dev):
    made, table, refs, host = _cache(8, 1, 64, 2, 5, 6, 4)
    wp.pages_extend(table, refs, [0, 1], [0, 0], [20, 9], 8)      # 3 + 2 of 5 pages
    host.extend([0, 1], [0, 0], [20, 9])
    assert wp.device_status() == wp.OK
    wp.pages_extend(table, refs, [1, 2], [9, 0], [17, 8], 8)
    host.extend([1, 2], [9, 0], [17, 8])
    assert wp.device_status() == wp.EPAGES
    host.check(made, table, refs)
    wp.pages_free(table, refs, [1], [9], 8)
    host.free([1], [9])
    assert wp.device_status() == wp.OK
    wp.pages_fork(made, table, refs, [0, 0, 0], [3, 4, 5], [20, 20, 20])  # 2 pages for 3 begun ones
    host.fork([0, 0, 0], [3, 4, 5], [20, 20, 20])
    assert wp.device_status() == wp.EPAGES
    host.check(made, table, refs)


def test_bad_entries_are_reported(cuda_dev):
    made, table, refs, _ = _cache(8, 1, 64, 1, 6, 4, 3)
    before = made[0].clone()
    table[0] = torch.tensor([5, 6, -1], dtype=torch.int32)
    refs[5] = 1
    wp.pages_fork(made, table, refs, [0], [1], [17])               # entries 6 and -1 are outside
    assert wp.device_status() == wp.EINDEX and torch.equal(made[0], before)
    wp.pages_free(table, refs, [0], [24], 8)
    assert wp.device_status() == wp.EINDEX and refs.tolist()[5] == 1
    table[2, 0] = 3                                                # a page that is free
    wp.pages_free(table, refs, [2], [8], 8)
    assert wp.device_status() == wp.EINDEX and refs.tolist()[3] == 0
    src = torch.tensor([0, 6, 1], dtype=torch.int32, device="cuda")
    dst = torch.tensor([2, 3, -1], dtype=torch.int32, device="cuda")
    wp.pages_copy(made, src, dst)
    assert wp.device_status() == wp.EINDEX
    before[2] = before[0]
    assert torch.equal(made[0], before)


@pytest.mark.parametrize("n,pools", [(1, 1), (300, 3), (5, 12)])
def test_copy(cuda_dev, n, pools):
    made = [_rand((2 * n + 1, 16, 2, 64), i) for i in range(pools)]
    perm = torch.randperm(2 * n + 1, generator=torch.Generator().manual_seed(n)).to(torch.int32).cuda()
    want = [p.clone() for p in made]
    for p in want:
        p[perm[n:2 * n].long()] = p[perm[:n].long()]
    wp.pages_copy(made, perm[:n].contiguous(), perm[n:2 * n].contiguous())
    assert wp.device_status() == wp.OK
    assert all(torch.equal(a, b) for a, b in zip(made, want))


def test_pages_captured_and_replayed(cuda_dev):
    made, table, refs, host = _cache(16, 2, 64, 2, 60, 8, 6)
    wp.pages_extend(table, refs, [0, 1], [0, 0], [50, 33], 16)
    wp.pages_free(table, refs, [0], [50], 16)
    torch.cuda.synchronize()
    host = Host(made, table, refs, 16)
    t0, r0, p0 = table.clone(), refs.clone(), [p.clone() for p in made]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wp.pages_fork(made, table, refs, [1, 1], [2, 5], [33, 20])
        wp.pages_extend(table, refs, [2], [33], [70], 16)
        wp.pages_free(table, refs, [1], [33], 16)
        live = wp.pages_compact(made, table, refs)
    host.fork([1, 1], [2, 5], [33, 20])
    host.extend([2], [33], [70])
    host.free([1], [33])
    n = host.compact()
    for _ in range(2):
        for a, b in [(table, t0), (refs, r0)] + list(zip(made, p0)):
            a.copy_(b)
        graph.replay()
        assert int(live) == n
        host.check(made, table, refs)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("D,g,alpha,page", [(64, 8, 1.0, 16), (128, 1, 1.0, 32)])
def test_serving_steps(cuda_dev, D, g, alpha, page):
    """Prompts in chunks, a fork, drafts and single tokens, a sequence that leaves, a compaction: what
    each step attends must be what the sequences' own rows say."""
    Hq, Hkv, base = 6, 2, 1e4
    win = wp.Window(D, base, alpha, g)
    made, table, refs, _ = _cache(page, Hkv, D, 2, 120, 6, 40)
    for p in made:
        p.fill_(float("nan"))                     # nothing may come from rows that no one wrote
    kp, vp = made
    seqs = {}                                     # row -> (rotated keys, values), as they were stored
    gen = torch.Generator().manual_seed(5)

    def step(rows, new):
        lens = [len(seqs[r][0]) if r in seqs else 0 for r in rows]
        kv = [a + b for a, b in zip(lens, new)]
        wp.pages_extend(table, refs, rows, lens, kv, page)
        qkv = torch.randn((sum(new), (Hq + 2 * Hkv) * D), generator=gen).to(torch.bfloat16).cuda()
        q, k, v = (t.view(sum(new), -1, D) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
        mine = table[torch.tensor(rows, device="cuda")].contiguous()
        qr = wp.append_paged(k, v, kp, vp, mine, new, kv, q=q, base=base)
        out, lse = wp.prefill_paged(qr, kp, vp, mine, new, kv, win)
        assert wp.device_status() == wp.OK
        pos = torch.tensor([a + t for a, n in zip(lens, new) for t in range(n)], dtype=torch.int32).cuda()
        _, kr = wp.rope_axes(q, k, pos, base=base)
        at = 0
        for r, n in zip(rows, new):
            old = seqs.get(r, (kr[:0].cpu(), v[:0].cpu()))
            seqs[r] = (torch.cat([old[0], kr[at:at + n].cpu()]), torch.cat([old[1], v[at:at + n].cpu()]))
            at += n
        ref = attention64(qr, [seqs[r][0] for r in rows], [seqs[r][1] for r in rows], new, kv, Hq, Hkv, D, base, alpha, g)
        check_attention(out, lse, ref, D, max(kv))
        if all(n == 1 for n in new):
            dec, dl = wp.decode_paged(qr, kp, vp, mine, kv, win)
            check_attention(dec, dl, ref, D, max(kv))

    step([0, 3], [300, 45])
    step([0, 3], [129, 1])
    n = len(seqs[0][0])
    wp.pages_fork(made, table, refs, [0, 3], [1, 4], [n, len(seqs[3][0])])
    seqs[1], seqs[4] = seqs[0], seqs[3]
    step([0, 1, 3, 4], [3, 5, 1, 2])              # the forks part ways
    wp.pages_free(table, refs, [0], [len(seqs[0][0])], page)
    del seqs[0]
    live = int(wp.pages_compact(made, table, refs))
    assert live == int((refs > 0).sum()) and not refs[live:].any()
    step([1, 3, 4], [1, 1, 1])
    step([1, 2, 4], [1, 60, 17])
