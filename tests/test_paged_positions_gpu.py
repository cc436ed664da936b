"""Caches whose keys were rotated by positions of their own: prefill_paged (and decode_paged without positions) prunes
by the distance of cache rows whatever turned the keys; decode_paged with q_pos and k_pos by the distance of those."""
import math

import pytest
import torch

import oracle
import rope_wavelength_sparsity_b200 as wp

from _paged import attention64, check_attention, pages_of

pytestmark = pytest.mark.gpu


def _case(D, Hq, Hkv, page, new, seed=0):
    """An empty cache, its table, and the new tokens of each sequence with time, height and width of frames 6 x 6."""
    gen = torch.Generator().manual_seed(seed)
    T, need = sum(new), [pages_of(n, page) for n in new]
    table = torch.full((len(new), max(need)), -1, dtype=torch.int32)
    ids = torch.randperm(sum(need) + 2, generator=gen).to(torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = ids[sum(need[:b]):sum(need[:b]) + n]
    pools = [torch.full((sum(need) + 2, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q, k, v = (torch.randn((T, h, D), generator=gen).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
    row = torch.cat([torch.arange(n) for n in new])
    pos = torch.stack([row // 36, row // 6 % 6, row % 6]).to(torch.int32).cuda()
    return q, k, v, *pools, table.cuda(), pos


@pytest.mark.parametrize("D,g", [(64, 8), (128, 1)])
def test_chunk_after_an_append_on_three_axes(cuda_dev, D, g):
    Hq, Hkv, page, base, alpha, new = 6, 2, 16, 1e4, 1.0, [200, 77, 1]
    q, k, v, kp, vp, table, pos = _case(D, Hq, Hkv, page, new)
    pair_axes = [p % 3 for p in range(D // 2)]
    qr, kr = wp.rope_axes(q, k, pos, pair_axes, base=base)
    got = wp.append_paged(k, v, kp, vp, table, new, new, q=q, base=base, positions=pos, pair_axes=pair_axes)
    assert torch.equal(got, qr)
    win = wp.Window(D, base, alpha, g)
    out, lse = wp.prefill_paged(got, kp, vp, table, new, new, win)
    # the definition: turned queries and keys, distances of rows (so the time axis, a step per 36 rows, is
    # left out after a 36th of its pairs' wavelengths)
    ref = attention64(qr, list(kr.cpu().split(new)), list(v.cpu().split(new)), new, new, Hq, Hkv, D, base, alpha, g)
    check_attention(out, lse, ref, D, max(new), "chunk")
    # single tokens of the same cache, without positions: the same rule
    last = torch.tensor(new, device="cuda").cumsum(0) - 1
    dec, dl = wp.decode_paged(qr[last].contiguous(), kp, vp, table, new, win)
    one = [x[last] for x in ref]
    check_attention(dec, dl, one, D, max(new), "decode")
    # with alpha = inf no distance matters, and the chunk attends what any positions mean
    off = wp.Window(D, base, math.inf, g)
    out, lse = wp.prefill_paged(got, kp, vp, table, new, new, off)
    ref = attention64(qr, list(kr.cpu().split(new)), list(v.cpu().split(new)), new, new, Hq, Hkv, D, base, math.inf, g)
    check_attention(out, lse, ref, D, max(new), "no window")


@pytest.mark.parametrize("D,g", [(64, 8), (128, 1)])
def test_decode_by_given_positions_after_an_append(cuda_dev, D, g):
    """Positions of 36 rows each: the decode by them keeps pairs that the distance of rows leaves out."""
    Hq, Hkv, page, base, alpha, new = 6, 2, 16, 1e4, 0.25, [200, 77, 37]
    q, k, v, kp, vp, table, pos = _case(D, Hq, Hkv, page, new, 1)
    time = pos[0].contiguous()
    qr = wp.append_paged(k, v, kp, vp, table, new, new, q=q, base=base, positions=time)
    _, kr = wp.rope_axes(q, k, time, base=base)
    last = torch.tensor(new, device="cuda").cumsum(0) - 1
    kpos = torch.zeros((len(new), max(new)), dtype=torch.int32, device="cuda")
    for b, t in enumerate(time.split(new)):
        kpos[b, :new[b]] = t
    one, win = qr[last].contiguous(), wp.Window(D, base, alpha, g)
    dec, dl = wp.decode_paged(one, kp, vp, table, new, win, q_pos=time[last].tolist(), k_pos=kpos)
    assert wp.device_status() == wp.OK
    T = torch.as_tensor(oracle.thresholds(D, base, alpha, g)[0].astype("int64")).cuda()
    P, G = D // 2, Hq // Hkv
    ref = [torch.zeros((len(new), Hq, D), dtype=torch.float64, device="cuda"), None,
           torch.zeros((len(new), Hq, D), dtype=torch.float64, device="cuda"), None]
    ref[1], ref[3] = (torch.zeros((len(new), Hq), dtype=torch.float64, device="cuda") for _ in range(2))
    for b, (kb, vb) in enumerate(zip(kr.double().split(new), v.double().split(new))):
        d = time[last[b]] - kpos[b, :new[b]]
        keep = (d[:, None] <= T).double()
        for h in range(Hq):
            x, y = one[b, h].double(), kb[:, h // G]
            term = x[:P] * y[:, :P] + x[P:] * y[:, P:]
            size = x[:P].abs() * y[:, :P].abs() + x[P:].abs() * y[:, P:].abs()
            s = (term * keep).sum(1) / math.sqrt(D)
            ref[1][b, h] = torch.logsumexp(s, 0)
            w = torch.softmax(s, 0)
            ref[0][b, h], ref[2][b, h] = w @ vb[:, h // G], w @ vb[:, h // G].abs()
            ref[3][b, h] = size.sum(1).amax() / math.sqrt(D)
    check_attention(dec, dl, ref, D, max(new), "by positions")
    rows, rl = wp.decode_paged(one, kp, vp, table, new, win)
    assert not torch.equal(rl, dl)               # the two rules differ here


@pytest.mark.parametrize("given", [False, True])
def test_append_turns_keys_without_queries(cuda_dev, given):
    D, Hq, Hkv, page, new = 128, 4, 2, 32, [65, 3, 31]
    q, k, v, kp, vp, table, pos = _case(D, Hq, Hkv, page, new, 2)
    kw = dict(positions=pos, pair_axes=[p % 3 for p in range(D // 2)]) if given else {}
    a, b = kp.clone(), vp.clone()
    assert wp.append_paged(k, v, kp, vp, table, new, new, base=5e5, **kw) is None
    qo = wp.append_paged(k, v, a, b, table, new, new, q=q, base=5e5, **kw)
    row = torch.cat([torch.arange(n) for n in new]).to(torch.int32).cuda()
    at = (pos, kw["pair_axes"]) if given else (row, None)
    want = wp.rope_axes(q, k, *at, base=5e5)
    assert torch.equal(qo, want[0])
    for x, y in ((kp, a), (vp, b)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    seq = torch.cat([torch.full((n,), i) for i, n in enumerate(new)]).cuda()
    slot = table[seq, (row // page).long()].long() * page + row % page
    assert torch.equal(kp.view(-1, Hkv, D)[slot], want[1]) and torch.equal(vp.view(-1, Hkv, D)[slot], v)
    assert wp.device_status() == wp.OK
