"""Shared by the paged-cache tests: caches with scattered pages, and attention in 64 bits."""
import math

import torch

import oracle

BF16 = torch.finfo(torch.bfloat16).eps / 2   # a rounding to bf16, relative
F32 = torch.finfo(torch.float32).eps / 2


def pages_of(n, page):
    return -(-n // page)


def make_cache(kv_len, page, Hkv, D, seed, spare=3, fill=float("nan"), max_pages=None):
    """(k_pages, v_pages, table, k, v): pools with every sequence's rows on scattered pages and
    `fill` wherever no sequence has a row; k, v: the sequences' rows, one tensor each."""
    gen = torch.Generator().manual_seed(seed)
    need = [pages_of(n, page) for n in kv_len]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=gen).tolist()
    pools = [torch.full((total, page, Hkv, D), fill, dtype=torch.bfloat16) for _ in range(2)]
    table = torch.full((len(kv_len), max_pages or max(max(need), 1)), -7, dtype=torch.int32)
    rows, at = ([], []), 0
    for b, n in enumerate(kv_len):
        ids = perm[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = torch.tensor(ids, dtype=torch.int32)
        for pool, kept in zip(pools, rows):
            x = torch.randn((n, Hkv, D), generator=gen).to(torch.bfloat16)
            kept.append(x)
            for i, pg in enumerate(ids):
                part = x[i * page:(i + 1) * page]
                pool[pg, :len(part)] = part
    return pools[0].cuda(), pools[1].cuda(), table.cuda(), rows[0], rows[1]


def attention64(q, k, v, q_len, kv_len, Hq, Hkv, D, base, alpha, g, scale=None):
    """(out, lse, spread, reach) of every row of q [T, Hq, D] in 64 bits: spread = sum of weight
    times |v|, reach = the row's largest sum of |q k| terms times the scale."""
    scale = 1 / math.sqrt(D) if scale is None else scale
    T = torch.as_tensor(oracle.thresholds(D, base, alpha, g)[0].astype("int64")).cuda()
    P, G = D // 2, Hq // Hkv
    total = sum(q_len)
    out = torch.zeros((total, Hq, D), dtype=torch.float64, device="cuda")
    spread, reach = torch.zeros_like(out), torch.zeros((total, Hq), dtype=torch.float64, device="cuda")
    lse = torch.full((total, Hq), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, L) in enumerate(zip(q_len, kv_len)):
        if n and L:
            kb, vb = k[b].cuda().double(), v[b].cuda().double()
            qb = q[at:at + n].cuda().double()
            d = (torch.arange(L - n, L, device="cuda")[:, None] - torch.arange(L, device="cuda")[None])
            for h in range(Hq):
                qh, kh = qb[:, h], kb[:, h // G]
                s = torch.zeros((n, L), dtype=torch.float64, device="cuda")
                r = torch.zeros_like(s)
                for p in range(P):
                    term = qh[:, [p, p + P]] @ kh[:, [p, p + P]].T
                    s += torch.where(d <= T[p], term, 0.0)
                    r += qh[:, [p, p + P]].abs() @ kh[:, [p, p + P]].abs().T
                s = torch.where(d >= 0, s * scale, -math.inf)
                z = torch.logsumexp(s, -1)
                w = torch.where(torch.isfinite(z)[:, None], torch.exp(s - z[:, None]), 0.0)
                out[at:at + n, h] = w @ vb[:, h // G]
                spread[at:at + n, h] = w @ vb[:, h // G].abs()
                reach[at:at + n, h] = torch.where(d >= 0, r * scale, 0.0).amax(-1)
                lse[at:at + n, h] = z
        at += n
    return out, lse, spread, reach


def check_attention(out, lse, ref, D, longest, what=""):
    """Against attention64.  The scores are fp32 sums of at most 3 D terms (the contraction and
    its corrections), each addition off by F32 of sums no larger than reach; the exponentials and
    the logarithm (ex2 and lg2 approximations, 2^-22 of their result or of one) and a sum of
    `longest` weights come on top; weights and the result are rounded to bf16 once each."""
    o64, l64, spread, reach = ref
    out, lse = out[:len(o64)].double(), lse[:len(l64)].double()
    none = torch.isneginf(l64)
    assert torch.equal(torch.isneginf(lse), none), f"{what}: rows without keys differ"
    assert (out[none] == 0).all(), f"{what}: a row without keys is not 0"
    score = 3 * D * F32 * reach
    tol_l = score + 2.0 ** -20 + longest * F32 + 2 * F32 * l64.abs()
    err_l = torch.where(none, 0.0, (lse - l64).abs())
    assert not torch.isnan(err_l).any() and (err_l <= torch.where(none, 1.0, tol_l)).all(), \
        f"{what}: lse off by {float(err_l.max()):.3e}, allowed {float(tol_l[~none].min()):.3e}"
    tol_o = BF16 * (spread + o64.abs()) + 2 * torch.where(none, 0.0, tol_l)[..., None] * spread + 1e-30
    err_o = (out - o64).abs()
    assert not torch.isnan(err_o).any() and (err_o <= tol_o).all(), \
        f"{what}: out off by up to {float((err_o / tol_o).max()):.2f} of what is allowed"
