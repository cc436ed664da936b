"""Cases of the paged-serving operators: what a serving step does with a paged KV cache.

Operators (each with a plain form in elementary torch operations and, where ``own`` is
true, the library's calls):

- ``prefill_paged``: windowed attention of a ragged batch of chunks over a paged cache;
- ``append_paged``: the step's new keys and values rotated and written into the pages,
  its queries rotated, in one call;
- ``rope_axes``: RoPE with positions along several axes (time, height, width);
- ``fork`` and ``compact``: page maintenance, as a beam-search step (fork the survivors,
  free their parents) and a defragmentation of the pools.

Lengths of ragged cases come from the case's own ``lens`` number, values from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # drafts checked by the model: up to 8 new tokens in each of a few sequences
        dict(name="chunk drafts", op="prefill_paged", D=128, Hq=24, Hkv=8, base=5e5, alpha=1.0, g=1,
             page=16, ones=2, chunks=6, q_min=2, q_max=8, ctx_min=700, ctx_max=4000, lens=1),
        # a serving step that mixes single tokens with chunks of prompts
        dict(name="chunk mixed step", op="prefill_paged", D=64, Hq=14, Hkv=2, base=1e6, alpha=1.0, g=8,
             page=16, ones=20, chunks=4, q_min=200, q_max=700, ctx_min=500, ctx_max=9000, lens=2),
        # one chunk of a long prompt, every pair with its own window
        dict(name="chunk 2048 at 32K", op="prefill_paged", D=128, Hq=24, Hkv=8, base=5e5, alpha=1.0, g=1,
             page=64, ones=0, chunks=1, q_min=2048, q_max=2048, ctx_min=30720, ctx_max=30720, lens=3),
        # the largest: one chunk far into a 128K context
        dict(name="chunk 4096 at 128K", op="prefill_paged", D=128, Hq=28, Hkv=4, base=1e7, alpha=1.0, g=8,
             page=128, ones=0, chunks=1, q_min=4096, q_max=4096, ctx_min=126976, ctx_max=126976, lens=4),
        # one token of each of 64 sequences, rotated and stored
        dict(name="append one token", op="append_paged", D=128, Hq=24, Hkv=8, base=5e5, page=16, axes=1,
             ones=64, chunks=0, q_min=1, q_max=1, ctx_min=100, ctx_max=6000, lens=5),
        # chunks of prompts with image tokens (three position axes)
        dict(name="append chunks", op="append_paged", D=128, Hq=28, Hkv=4, base=1e6, page=64, axes=3,
             ones=7, chunks=5, q_min=900, q_max=2300, ctx_min=0, ctx_max=9000, lens=6),
        # one image's tokens
        dict(name="axes one image", op="rope_axes", D=128, Hq=28, Hkv=4, base=1e6, axes=3, tokens=1297,
             inverse=False),
        # the gradient's direction over a long video
        dict(name="axes video inverse", op="rope_axes", D=64, Hq=14, Hkv=2, base=1e6, axes=3, tokens=65000,
             inverse=True),
        # a beam-search step of a few beams
        dict(name="fork beams", op="fork", D=128, Hkv=8, page=16, pools=2, rows=8, forks=8, ctx_min=150,
             ctx_max=1200, lens=7),
        # many samples of shared prompts, two layers' pools at once
        dict(name="fork samples", op="fork", D=128, Hkv=8, page=64, pools=4, rows=48, forks=200,
             ctx_min=900, ctx_max=4000, lens=8),
        # a small pool with holes
        dict(name="compact small", op="compact", D=64, Hkv=2, page=16, pools=2, pages=1000, live=0.5,
             rows=24),
        # a large pool after many sequences have left
        dict(name="compact large", op="compact", D=128, Hkv=8, page=32, pools=4, pages=8192, live=0.6,
             rows=96),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill_paged", "prefill_paged", "prefill_paged", "append_paged", "rope_axes", "fork",
                     "compact"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    base = rng.choice([1e4, 5e5, 1e6, 1e7])
    page = rng.choice([8, 16, 32, 64, 96, 128, 256])
    lens = rng.randrange(1 << 30)
    if op == "prefill_paged":
        ctx = _log(rng, 64, 60000)
        q_max = _log(rng, 1, 3000)
        chunks = max(1, min(12, int(2e8 / (G * Hkv * q_max * (ctx + q_max)))))
        return dict(op=op, D=D, Hq=G * Hkv, Hkv=Hkv, base=base, alpha=rng.choice([0.5, 1.0, 2.0, math.inf]),
                    g=rng.choice([1, 8]), page=page, ones=rng.randint(0, 20), chunks=chunks,
                    q_min=max(1, q_max // 2), q_max=q_max, ctx_min=rng.choice([0, ctx // 4]), ctx_max=ctx,
                    lens=lens)
    if op == "append_paged":
        q_max = _log(rng, 1, 3000)
        return dict(op=op, D=D, Hq=G * Hkv, Hkv=Hkv, base=base, page=page, axes=rng.choice([1, 3]),
                    ones=rng.randint(0, 100), chunks=rng.randint(1, 5), q_min=max(1, q_max // 3), q_max=q_max,
                    ctx_min=0, ctx_max=_log(rng, 16, 9000), lens=lens)
    if op == "rope_axes":
        return dict(op=op, D=D, Hq=G * Hkv, Hkv=Hkv, base=base, axes=rng.choice([1, 2, 3, 4]),
                    tokens=_log(rng, 1, 40000), inverse=rng.random() < 0.5)
    if op == "fork":
        ctx = _log(rng, 100, 4000)
        rows = rng.randint(1, 40)
        return dict(op=op, D=D, Hkv=Hkv, page=page, pools=rng.choice([2, 4]), rows=rows,
                    forks=rng.randint(1, 150), ctx_min=ctx // 4, ctx_max=ctx, lens=lens)
    return dict(op=op, D=D, Hkv=Hkv, page=rng.choice([8, 16, 32]), pools=rng.choice([2, 4]),
                pages=_log(rng, 64, 8000), live=rng.uniform(0.2, 0.9), rows=rng.randint(1, 60))


def _lens(c):
    """(new tokens, keys after them) of each sequence of a ragged case."""
    r = random.Random(c["lens"])
    q = [1] * c["ones"] + [r.randint(c["q_min"], c["q_max"]) for _ in range(c["chunks"])]
    r.shuffle(q)
    return q, [n + r.randint(c["ctx_min"], c["ctx_max"]) for n in q]


def _fork_plan(c):
    """(keys of each parent row, parent of each fork, its new row)."""
    r = random.Random(c["lens"])
    kv = [r.randint(c["ctx_min"], c["ctx_max"]) for _ in range(c["rows"])]
    src = [r.randrange(c["rows"]) for _ in range(c["forks"])]
    return kv, src, [c["rows"] + i for i in range(c["forks"])]


def _pages(n, page):
    return -(-n // page)


# ------------------------------------------------------------------ the inputs
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16)


def _pool(gen, pages, c):
    x = torch.empty((pages, c["page"], c["Hkv"], c["D"]), device=DEV, dtype=torch.bfloat16)
    step = max(1, (1 << 27) // (c["page"] * c["Hkv"] * c["D"]))
    for i in range(0, pages, step):  # in pieces: the float draws are twice as wide
        x[i:i + step] = _randn(gen, *x[i:i + step].shape)
    return x


def _axis_positions(gen, axes, tokens):
    """Positions of image or video tokens: the first axis steps frame by frame, the others run over each frame."""
    t = torch.arange(tokens, device=DEV, dtype=torch.int32)
    side = 36
    off = torch.randint(0, 5000, (1,), generator=gen, device=DEV, dtype=torch.int32)
    every = [t // (side * side), (t // side) % side, t % side, t]
    return torch.stack([(every[a] if axes > 1 else t) + off for a in range(axes)]).contiguous()


def _pair_axes(D, axes):
    """The axis of each pair: sections of consecutive pairs, the last one longest."""
    P = D // 2
    return [min(p * axes // P if axes < 3 else (p * 8 // P + 1) // 3, axes - 1) for p in range(P)]


def _tables(gen, rows, per_row, max_pages, pages):
    """Block table with every row's pages drawn without order from the pool, -1 behind them."""
    perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    start = torch.tensor([0] + per_row, device=DEV).cumsum(0)
    col = torch.arange(max_pages, device=DEV)
    n = torch.tensor(per_row, device=DEV)[:, None]
    at = (start[:-1, None] + col).clamp(max=pages - 1)
    return torch.where(col < n, perm[at], -1).to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] in ("prefill_paged", "append_paged"):
        s["new"], s["kv"] = _lens(c)
        T = sum(s["new"])
        need = [_pages(n, c["page"]) for n in s["kv"]]
        pages = sum(need) + 3
        s["k_pages"], s["v_pages"] = _pool(gen, pages, c), _pool(gen, pages, c)
        s["table"] = _tables(gen, len(need), need, max(need), pages)
        s["q"] = _randn(gen, T, c["Hq"], c["D"])
        if c["op"] == "append_paged":
            s["k"], s["v"] = _randn(gen, T, c["Hkv"], c["D"]), _randn(gen, T, c["Hkv"], c["D"])
            # the sequence of each new token and its row there
            s["seq"] = torch.tensor([b for b, n in enumerate(s["new"]) for _ in range(n)], device=DEV)
            s["row"] = torch.tensor([m - n + t for n, m in zip(s["new"], s["kv"]) for t in range(n)], device=DEV)
            if c["axes"] == 1:
                s["pos"], s["pair_axes"] = s["row"][None].to(torch.int32), None
            else:
                s["pos"], s["pair_axes"] = _axis_positions(gen, c["axes"], T), _pair_axes(c["D"], c["axes"])
    elif c["op"] == "rope_axes":
        s["q"], s["k"] = _randn(gen, c["tokens"], c["Hq"], c["D"]), _randn(gen, c["tokens"], c["Hkv"], c["D"])
        s["pos"], s["pair_axes"] = _axis_positions(gen, c["axes"], c["tokens"]), _pair_axes(c["D"], c["axes"])
    elif c["op"] == "fork":
        s["kv"], s["src"], s["dst"] = _fork_plan(c)
        need = [_pages(n, c["page"]) for n in s["kv"]]
        pages = sum(need) + len(s["src"]) + 5
        s["pools"] = [_pool(gen, pages, c) for _ in range(c["pools"])]
        table = _tables(gen, c["rows"], need, max(need), pages)
        s["table"] = torch.cat([table, torch.full((c["forks"], max(need)), -1, device=DEV, dtype=torch.int32)])
        s["refs"] = torch.zeros(pages + 1, device=DEV, dtype=torch.int32).index_add_(
            0, torch.where(table < 0, pages, table).reshape(-1), torch.ones_like(table).reshape(-1))[:pages].contiguous()
        # the same plan on the device, for the plain form
        kv = torch.tensor([s["kv"][i] for i in s["src"]], device=DEV)
        s["dev"] = (torch.tensor(s["src"], device=DEV), torch.tensor(s["dst"], device=DEV), kv // c["page"],
                    kv % c["page"], [i for i, r in enumerate(s["src"]) if s["kv"][r] % c["page"]])
    else:
        pages, live = c["pages"], max(1, int(c["pages"] * c["live"]))
        per = [live // c["rows"] + (1 if i < live % c["rows"] else 0) for i in range(c["rows"])]
        s["pools"] = [_pool(gen, pages, c) for _ in range(c["pools"])]
        s["table"] = _tables(gen, c["rows"], per, max(per) + 2, pages)
        s["refs"] = torch.zeros(pages + 1, device=DEV, dtype=torch.int32).index_add_(
            0, torch.where(s["table"] < 0, pages, s["table"]).reshape(-1),
            torch.ones_like(s["table"]).reshape(-1))[:pages].contiguous()
    return s


# ------------------------------------------------------------------ plain forms
def _threshold_runs(D, base, alpha, g):
    """Pairs of equal threshold: [(first pair, one past the last, threshold)]."""
    P = D // 2
    T = []
    for p in range(P):
        top = p if g == 1 else p // 8 * 8 + 7
        reach = alpha * (2 * math.pi * base ** (2 * top / D)) if alpha != math.inf else math.inf
        T.append(math.floor(reach) if reach < 4e18 else 1 << 62)
    runs = []
    for p in range(P):
        if runs and runs[-1][2] == T[p]:
            runs[-1][1] = p + 1
        else:
            runs.append([p, p + 1, T[p]])
    return runs


def _plain_prefill(s):
    c = s["case"]
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    G, P, scale = Hq // Hkv, D // 2, 1 / math.sqrt(D)
    runs = _threshold_runs(D, c["base"], c["alpha"], c["g"])
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], device=DEV, dtype=torch.float32)
    at = 0
    for b, (n, L) in enumerate(zip(s["new"], s["kv"])):  # the sequences have lengths of their own
        ids = s["table"][b, :_pages(L, c["page"])].long()
        k = s["k_pages"][ids].reshape(-1, Hkv, D)[:L].permute(1, 2, 0).float()      # [Hkv, D, L]
        v = s["v_pages"][ids].reshape(-1, Hkv, D)[:L].transpose(0, 1).float()       # [Hkv, L, D]
        step = max(1, (1 << 31) // (Hq * max(L, 1)))                                # bounds the scores' memory
        for t0 in range(0, n, step):
            m = min(step, n - t0)
            q = s["q"][at + t0:at + t0 + m].view(m, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * m, D).float()
            pos = torch.arange(L - n + t0, L - n + t0 + m, device=DEV).repeat(G)
            dist = pos[:, None] - torch.arange(L, device=DEV)                       # [G * m, L]
            far = [r for r in runs if r[2] < L - 1]
            p0 = far[-1][1] if far else 0                                           # pairs kept everywhere
            w = torch.cat([q[..., p0:P], q[..., P + p0:]], -1)
            x = torch.bmm(w, torch.cat([k[:, p0:P], k[:, P + p0:]], 1))
            for a, e, T in far:                                                     # pairs that end inside
                part = torch.bmm(torch.cat([q[..., a:e], q[..., P + a:P + e]], -1),
                                 torch.cat([k[:, a:e], k[:, P + a:P + e]], 1))
                x += part.mul_(dist <= T)
            x = x.mul_(scale).masked_fill_(dist < 0, -math.inf)
            top = x.amax(-1, keepdim=True).clamp(min=-3e38)
            x = x.sub_(top).exp_()
            total = x.sum(-1, keepdim=True)
            o = torch.bmm(x, v) / total.clamp(min=1e-38)
            l = torch.where(total > 0, top + total.log(), -math.inf)
            out[at + t0:at + t0 + m] = o.view(Hkv, G, m, D).permute(2, 0, 1, 3).reshape(m, Hq, D).to(out.dtype)
            lse[at + t0:at + t0 + m] = l.view(Hkv, G, m).permute(2, 0, 1).reshape(m, Hq)
        at += n
    return out, lse


def _turn(x, pos, pair_axes, base, inverse):
    """x [T, H, D] with pair p of token t turned by its axis' position times base^(-2p/D)."""
    P = x.shape[-1] // 2
    theta = base ** (torch.arange(P, device=DEV, dtype=torch.float64) * (-2.0 / x.shape[-1]))
    at = pos[torch.tensor(pair_axes, device=DEV)].T if pair_axes else pos[0][:, None]
    angle = at.double() * theta
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inverse:
        sin = -sin
    lo, hi = x[..., :P].float(), x[..., P:].float()
    return torch.cat([lo * cos - hi * sin, lo * sin + hi * cos], -1).to(x.dtype)


def _plain_append(s):
    c = s["case"]
    page = s["table"][s["seq"], s["row"] // c["page"]].long()
    slot = page * c["page"] + s["row"] % c["page"]
    s["k_pages"].view(-1, c["Hkv"], c["D"])[slot] = _turn(s["k"], s["pos"], s["pair_axes"], c["base"], False)
    s["v_pages"].view(-1, c["Hkv"], c["D"])[slot] = s["v"]
    return _turn(s["q"], s["pos"], s["pair_axes"], c["base"], False), s["k_pages"], s["v_pages"]


def _plain_fork(s):
    """Full pages shared, the begun page copied into the lowest free one; then the parents leave."""
    c = s["case"]
    table, refs = s["table"].clone(), s["refs"].clone()
    src, dst, full, part, some = s["dev"]
    rows = table[src]
    col = torch.arange(rows.shape[1], device=DEV)
    keep = col < full[:, None]
    new = torch.where(keep, rows, -1)
    if some:
        fork = torch.tensor(some, device=DEV)
        free = torch.argsort((refs > 0).to(torch.int8), stable=True)[:len(some)]
        old = rows[fork, full[fork]].long()
        new[fork, full[fork]] = free.to(torch.int32)
        refs[free] = 1
        begun = (torch.arange(c["page"], device=DEV) < part[fork][:, None])[..., None, None]
        for p in s["pools"]:
            p[free] = torch.where(begun, p[old], p[free])
    table[dst] = new
    refs.scatter_add_(0, torch.where(keep, rows, 0).reshape(-1).long(), keep.reshape(-1).to(torch.int32))
    gone = table[:c["rows"]]
    refs.scatter_add_(0, gone.clamp(min=0).reshape(-1).long(), -(gone >= 0).reshape(-1).to(torch.int32))
    table[:c["rows"]] = -1
    return [table, refs] + s["pools"]


def _plain_compact(s):
    """The k-th live page behind the first `live` slots moves to the k-th free slot among them."""
    table, refs = s["table"].clone(), s["refs"].clone()
    live = (refs > 0).sum()
    i = torch.arange(len(refs), device=DEV)
    old = ((refs > 0) & (i >= live)).nonzero()[:, 0]
    new = ((refs == 0) & (i < live)).nonzero()[:, 0]
    to = i.to(torch.int32)
    to[old] = new.to(torch.int32)
    for p in s["pools"]:
        p[new] = p[old]
    refs[new] = refs[old]
    refs[old] = 0
    table = torch.where(table >= 0, to[table.clamp(min=0).long()], table)
    return [table, refs, live.to(torch.int32).view(1)] + s["pools"]


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    c = s["case"]
    if not own:
        if c["op"] == "prefill_paged":
            return _plain_prefill(s)
        if c["op"] == "append_paged":
            return _plain_append(s)
        if c["op"] == "rope_axes":
            return (_turn(s["q"], s["pos"], s["pair_axes"], c["base"], c["inverse"]),
                    _turn(s["k"], s["pos"], s["pair_axes"], c["base"], c["inverse"]))
        return _plain_fork(s) if c["op"] == "fork" else _plain_compact(s)
    import rope_wavelength_sparsity_b200 as wp
    if c["op"] == "prefill_paged":
        return wp.prefill_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["new"], s["kv"],
                                wp.Window(c["D"], c["base"], c["alpha"], c["g"]))
    if c["op"] == "append_paged":
        q = wp.append_paged(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["new"], s["kv"],
                            q=s["q"], base=c["base"], positions=s["pos"], pair_axes=s["pair_axes"])
        return q, s["k_pages"], s["v_pages"]
    if c["op"] == "rope_axes":
        return wp.rope_axes(s["q"], s["k"], s["pos"], s["pair_axes"], base=c["base"], inverse=c["inverse"])
    table, refs = s["table"].clone(), s["refs"].clone()
    if c["op"] == "fork":
        wp.pages_fork(s["pools"], table, refs, s["src"], s["dst"], [s["kv"][i] for i in s["src"]])
        wp.pages_free(table, refs, range(c["rows"]), s["kv"], c["page"])
        return [table, refs] + s["pools"]
    live = wp.pages_compact(s["pools"], table, refs)
    return [table, refs, live] + s["pools"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "prefill_paged":
        new, kv = _lens(c)
        runs = _threshold_runs(c["D"], c["base"], c["alpha"], c["g"])
        flops = 0
        for n, L in zip(new, kv):
            lo = L - n + 1                                   # keys of the first query, L of the last
            flops += c["Hq"] * 2 * c["D"] * (lo + L) * n // 2
            for a, e, T in runs:                             # min(keys, T + 1) kept keys of each query
                cut = min(max(T + 1 - lo, 0), n)             # queries that reach all their keys
                kept = cut * (2 * lo + cut - 1) // 2 + (n - cut) * (T + 1)
                flops += c["Hq"] * 4 * (e - a) * kept
        T = sum(new)
        return {"bytes": 4 * sum(kv) * c["Hkv"] * c["D"] + T * c["Hq"] * (4 * c["D"] + 4), "flops": flops}
    if c["op"] in ("append_paged", "rope_axes"):
        T = sum(_lens(c)[0]) if c["op"] == "append_paged" else c["tokens"]
        heads = c["Hq"] + c["Hkv"] * (2 if c["op"] == "append_paged" else 1)
        return {"bytes": T * (4 * heads * c["D"] + 4 * c["axes"]), "flops": T * (c["Hq"] + c["Hkv"]) * 3 * c["D"]}
    one = c["page"] * c["Hkv"] * c["D"] * 2
    if c["op"] == "fork":
        kv, src, _ = _fork_plan(c)
        begun = sum(kv[i] % c["page"] for i in src)
        pages = sum(_pages(kv[i], c["page"]) for i in src) + sum(_pages(n, c["page"]) for n in kv)
        return {"bytes": 2 * c["pools"] * begun * one // c["page"] + 16 * pages, "flops": 0}
    live = max(1, int(c["pages"] * c["live"]))
    moved = live * (c["pages"] - live) / c["pages"]          # expected, of slots in random order
    return {"bytes": int(2 * c["pools"] * moved * one) + 8 * c["pages"] + 8 * live, "flops": 0}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _exact_rotation(x, pos, pair_axes, base, sign):
    D = x.shape[-1]
    y = x.double().clone()
    for p in range(D // 2):
        turn = torch.polar(torch.ones(x.shape[0], device=DEV, dtype=torch.float64),
                           sign * pos[pair_axes[p] if pair_axes else 0].double() * math.pow(base, -2 * p / D))
        z = torch.complex(x[..., p].double(), x[..., p + D // 2].double()) * turn[:, None]
        y[..., p], y[..., p + D // 2] = z.real, z.imag
    return y


def _exact_prefill(s):
    """Term by term: each pair's product is added where its distance is within the pair's window."""
    c = s["case"]
    D, Hq, P = c["D"], c["Hq"], c["D"] // 2
    G = Hq // c["Hkv"]
    out = torch.zeros(s["q"].shape, device=DEV, dtype=torch.float64)
    lse = torch.full(s["q"].shape[:2], -math.inf, device=DEV, dtype=torch.float64)
    at = 0
    for b, (n, L) in enumerate(zip(s["new"], s["kv"])):
        slots = (s["table"][b, :_pages(L, c["page"])].long()[:, None] * c["page"]
                 + torch.arange(c["page"], device=DEV)).reshape(-1)[:L]
        for h in range(Hq):
            k = s["k_pages"][:, :, h // G].reshape(-1, D)[slots].double()
            v = s["v_pages"][:, :, h // G].reshape(-1, D)[slots].double()
            q = s["q"][at:at + n, h].double()
            step = max(1, (1 << 28) // max(L, 1))
            for t0 in range(0, n, step):
                qs = q[t0:t0 + step]
                i = torch.arange(L - n + t0, L - n + t0 + len(qs), device=DEV)[:, None]
                d = i - torch.arange(L, device=DEV)[None]
                z = torch.zeros(d.shape, device=DEV, dtype=torch.float64)
                for p in range(P):
                    last = p if c["g"] == 1 else (p | 7)
                    wave = 2 * math.pi * math.pow(c["base"], 2 * last / D)
                    term = torch.outer(qs[:, p], k[:, p]).addr_(qs[:, p + P], k[:, p + P])
                    if math.floor(min(c["alpha"] * wave, 4e18)) < L:
                        term = torch.where(d <= math.floor(c["alpha"] * wave), term, 0.0)
                    z += term
                z = torch.where(d >= 0, z / math.sqrt(D), -math.inf)
                l = torch.logsumexp(z, -1)
                w = torch.where(torch.isfinite(l)[:, None], torch.exp(z - l[:, None]), 0.0)
                out[at + t0:at + t0 + len(qs), h] = w @ v
                lse[at + t0:at + t0 + len(qs), h] = l
        at += n
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "prefill_paged":
        return _exact_prefill(s)
    if c["op"] == "rope_axes":
        sign = -1.0 if c["inverse"] else 1.0
        return (_exact_rotation(s["q"], s["pos"], s["pair_axes"], c["base"], sign),
                _exact_rotation(s["k"], s["pos"], s["pair_axes"], c["base"], sign))
    if c["op"] == "append_paged":
        k = _exact_rotation(s["k"], s["pos"], s["pair_axes"], c["base"], 1.0)
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        table, t = s["table"].tolist(), 0
        for b, (n, m) in enumerate(zip(s["new"], s["kv"])):
            for j in range(m - n, m):
                kp[table[b][j // c["page"]], j % c["page"]] = k[t]
                vp[table[b][j // c["page"]], j % c["page"]] = s["v"][t].double()
                t += 1
        return _exact_rotation(s["q"], s["pos"], s["pair_axes"], c["base"], 1.0), kp, vp
    table, refs = s["table"].tolist(), s["refs"].tolist()
    if c["op"] == "fork":
        free, moves = [i for i, r in enumerate(refs) if r == 0], []
        for r in s["src"]:
            if s["kv"][r] % c["page"]:
                moves.append((table[r][s["kv"][r] // c["page"]], free[len(moves)], s["kv"][r] % c["page"]))
        lead = [None, None]
    else:
        live = sum(r > 0 for r in refs)
        holes = [i for i in range(live) if refs[i] == 0]
        late = [i for i in range(live, len(refs)) if refs[i] > 0]
        moves = [(a, b, c["page"]) for a, b in zip(late, holes)]
        lead = [None, None, None]
    done = []
    for p in s["pools"]:
        x = p.double()
        for a, b, rows in moves:
            x[b, :rows] = x[a, :rows]
        done.append(x)
    return lead + done
