"""Attention of a ragged batch of chunks over a paged cache, against 64 bits: odd lengths, rows
without keys, pages that end inside a tile, NaN wherever no key is, every head grouping; then bad
pages, streams, graphs, and agreement with the contiguous prefill and the paged decode."""
import pytest
import torch

import rope_wavelength_sparsity_b200 as wp

from _paged import attention64, check_attention, make_cache

pytestmark = pytest.mark.gpu

INF = float("inf")
CASES = {
    # D, g, alpha, base, Hq, Hkv, page, q_len, kv_len
    "one_token_one_key": (64, 1, 1.0, 1e4, 1, 1, 8, [1], [1]),
    "single_tokens": (128, 1, 1.0, 5e5, 24, 8, 16, [1, 1, 1, 1], [1, 517, 64, 2000]),
    "drafts": (128, 8, 1.0, 1e6, 28, 4, 16, [3, 8, 1, 5], [700, 8, 333, 1025]),
    "empty_among": (64, 8, 1.0, 1e6, 14, 2, 32, [0, 5, 0, 70, 0], [12, 5, 0, 300, 64]),
    "queries_before_keys": (128, 1, 1.0, 5e5, 6, 2, 16, [9, 40, 3], [4, 0, 3]),
    "first_chunks": (64, 1, 1.0, 1e4, 9, 3, 96, [130, 257, 1], [130, 257, 1]),
    "two_tiles": (128, 8, 1.0, 1e4, 14, 2, 64, [50], [700]),
    "long_chunk_g1": (128, 1, 1.0, 5e5, 6, 2, 64, [300], [1500]),
    "long_chunk_g1_d64": (64, 1, 2.0, 1e4, 4, 4, 8, [400], [1111]),
    "long_chunk_g8": (64, 8, 1.0, 1e6, 14, 2, 256, [513], [1400]),
    "tiny_window": (128, 1, 0.05, 1e4, 4, 1, 32, [200], [900]),
    "zero_window": (128, 8, 1e-9, 1e4, 4, 2, 32, [100], [300]),
    "window_off": (128, 1, INF, 5e5, 8, 1, 160, [190, 2], [800, 450]),
    "mqa_wide": (64, 1, 1.0, 1e4, 128, 1, 16, [5, 2], [100, 129]),
    "group_16": (128, 8, 2.0, 1e7, 32, 2, 128, [17, 33], [128, 127]),
    "group_65": (64, 8, 1.0, 1e6, 65, 1, 16, [6], [260]),
    "tile_edges": (128, 1, 1.0, 5e5, 3, 3, 128, [128, 256, 129, 127], [128, 256, 257, 383]),
    "mixed_batch": (64, 8, 1.0, 1e6, 14, 2, 16, [1, 200, 1, 1, 37, 1, 90], [900, 1200, 5, 128, 37, 640, 91]),
    "many_single_tokens": (128, 1, 1.0, 5e5, 8, 4, 16, [1] * 40, [2048 - 7 * i for i in range(40)]),
    "many_drafts": (64, 8, 1.0, 1e6, 8, 2, 32, [3] * 80, [1500 - 11 * i for i in range(80)]),
    "long_context": (64, 1, 1.0, 1e6, 4, 2, 16, [2, 1], [20000, 9001]),
    "long_context_chunk": (128, 8, 1.0, 1e7, 7, 1, 64, [150], [12000]),
    "million_keys": (64, 8, 1.0, 1e7, 2, 1, 256, [3], [(1 << 20) + 5]),
    "most_sequences": (128, 8, 1.0, 1e4, 2, 1, 8, [i % 4 for i in range(1024)], [1 + i % 97 for i in range(1024)]),
}


def _run(case, seed=0, **kw):
    D, g, alpha, base, Hq, Hkv, page, q_len, kv_len = case
    kp, vp, table, k, v = make_cache(kv_len, page, Hkv, D, seed)
    q = torch.randn((sum(q_len), Hq, D), generator=torch.Generator().manual_seed(seed + 1)).to(torch.bfloat16).cuda()
    out, lse = wp.prefill_paged(q, kp, vp, table, q_len, kv_len, wp.Window(D, base, alpha, g), **kw)
    return q, kp, vp, table, k, v, out, lse


@pytest.mark.parametrize("name", CASES)
def test_against_64_bits(cuda_dev, name):
    D, g, alpha, base, Hq, Hkv, page, q_len, kv_len = CASES[name]
    q, _, _, _, k, v, out, lse = _run(CASES[name])
    assert wp.device_status() == wp.OK
    ref = attention64(q, k, v, q_len, kv_len, Hq, Hkv, D, base, alpha, g)
    check_attention(out, lse, ref, D, max(kv_len), name)


def test_scale_and_given_outputs(cuda_dev):
    D, g, alpha, base, Hq, Hkv, page, q_len, kv_len = CASES["mixed_batch"]
    kp, vp, table, k, v = make_cache(kv_len, page, Hkv, D, 3)
    T = sum(q_len) + 5                       # rows behind the last sequence stay as they are
    q = torch.randn((T, Hq, D), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    win = wp.Window(D, base, alpha, g)
    out = torch.full_like(q, 7.0)
    lse = torch.full((T, Hq), 9.0, device="cuda")
    n = wp.prefill_paged_workspace_size(win, q_len, kv_len, Hq, Hkv)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
    got = wp.prefill_paged(q, kp, vp, table, q_len, kv_len, win, scale=0.3, out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse and wp.device_status() == wp.OK
    assert (out[-5:] == 7).all() and (lse[-5:] == 9).all() and (ws[n:] == 255).all()
    ref = attention64(q, k, v, q_len, kv_len, Hq, Hkv, D, base, alpha, g, scale=0.3)
    check_attention(out, lse, ref, D, max(kv_len))
    out2, none = wp.prefill_paged(q[:-5], kp, vp, table, q_len, kv_len, win, scale=0.3, want_lse=False)
    assert none is None and torch.equal(out2, out[:-5])


@pytest.mark.parametrize("name", ["mixed_batch", "long_context_chunk", "drafts"])
def test_same_bits_every_time(cuda_dev, name):
    first = _run(CASES[name])[-2:]
    for _ in range(3):
        again = _run(CASES[name])[-2:]
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("spot", ["last", "first"])
def test_bad_page_is_reported(cuda_dev, spot):
    D, g, alpha, base, Hq, Hkv, page, q_len, kv_len = CASES["mixed_batch"]
    kp, vp, table, k, v = make_cache(kv_len, page, Hkv, D, 5, fill=0.0)
    q = torch.randn((sum(q_len), Hq, D), device="cuda").to(torch.bfloat16)
    bad = table.clone()
    bad[1, 0 if spot == "first" else (kv_len[1] - 1) // page] = kp.shape[0] if spot == "last" else -1
    win = wp.Window(D, base, alpha, g)
    wp.prefill_paged(q, kp, vp, bad, q_len, kv_len, win)
    assert wp.device_status() == wp.EINDEX and wp.device_status() == wp.OK
    # entries behind a sequence's last page are not looked at
    wp.prefill_paged(q, kp, vp, table, q_len, kv_len, win)
    assert wp.device_status() == wp.OK


def test_other_stream_and_two_at_once(cuda_dev):
    cases = [CASES["mixed_batch"], CASES["long_context_chunk"]]
    want = [_run(c)[-2:] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = [_run(c, stream=s)[-2:] for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for (a, b), (x, y) in zip(want, got):
            assert torch.equal(a, x) and torch.equal(b, y)


@pytest.mark.parametrize("name", ["mixed_batch", "long_context_chunk"])
def test_captured_and_replayed(cuda_dev, name):
    D, g, alpha, base, Hq, Hkv, page, q_len, kv_len = CASES[name]
    kp, vp, table, k, v = make_cache(kv_len, page, Hkv, D, 8)
    q = torch.zeros((sum(q_len), Hq, D), dtype=torch.bfloat16, device="cuda")
    win = wp.Window(D, base, alpha, g)
    wp.prefill_paged(q, kp, vp, table, q_len, kv_len, win)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = wp.prefill_paged(q, kp, vp, table, q_len, kv_len, win)
    for seed in range(2):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16))
        graph.replay()
        want = wp.prefill_paged(q, kp, vp, table, q_len, kv_len, win)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_agrees_with_contiguous_prefill_and_paged_decode(cuda_dev):
    D, Hq, Hkv, page, L = 128, 6, 2, 32, 640
    win = wp.Window(D, 5e5, 1.0, 1)
    kp, vp, table, k, v = make_cache([L, L], page, Hkv, D, 11, fill=0.0)
    q = torch.randn((2 * 50, Hq, D), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    out, lse = wp.prefill_paged(q, kp, vp, table, [50, 50], [L, L], win)
    ref, ref_lse = wp.prefill(q.view(2, 50, Hq, D), torch.stack(k).cuda(), torch.stack(v).cuda(), win, q_pos0=L - 50)
    # two kernels, each with its weights and its result rounded to bf16: 4 roundings of values below 4
    assert (out.view(2, 50, Hq, D).float() - ref.float()).abs().max() <= 4 * 4 * 2.0 ** -8
    assert (lse.view(2, 50, Hq) - ref_lse.transpose(1, 2)).abs().max() <= 1e-4
    last = torch.tensor([49, 99], device="cuda")
    dec, dec_lse = wp.decode_paged(q[last].contiguous(), kp, vp, table, [L, L], win)
    assert (out[last].float() - dec.float()).abs().max() <= 4 * 4 * 2.0 ** -8
    assert (lse[last] - dec_lse).abs().max() <= 1e-4


@pytest.mark.parametrize("name", ["two_tiles", "long_chunk_g8", "drafts", "long_context", "long_context_chunk"])
def test_nan_in_a_query_row_stays_there(cuda_dev, name):
    """The row comes out as NaN (also where its keys are split), every other as without it."""
    D, g, alpha, base, Hq, Hkv, page, q_len, kv_len = CASES[name]
    kp, vp, table, _, _ = make_cache(kv_len, page, Hkv, D, 21)
    q = torch.randn((sum(q_len), Hq, D), generator=torch.Generator().manual_seed(22)).to(torch.bfloat16).cuda()
    win = wp.Window(D, base, alpha, g)
    want, want_lse = wp.prefill_paged(q, kp, vp, table, q_len, kv_len, win)
    rows = {(0, 0), (sum(q_len) // 2, Hq - 1), (sum(q_len) - 1, Hq // 2)}
    for t, h in rows:
        q[t, h, D // 2 - 1] = float("nan")
    out, lse = wp.prefill_paged(q, kp, vp, table, q_len, kv_len, win)
    hit = torch.zeros((sum(q_len), Hq), dtype=torch.bool, device="cuda")
    for t, h in rows:
        hit[t, h] = True
    assert out[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
    assert wp.device_status() == wp.OK


def test_rows_far_into_a_large_pool(cuda_dev):
    """Pages whose byte offset passes 2^31 and whose element offset passes 2^31."""
    D, Hkv, page = 128, 8, 128
    pages = (1 << 31) // (page * Hkv * D) + 40
    kp = torch.zeros((pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    gen = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.tensor([[pages - 1, 3, pages - 30]], dtype=torch.int32, device="cuda")
    for pool in (kp, vp):
        for i in ids[0].tolist():
            pool[i] = torch.randn(pool[i].shape, generator=gen, device="cuda").to(torch.bfloat16)
    q = torch.randn((20, 16, D), generator=gen, device="cuda").to(torch.bfloat16)
    out, lse = wp.prefill_paged(q, kp, vp, ids, [20], [300], wp.Window(D, 1e4, 1.0, 8))
    k = kp[ids[0].long()].view(-1, Hkv, D)[:300].cpu()
    v = vp[ids[0].long()].view(-1, Hkv, D)[:300].cpu()
    check_attention(out, lse, attention64(q, [k], [v], [20], [300], 16, Hkv, D, 1e4, 1.0, 8), D, 300)
