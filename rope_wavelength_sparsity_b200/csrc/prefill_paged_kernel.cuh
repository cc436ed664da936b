// Windowed causal attention of a ragged batch of chunks over a paged KV cache
// (TMA + tcgen05 + TMEM).
//
// "ATFlash: Per-RoPE-Wavelength Attention Windows", Abstract: the window is a
// slice of the query-key contraction axis and the online softmax is left
// untouched.  Query t of sequence b sits at kv_len - q_len + t and attends
// the sequence's keys 0 .. its position, found through the block table.
//
// Rows.  A tile's 128 rows are (token, head of one kv group) pairs, token
// by token: 128 / G tokens (rounded down) of all G query heads that read one
// kv head.  A cached key is thus read once for the whole group even when a
// sequence brings a single token, and a tile spans few positions, so fewer
// pairs are kept at some but not all of a key tile's distances.
//
// One CTA owns a row block (two row tiles that share every key tile) of one
// kv head of one sequence, over all or a part of the keys.  A row block with
// one tile runs it twice: its key tiles alternate between the two softmax
// groups (`dup`), which merge their halves at the end, so that one group's
// softmax overlaps the other's products there too.  Parts of a key range leave
// normalised fp32 results, merged by prefill_paged_merge_kernel.
//
// Warp roles (12 warps) as in the contiguous prefill:
//   warps 0-3, 4-7  softmax of tile 0 / 1: row r is TMEM lane r.  They bring Q
//              in, correct the pairs kept at some but not all distances of a
//              tile, mask, run the online softmax, write P (bf16) over S.
//   warps 8, 11  TMA producers of K and V: lane u copies unit u of a key tile
//              (R keys of one page, R = the largest power of two that divides
//              the page, up to 128).  One warp issues a copy every 40-54 ns,
//              whatever its size; 16-key pages need 16 a step, so K and V have
//              a warp each.
//   warps 9, 10  MMA issuers of tile 0 / 1; warp 9 owns the TMEM.  They issue as
//              whole warps, see warp_mma_ss.
//   The V producer also zeroes the V rows behind the sequence's last key.
//
// What bounds it.  A two-tile step is 2 x (QK + PV): 2070 tensor cycles at D =
// 128, and 2048 of the SM's exponentials, at 16 a clock.  At D = 128 a tile's
// chain is longer than either: its scores' way to registers and their maximum
// (450 cycles), 128 exponentials a thread (1350 alone, 2240 when both tiles'
// warps of an SM partition are at theirs), P's hand-over, the last quarter of
// PV and the next QK (1150).  Measured: 3650 cycles a step (4100 with the
// tiles' exponentials side by side).  At D = 64 the next QK runs early, beside
// the softmax, and a step is both tiles' softmax passes: 3000 cycles.  4096
// queries of 28 heads on 128K keys, 4 kv heads, g = 8: 5.55 to 6.3 ms (by GPU
// and power), 900 to 1000 TFLOP/s of kept terms.  One query in each of 64 sequences
// of 1000 to 32000 keys (D = 128, 16-key pages, 8 kv heads, g = 1): 677 to 689 us,
// 6.2 TB/s of K and V; all of 32000 keys (64-key pages, g = 8): 1.21 to 1.26 ms, 6.7
// to 6.9 TB/s.
//
// Shared-memory layouts.  K and V tiles are groups of 8 keys, each D / 64
// panels of 8 rows x 128 bytes, 128-byte swizzled: the layout one 4-D copy
// (64 dims, 8 keys, panels, groups) leaves, whatever the page size.  16-byte
// wide boxes, which would let a contraction step pair any two 8-dim columns,
// move a 32 KB tile in 1.17 us against 0.69 us at 128 bytes (0.31 us from
// L2), as long as the tile's whole arithmetic; so a step takes 16 dims of one
// half, and a unit of 16 pairs is two steps.  Q is no-swizzle K-major:
// 16-byte columns of 128 rows, 2 KB apart.
//
// TMEM columns: S_t at 128 t, O_t at 256 + t D; P_t (bf16) over the first half of
// S_t at D = 128, at 384 + 64 t at D = 64.  (Two score buffers of 64 keys per
// tile, which fit at D = 128 too and take QK off a tile's chain, were slower,
// 2.7 us a step: what a step costs beside its exponentials doubles.)
#pragma once

#include "device_util.cuh"
#include "prefill_kernel.cuh"

namespace wpattn {

constexpr int kPagedMaxB = 1024;

template <int MAXB>
struct PrefillPagedParams {
  const uint16_t* q;        // [T, Hq, D]
  const int32_t* block_table;  // [B, max_pages]
  uint16_t* out;            // [T, Hq, D]
  float* lse;               // [T, Hq] or null
  // parts: row r of CTA c at part_l[c * 256 + r], its dims 8 e .. 8 e + 7 at
  // part_o[((c * D / 8 + e) * 256 + r) * 8]
  float* part_o;
  float* part_l;            // log2-sum-exp, -inf: no key
  int B, Hq, Hkv, G, num_pages, page_size, max_pages;
  int unit;                 // keys per copy
  int tile_tokens;          // 128 / G
  float scale_log2;         // softmax scale * log2(e)
  int T[64];                // per-pair thresholds, clamped to int32
  // sequences in the order of the grid: CTA c belongs to the i-th when item0[i] <= c < item0[i + 1]
  int item0[MAXB + 1];
  uint16_t seq[MAXB];
  uint16_t parts[MAXB];     // key ranges of each of its row blocks,
  uint16_t lead[MAXB];      // equal but for the one of the last keys, which is this many tiles shorter
  int q_start[MAXB + 1];    // by sequence: first row in q
  int kv_len[MAXB];
};

// The i with start[i] <= at < start[i + 1] (start: n + 1 non-decreasing offsets, at < start[n]).
__device__ __forceinline__ int find_sequence(const int* start, int n, int at) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= at) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// What CTA c works on.
struct PagedItem {
  int b, kvh, rb, part, parts, lead;
  int q_len, kv_len, row0;  // row0: the sequence's first row in q
  int tok[2], ntok[2];      // first token and tokens of each row tile
  bool dup;
};

template <int MAXB>
__device__ __forceinline__ PagedItem paged_item(const PrefillPagedParams<MAXB>& p, int c) {
  PagedItem it;
  const int i = find_sequence(p.item0, p.B, c);
  const int local = c - p.item0[i];
  it.b = p.seq[i];
  it.parts = p.parts[i];
  it.lead = p.lead[i];
  it.row0 = p.q_start[it.b];
  it.q_len = p.q_start[it.b + 1] - it.row0;
  it.kv_len = p.kv_len[it.b];
  const int tiles = (it.q_len + p.tile_tokens - 1) / p.tile_tokens, blocks = (tiles + 1) >> 1;
  it.rb = blocks - 1 - local % blocks;   // longest rows first
  it.kvh = local / blocks % p.Hkv;
  it.part = local / blocks / p.Hkv;
  it.dup = 2 * it.rb + 1 >= tiles;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    it.tok[t] = (2 * it.rb + (it.dup ? 0 : t)) * p.tile_tokens;
    it.ntok[t] = min(p.tile_tokens, it.q_len - it.tok[t]);
  }
  return it;
}

// A block-table entry; one outside the pool is recorded and page 0 stands in for it.
__device__ __forceinline__ int checked_page(int pg, int num_pages) {
  if (pg < 0 || pg >= num_pages) {
    record_status(6 /* WPATTN_EINDEX */);
    return 0;
  }
  return pg;
}

template <int D>
struct PagedSmem {
  static constexpr int KT = 128;                     // keys of a key tile
  // K and V ring depths: even, so that with `dup` a stage's steps all belong to
  // one row tile.  A row tile's warps follow their own steps only, and a parity
  // wait cannot tell a phase from the one after next.
  static constexpr int NSK = D == 64 ? 4 : 2, NSV = NSK;
  static constexpr int TILE = KT * D * 2;            // a tile of K or V
  static constexpr int GROUP = 8 * D * 2;            // 8 keys
  static constexpr int COL = 128 * 16;               // 16-byte column of Q
  static constexpr int OFF_V = 0;
  static constexpr int OFF_K = NSV * TILE;
  static constexpr int OFF_Q1 = OFF_K + NSK * TILE;
  static constexpr int OFF_Q0 = OFF_Q1 + 128 * D * 2;
  static constexpr int OFF_QM = OFF_Q0 + 128 * D * 2;    // per tile: Q's first unit with its left-out pairs zeroed
  static constexpr int OFF_T = OFF_QM + 2 * 4 * COL;
  static constexpr int OFF_PS = OFF_T + 64 * 4;      // plan of each tile's next step
  static constexpr int OFF_LEFT = OFF_PS + 4 * 4;    // warps of each softmax group that left a corrected K tile
  static constexpr int OFF_TURN = OFF_LEFT + 4 * 4;  // per softmax warp: the step whose exponentials are its next
  static constexpr int OFF_BAR = OFF_TURN + 8 * 4;
  // k_full, k_empty [NSK], v_full, v_empty [NSV], s_full, p_most, p_full, o_final, q_ready, s_left, pv_done [2], v_fix
  static constexpr int NBAR = 2 * NSK + 2 * NSV + 15;
  static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
  static constexpr int ALLOC = OFF_TMEM + 16;
};
static_assert(PagedSmem<64>::NSK % 2 == 0 && PagedSmem<128>::NSK % 2 == 0, "even rings");
static_assert(PagedSmem<128>::ALLOC <= 232448 && PagedSmem<64>::ALLOC <= 232448, "shared memory of one CTA");

// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16u(uint32_t taddr, uint32_t* u) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15])
      : "r"(taddr));
}

// 32 columns of 16 TMEM lanes in the layout of four m16n8 MMA accumulators: register
// 4 i + e is row lane / 4 + 8 (e >> 1), column 8 i + 2 (lane % 4) + (e & 1).
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&u)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&u)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one)::"memory");
  return one;
}

// The products and commits of a whole, converged warp, issued by the lane whose
// `leader` is 1.  Every operand is the same in all lanes, so that the
// compiler can keep them in uniform registers, where the instructions take
// them from; in a one-lane branch each product cost 75 cycles to issue.  A
// descriptor's upper word is a constant, its lower one an address in
// 16-byte units plus a constant.
__device__ __forceinline__ void warp_mma_ss(uint32_t leader, uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo,
                                            uint32_t bhi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 q, %0, 0;\n\tsetp.ne.b32 p, %7, 0;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %6, p;\n\t}" ::"r"(leader),
      "r"(d), "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void warp_mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t blo, uint32_t bhi,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tsetp.ne.b32 q, %0, 0;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], b, %5, p;\n\t}" ::"r"(leader),
      "r"(d), "r"(a), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void warp_commit(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(leader),
      "r"(bar)
      : "memory");
}

template <int D, bool G8, int MAXB>
__global__ void __launch_bounds__(384, 1)
prefill_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ PrefillPagedParams<MAXB> p) {
  using L = PagedSmem<D>;
  constexpr int P = D / 2;
  constexpr int KT = L::KT, NSK = L::NSK, NSV = L::NSV, TILE = L::TILE, COL = L::COL;
  constexpr int W_PROD_K = 8, W_MMA = 9, W_PROD_V = 11;   // W_MMA + t issues tile t's products
  constexpr uint32_t TMEM_O = 256;
  // D = 64 leaves 128 TMEM columns free: P has columns of its own, and the next
  // QK starts as soon as the softmax group has its scores in registers
  constexpr bool EARLY = D == 64;
  // keys of P's first hand-over: at D = 128 most of PV runs under the last
  // exponentials; where PV is off the tile's chain the stores' wait costs more
  constexpr int kMost = EARLY ? 0 : KT * 3 / 4;
  constexpr int kCorr = 1 << 8, kSpecial = 1 << 9;   // of a step's plan, beside its split pair
  constexpr uint32_t FULL = 0xffffffffu;

  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar = sbase + L::OFF_BAR;
  auto k_full = [&](int s) { return bar + 8 * s; };
  auto k_empty = [&](int s) { return bar + 8 * (NSK + s); };
  auto v_full = [&](int s) { return bar + 8 * (2 * NSK + s); };
  auto v_empty = [&](int s) { return bar + 8 * (2 * NSK + NSV + s); };
  constexpr int B0 = 2 * NSK + 2 * NSV;
  auto s_full = [&](int t) { return bar + 8 * (B0 + t); };
  auto p_most = [&](int t) { return bar + 8 * (B0 + 2 + t); };
  auto p_full = [&](int t) { return bar + 8 * (B0 + 4 + t); };
  auto o_final = [&](int t) { return bar + 8 * (B0 + 6 + t); };
  auto q_ready = [&](int t) { return bar + 8 * (B0 + 8 + t); };
  auto s_left = [&](int t) { return bar + 8 * (B0 + 10 + t); };
  auto pv_done = [&](int t) { return bar + 8 * (B0 + 12 + t); };
  const uint32_t v_fix = bar + 8 * (B0 + 14);
  int* sT = reinterpret_cast<int*>(smem + L::OFF_T);
  volatile int* sPS = reinterpret_cast<volatile int*>(smem + L::OFF_PS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_TMEM);

  // the merge kernel may take its place on an SM as soon as there is room
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the swizzled tiles need a 1024-byte aligned shared window
  if (sbase & 1023u) {
    if (threadIdx.x == 0) record_status(2 /* WPATTN_EUNSUPPORTED */);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedItem it = paged_item(p, blockIdx.x);
  const bool dup = it.dup;
  const int nkt = (it.kv_len + KT - 1) / KT;
  const int per = it.parts > 1 ? (nkt + it.lead + it.parts - 1) / it.parts : nkt;
  const int kt_lo = it.part * per, kt_hi = min(kt_lo + per, nkt) - 1;
  const int pos0 = it.kv_len - it.q_len;              // the chunk's first position
  auto q_first = [&](int t) { return pos0 + (t == 0 ? it.tok[0] : it.tok[1]); };
  // key tiles of row tile t: kt_lo .. kt_last[t], walked downwards; none: kt_lo - 1
  int kt_last[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int i_max = q_first(t) + it.ntok[t] - 1;
    kt_last[t] = i_max < 0 ? kt_lo - 1 : max(min(i_max / KT, kt_hi), kt_lo - 1);
  }
  const int top = max(kt_last[0], kt_last[1]);
  const int steps = top - kt_lo + 1;                  // step j is key tile top - j
  auto attends = [&](int t, int j) { return dup ? (j & 1) == t : top - j <= kt_last[t]; };
  const bool tail = steps > 0 && top == nkt - 1 && it.kv_len % KT != 0;

  if (threadIdx.x < 64) sT[threadIdx.x] = p.T[threadIdx.x];
  if (threadIdx.x < 4) reinterpret_cast<int*>(smem + L::OFF_LEFT)[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NSK; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), dup ? 1 : 2);   // a release by each row tile that takes the stage
    }
    for (int s = 0; s < NSV; ++s) {
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), dup ? 1 : 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full(t), 1);
      mbar_init(p_most(t), 4);
      mbar_init(p_full(t), 4);
      mbar_init(s_left(t), 4);
      mbar_init(pv_done(t), 1);
      mbar_init(o_final(t), 1);
      mbar_init(q_ready(t), 4);
    }
    mbar_init(v_fix, 1);
    fence_barrier_init();
  }
  if (warp == W_MMA) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;          // an allocation of all 512 columns starts at the first

  if (warp >= 8) {
    regs_decrease<56>();
    if (warp == W_PROD_K || warp == W_PROD_V) {
      // --------------------------------------------------------- producers
      const bool is_k = warp == W_PROD_K;
      const CUtensorMap* map = is_k ? &tmK : &tmV;
      const uint32_t ring = sbase + (is_k ? L::OFF_K : L::OFF_V);
      const uint32_t full = is_k ? k_full(0) : v_full(0), empty = is_k ? k_empty(0) : v_empty(0);
      constexpr int stages = NSK;
      const int R = p.unit, units = KT / R;
      const int32_t* table = p.block_table + static_cast<size_t>(it.b) * p.max_pages;
      // this lane's unit of key tile kt: its 8-key group in the pool, -1: no key
      auto fetch = [&](int kt) -> int {
        const int key = KT * kt + lane * R;
        if (kt < kt_lo || lane >= units || key >= it.kv_len) return -1;
        const int pg = checked_page(__ldg(table + key / p.page_size), p.num_pages);
        return (pg * p.page_size + key % p.page_size) >> 3;
      };
      if (lane == 0) prefetch_tensormap(map);
      // V rows behind the sequence's last key may hold anything, and 0 * NaN would
      // reach every row's output: they are zeroed once the first tile is there
      auto zero_tail = [&]() {
        if (!__all_sync(FULL, mbar_wait(v_full(0), 0))) return;
        constexpr int ROW_CHUNKS = D / 8;
        for (int i = it.kv_len % KT * ROW_CHUNKS + lane; i < KT * ROW_CHUNKS; i += 32) {
          const int row = i / ROW_CHUNKS, c = i % ROW_CHUNKS;
          *reinterpret_cast<uint4*>(smem + L::OFF_V + (row >> 3) * L::GROUP + (c >> 3) * 1024 + (row & 7) * 128 +
                                    (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_fix);
      };
      int next = fetch(top), issued = 0;       // issued: tiles whose copies were issued
      int s = 0, ph = 0;
      for (int j = 0; j < steps; ++j) {
        if (tail && !is_k && j == stages) zero_tail();
        const int at = next;
        next = fetch(top - j - 1);
        const uint32_t bytes = __popc(__ballot_sync(FULL, at >= 0)) * R * D * 2;
        if (j >= stages && !__all_sync(FULL, mbar_wait(empty + 8 * s, ph ^ 1))) break;
        if (lane == 0) mbar_arrive_expect_tx(full + 8 * s, bytes);
        __syncwarp();
        if (at >= 0)
          tma_load_4d(ring + s * TILE + lane * R * D * 2, map, full + 8 * s, 0, 0, it.kvh * (D / 64), at);
        issued = j + 1;
        if (++s == stages) { s = 0; ph ^= 1; }
      }
      if (tail && !is_k && steps <= stages) zero_tail();
      if (issued < steps)   // a wait ran out: wait (bounded) for the copies that may still be landing
        for (int j = max(0, issued - stages); j < issued; ++j) (void)mbar_wait(full + 8 * (j % stages), (j / stages) & 1);
    } else {
      // ------------------------------------------------------- MMA issuers
      const int t = warp - W_MMA;
      constexpr uint32_t idesc_qk = make_idesc_bf16(128, KT, 0, 0);
      constexpr uint32_t idesc_pv = make_idesc_bf16(128, D, 0, 1);
      // descriptors: upper words (stride between 8-row groups, layout), lower words without the address
      constexpr uint32_t HI = 1u << 14;        // descriptor version
      constexpr uint32_t q_hi = HI | (128 >> 4), kv_hi = HI | (L::GROUP >> 4) | (2u << 29);
      constexpr uint32_t q_lo = (COL >> 4) << 16, k_lo = 1u << 16, v_lo = (1024u >> 4) << 16;
      const uint32_t leader = elect_one();
      const int stride = dup ? 2 : 1;
      const int j0 = dup ? t : top - (t == 0 ? kt_last[0] : kt_last[1]);
      const int mine = j0 < steps ? (steps - 1 - j0) / stride + 1 : 0;   // this tile's steps
      const uint32_t qa = q_lo | ((sbase + ((dup || t == 0) ? L::OFF_Q0 : L::OFF_Q1)) >> 4);
      const uint32_t qma = q_lo | ((sbase + L::OFF_QM + t * 4 * COL) >> 4);
      bool ok = true;
      int sk = 0, pk = 0, sv = 0, pv = 0;      // ring positions of the next QK's and the next PV's tile
      auto step_k = [&]() {
        if (++sk == NSK) { sk = 0; pk ^= 1; }
      };
      auto step_v = [&]() {
        if (++sv == NSV) { sv = 0; pv ^= 1; }
      };
      // steps that only the other tile takes: released once they are there
      for (int j = 0; ok && j < min(j0, steps); ++j) {
        if (!dup) {
          ok = __all_sync(FULL, mbar_wait(k_full(sk), pk) && mbar_wait(v_full(sv), pv));
          if (ok && leader) {
            mbar_arrive(k_empty(sk));
            mbar_arrive(v_empty(sv));
          }
        }
        step_k();
        step_v();
      }
      int plan = 0;                            // of the next QK's step
      // ready for the next QK: its K is there, and the plan that the softmax group
      // left beside its latest hand-over
      auto prepare_qk = [&]() {
        ok = ok && __all_sync(FULL, mbar_wait_handoff(k_full(sk), pk));
        plan = __shfl_sync(FULL, sPS[t], 0);
      };
      // S of this tile's next step, over the pairs from the split pair on
      auto issue_qk = [&]() {
        const int ps = plan & 0xFF, u0 = ps >> 4;
        const bool masked = (ps & 15) != 0;
        const uint32_t ka = k_lo | ((sbase + L::OFF_K + sk * TILE) >> 4);
#pragma unroll
        for (int u = 0; u < P / 16; ++u) {
          // the unit's second halves: the next 64-dim panel (D = 128), or 64 bytes on (D = 64)
          constexpr int HALF = (D == 128 ? 1024 : 64) >> 4;
          if (u == u0) {
            const uint32_t a = masked ? qma : qa + ((2 * u * COL) >> 4);
            const uint32_t a2 = masked ? qma + ((2 * COL) >> 4) : qa + (((2 * u + D / 16) * COL) >> 4);
            warp_mma_ss(leader, t * KT, a, q_hi, ka + 2 * u, kv_hi, idesc_qk, 0);
            warp_mma_ss(leader, t * KT, a2, q_hi, ka + 2 * u + HALF, kv_hi, idesc_qk, 1);
          } else if (u > u0) {
            warp_mma_ss(leader, t * KT, qa + ((2 * u * COL) >> 4), q_hi, ka + 2 * u, kv_hi, idesc_qk, 1);
            warp_mma_ss(leader, t * KT, qa + (((2 * u + D / 16) * COL) >> 4), q_hi, ka + 2 * u + HALF, kv_hi, idesc_qk, 1);
          }
        }
        warp_commit(leader, s_full(t));
        if (!(plan & kCorr)) warp_commit(leader, k_empty(sk));   // else the softmax group still reads K
        step_k();
        if (dup) step_k();
      };
      if (mine > 0) {
        ok = ok && __all_sync(FULL, mbar_wait(q_ready(t), 0));
        tc_fence_after();
        prepare_qk();
        if (ok) issue_qk();
      }
      const uint32_t tP = EARLY ? TMEM_O + 2 * D + t * (KT / 2) : t * KT;
      for (int n = 0; ok && n < mine; ++n) {
        const bool more = n + 1 < mine;
        if (EARLY && more) {
          ok = __all_sync(FULL, mbar_wait_handoff(s_left(t), n & 1));
          tc_fence_after();
          prepare_qk();
          if (!ok) break;
          issue_qk();
        }
        ok = __all_sync(FULL, mbar_wait_handoff(v_full(sv), pv));
        if (tail && n == 0 && j0 == 0) ok = ok && __all_sync(FULL, mbar_wait(v_fix, 0));
        const uint32_t va = v_lo | ((sbase + L::OFF_V + sv * TILE) >> 4);
#pragma unroll
        for (int last = kMost ? 0 : 1; last < 2; ++last) {
          ok = ok && __all_sync(FULL, mbar_wait_handoff(last ? p_full(t) : p_most(t), n & 1));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int ks = last ? kMost / 16 : 0; ks < (last ? KT : kMost) / 16; ++ks)
            warp_mma_ts(leader, TMEM_O + t * D, tP + ks * 8, va + ((ks * 2 * L::GROUP) >> 4), kv_hi, idesc_pv,
                        (n > 0 || ks > 0) ? 1u : 0u);
          if (!EARLY && !last && more) prepare_qk();
        }
        if (!ok) break;
        if (EARLY) warp_commit(leader, pv_done(t));
        else if (more) issue_qk();             // first: the softmax group waits for it
        warp_commit(leader, v_empty(sv));
        step_v();
        if (dup) step_v();
      }
      // every product of this tile has completed once this arrives
      warp_commit(leader, o_final(t));
      if (!ok) (void)mbar_wait(o_final(t), 0);
      __syncwarp();
    }
  } else {
    regs_increase<224>();
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;
    const int wq = warp & 3;
    const int r = wq * 32 + lane;              // row of the tile = TMEM lane
    const int tok = r / p.G;
    const int tok0 = t == 0 ? it.tok[0] : it.tok[1], ntok = t == 0 ? it.ntok[0] : it.ntok[1];
    const bool row_ok = r < p.tile_tokens * p.G && tok < ntok;
    const int i_pos = q_first(t) + min(tok, ntok - 1);   // rows without a token walk with the last
    const size_t qrow = (static_cast<size_t>(it.row0) + tok0 + (row_ok ? tok : 0)) * p.Hq +
                        static_cast<size_t>(it.kvh) * p.G + (row_ok ? r % p.G : 0);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t tO = lane_base + TMEM_O + t * D;
    uint8_t* smem_q = smem + ((dup || t == 0) ? L::OFF_Q0 : L::OFF_Q1);
    uint8_t* smem_qm = smem + L::OFF_QM + t * 4 * COL;
    const int my_last = t == 0 ? kt_last[0] : kt_last[1];
    volatile int* turn = reinterpret_cast<volatile int*>(smem + L::OFF_TURN);
    float m_ref = -INFINITY;   // exponent reference of O and l (log2 units)
    float l_run = 0.f;
    int cnt = 0;
    bool ok = true;

    if (steps > 0 && !(dup && t == 1)) {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + qrow * D);
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        *reinterpret_cast<uint4*>(smem_q + c * COL + r * 16) = row_ok ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
    }
    const int stride = dup ? 2 : 1;            // this tile's steps: every stride-th from j0 on
    const int j0 = dup ? t : top - my_last;
    if (lane == 0) turn[warp] = j0;
    asm volatile("bar.sync 1, 256;" ::: "memory");   // dup: group 1 reads group 0's rows

    // The first pair kept somewhere in step j (plo) and the split pair (ps) of a pair
    // of steps only move forward along the walk; each carries its threshold.
    struct Cursor { int pair, T; };
    auto advance = [&](Cursor& c, int d) {     // to the first pair whose threshold is at least d
      while (c.pair < P && c.T < d) {
        ++c.pair;
        c.T = c.pair < P ? sT[c.pair] : 0x7FFFFFFF;
      }
    };
    const int q0 = pos0 + tok0;                // positions of the tile's first and last row
    const int q1 = q0 + ntok - 1;
    auto nearest = [&](int j) { return q0 - (KT * (top - j) + KT - 1); };   // smallest distance of step j
    // Split pair of a step: pairs plo .. ps - 1 are
    // left out of the contraction and added back where they are kept; pairs ps
    // .. P - 1 are contracted and subtracted where they are pruned.  At the
    // pair first kept 32 past the tile's centre distance both sets are small
    // (thresholds grow geometrically).  Any ps >= plo gives the same scores.
    Cursor low{0, sT[0]}, far = low;
    int ps_now = P, T_ps = 0, T_before = 0;    // of the latest plan; thresholds of ps and the pair before
    int quiet = 0;                             // steps behind the latest planned one that have the same plan
    // Plan of step j (called for steps in turn): split pair, kCorr when some score
    // needs a correction, kSpecial when anything but the plain step is to be
    // done, and plo << 16.  From one step to the next all distances grow by
    // the same amount, so a plain plan holds until the first of three
    // thresholds is passed.
    auto plan_step = [&](int j) -> int {
      const int kp0 = KT * (top - j), d_min = nearest(j);
      advance(low, d_min);
      const int centre = max(q0 + (p.tile_tokens >> 1) - (kp0 + KT / 2), 0) + 32;
      advance(far, centre);
      const int ps = low.pair >= P ? P : min(max(far.pair, low.pair), P - (G8 ? 8 : 1));
      if (ps != ps_now || j == j0) {
        T_ps = ps < P ? sT[ps] : 0x7FFFFFFF;
        T_before = ps > 0 ? sT[ps - 1] : -1;
        ps_now = ps;
      }
      const bool corr = low.pair < P && (q1 - kp0 > T_ps || (ps > low.pair && d_min <= T_before));
      const bool special = corr || low.pair >= P || d_min < 0 || kp0 + KT > it.kv_len;
      const int shift = dup ? 8 : 7;
      static_assert(KT == 128, "steps are 128 keys, or 256, apart");
      quiet = special ? 0 : min(min(low.T - d_min, far.T - centre), T_ps - (q1 - kp0)) >> shift;
      return ps | (corr ? kCorr : 0) | (special ? kSpecial : 0) | low.pair << 16;
    };
    // pairs whose threshold is below d (thresholds grow; two a lane)
    const int T_lo = lane < P ? sT[lane] : 0x7FFFFFFF, T_hi = lane + 32 < P ? sT[lane + 32] : 0x7FFFFFFF;
    auto pairs_below = [&](int d) -> int {
      return __popc(__ballot_sync(FULL, T_lo < d)) + __popc(__ballot_sync(FULL, T_hi < d));
    };
    // Copy of Q's unit of 16 pairs that starts the contraction for split pair
    // ps, its pairs below ps zeroed.  The split pair only moves forward and
    // mostly stays put, so an unchanged copy is kept.
    int qm_ps = -1;
    auto write_masked_q = [&](int ps) {
      const int rz = ps & 15;
      if (rz == 0 || ps >= P || ps == qm_ps) return;
      qm_ps = ps;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int first = 8 * (c & 1);         // the column's first pair within the unit
        uint4 x = *reinterpret_cast<const uint4*>(smem_q + (2 * (ps >> 4) + (c & 1) + (c >> 1) * (D / 16)) * COL + r * 16);
        const int z = rz - first;              // pairs zeroed in this column
        x.x &= (z > 0 ? 0u : 0xFFFFu) | (z > 1 ? 0u : 0xFFFF0000u);
        x.y &= (z > 2 ? 0u : 0xFFFFu) | (z > 3 ? 0u : 0xFFFF0000u);
        x.z &= (z > 4 ? 0u : 0xFFFFu) | (z > 5 ? 0u : 0xFFFF0000u);
        x.w &= (z > 6 ? 0u : 0xFFFFu) | (z > 7 ? 0u : 0xFFFF0000u);
        *reinterpret_cast<uint4*>(smem_qm + c * COL + r * 16) = x;
      }
      fence_proxy_async_smem();
    };

    int plan = 0;
    if (j0 < steps) {
      plan = plan_step(j0);
      write_masked_q(plan & 0xFF);
      if (r == 0) sPS[t] = plan & 0xFFFF;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(q_ready(t));

    const uint32_t tS = lane_base + t * KT, tP = EARLY ? lane_base + TMEM_O + 2 * D + t * (KT / 2) : tS;
    // what the MMA warp needs for the next QK, before the arrival that lets it start
    auto tell_next = [&](int plan, int plan_next) {
      if (plan_next == plan) return;
      write_masked_q(plan_next & 0xFF);
      if (r == 0) sPS[t] = plan_next & 0xFFFF;
    };
    const float sl = p.scale_log2;
    // What a step that is not plain changes in S before the softmax reads it: scores
    // corrected, keys masked, every pair pruned.  In TMEM, in code of its own and in
    // loops: with these branches in the softmax's code every step took 800
    // cycles more, and a second copy of that code for them 2 us of a cold start.
    auto prepare_scores = [&](int j, int plan) {
      const int kp0 = KT * (top - j);
      const int d_row = i_pos - kp0;           // distance to the tile's first key
      // Per-element corrections, d = d_row - c for column c of the tile:
      // pairs plo .. ps - 1 were left out: add them where 0 <= d <= T;
      // pairs ps .. P - 1 were contracted: subtract them where d > T.
      const int plo = plan >> 16, ps = plan & 0xFF;
      if (plan & kCorr) {
        const int sk = j % NSK;
        const bool need_sub = __any_sync(FULL, d_row > sT[min(ps, P - 1)]);
        const int T_add = ps > plo ? sT[ps - 1] : -1;
        const bool need_add = ps > plo && __any_sync(FULL, d_row >= 0 && d_row - (KT - 1) <= T_add);
        // A pair's (g = 8: a group's) products are added to S, which comes from TMEM in
        // the layout of MMA accumulators (16 lanes x 256 bits), every element
        // choosing by its distance.  (Through a scratch and row by row a pair took
        // 450 cycles for 32 keys.)
        int pr[4];                             // distances of this lane's rows 8 k + lane / 4 to the tile's first key
#pragma unroll
        for (int k = 0; k < 4; ++k) pr[k] = __shfl_sync(FULL, d_row, (lane >> 2) + 8 * k) - 2 * (lane & 3);
        int d_first[2], d_last[2];             // of 16 rows
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          d_first[mt] = __shfl_sync(FULL, d_row, 16 * mt);
          d_last[mt] = __shfl_sync(FULL, d_row, 16 * mt + 15);
        }
#pragma unroll 1
        for (int cc = 0; cc < KT / 32; ++cc) {
          const int dmax = d_last[1] - 32 * cc, dmin = max(d_first[0] - 32 * cc - 31, 0);
          if (dmax < 0) continue;              // wholly acausal
          // pairs ps .. pb - 1 are pruned somewhere in the chunk, pa .. ps - 1 kept somewhere
          const int pb = need_sub ? max(ps, pairs_below(dmax)) : ps;
          const int pa = need_add ? min(ps, max(plo, pairs_below(dmin))) : ps;
          if (pa >= pb) continue;
          uint32_t v[2][16];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) tmem_ld_frag(tS + 32 * cc + (static_cast<uint32_t>(16 * mt) << 16), v[mt]);
          tmem_ld_wait();
          if constexpr (G8) {
            // the group's products by warp-level MMAs, m16n8k16: A = Q rows, dims 8 grp
            // .. then P + 8 grp .., B = K rows, S their addend
            const uint32_t kb = sbase + L::OFF_K + sk * TILE;
            const int qm = lane >> 3, qi = lane & 7;
            uint32_t af[2][4], bf[4][2];
#pragma unroll 1
            for (int pp = pa; pp < pb; pp += 8) {
              const int grp = pp >> 3;
#pragma unroll
              for (int mt = 0; mt < 2; ++mt)   // matrix m: rows 8 (m & 1) .., half m >> 1
                ldsm_x4(smem_u32(smem_q) + ((qm >> 1) ? P / 8 + grp : grp) * COL + (wq * 32 + 16 * mt + 8 * (qm & 1) + qi) * 16,
                        af[mt][0], af[mt][1], af[mt][2], af[mt][3]);
#pragma unroll
              for (int hp = 0; hp < 2; ++hp) { // matrix m: keys 8 (m >> 1) .., first (m even) or second half
                const int key = 32 * cc + 16 * hp + 8 * (qm >> 1) + qi;
                const int ch = (qm & 1) ? P / 8 + grp : grp;
                ldsm_x4(kb + (key >> 3) * L::GROUP + (ch >> 3) * 1024 + (key & 7) * 128 + (((ch & 7) ^ (key & 7)) << 4),
                        bf[2 * hp][0], bf[2 * hp][1], bf[2 * hp + 1][0], bf[2 * hp + 1][1]);
              }
              const bool sub = pp >= ps;
              const uint32_t flip = sub ? 0x80008000u : 0u;   // subtract: Q with its sign turned
              const int edge = 32 * cc + sT[pp];
#pragma unroll
              for (int mt = 0; mt < 2; ++mt) {
                // columns below d - edge are beyond the threshold: in none of the rows, or in all
                if (sub ? d_last[mt] <= edge : d_first[mt] - edge >= 32) continue;
                const int r0 = pr[2 * mt] - edge, r1 = pr[2 * mt + 1] - edge;
                float z[4][4];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) z[nt][e] = __uint_as_float(v[mt][4 * nt + e]);
                  mma_16816_bf16(z[nt], af[mt][0] ^ flip, af[mt][1] ^ flip, af[mt][2] ^ flip, af[mt][3] ^ flip,
                                 bf[nt][0], bf[nt][1]);
                }
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const bool beyond = 8 * nt + (e & 1) < (e < 2 ? r0 : r1);
                    v[mt][4 * nt + e] = beyond == sub ? __float_as_uint(z[nt][e]) : v[mt][4 * nt + e];
                  }
              }
            }
          } else {
            // One pair is two products an element, on the FMA pipe.  (As MMAs with all
            // but the pair's own dims zeroed, and the pairs searched one by one, a
            // tile on the diagonal took 9.9 us more than a plain one, now 6.2 us.)
            const int c0 = 2 * (lane & 3);     // this lane's columns: c0 and c0 + 1 of each 8
#pragma unroll 1
            for (int pp = pa; pp < pb; ++pp) {
              const bool sub = pp >= ps;
              const int edge = 32 * cc + sT[pp];
              const uint8_t* qa = smem_q + (pp >> 3) * COL + (wq * 32 + (lane >> 2)) * 16 + (pp & 7) * 2;
              float q[4][2], k[4][2][2];       // [row 8 i][half]; [8 columns][column][half]
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float x = bf16lo_to_f32(*reinterpret_cast<const uint16_t*>(qa + i * 128 + h * (P / 8) * COL));
                  q[i][h] = sub ? -x : x;
                }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int ch = (pp >> 3) + h * (P / 8);
                const uint8_t* ka = smem + L::OFF_K + sk * TILE + 4 * cc * L::GROUP + (ch >> 3) * 1024 + (pp & 7) * 2;
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                  for (int nt = 0; nt < 4; ++nt)
                    k[nt][e][h] = bf16lo_to_f32(*reinterpret_cast<const uint16_t*>(
                        ka + nt * L::GROUP + (c0 + e) * 128 + (((ch & 7) ^ (c0 + e)) << 4)));
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int rr = pr[i] - edge;   // columns below it are beyond the pair's threshold
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                  uint32_t& v0 = v[i >> 1][4 * nt + 2 * (i & 1)];
                  uint32_t& v1 = v[i >> 1][4 * nt + 2 * (i & 1) + 1];
                  float z0, z1;
                  fma2(z0, z1, q[i][0], q[i][0], k[nt][0][0], k[nt][1][0], __uint_as_float(v0), __uint_as_float(v1));
                  fma2(z0, z1, q[i][1], q[i][1], k[nt][0][1], k[nt][1][1], z0, z1);
                  v0 = (8 * nt < rr) == sub ? __float_as_uint(z0) : v0;
                  v1 = (8 * nt + 1 < rr) == sub ? __float_as_uint(z1) : v1;
                }
              }
            }
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) tmem_st_frag(tS + 32 * cc + (static_cast<uint32_t>(16 * mt) << 16), v[mt]);
        }
        tmem_st_wait();
        // the group's last warp to be through with K releases it
        __threadfence_block();
        __syncwarp();
        if (lane == 0 && (atomicAdd(reinterpret_cast<int*>(smem + L::OFF_LEFT) + t, 1) & 3) == 3)
          mbar_arrive(k_empty(sk));
      }
      // causal mask (d < 0) and the sequence's end: columns c > cm; every pair pruned: score 0
      const int cm = min(d_row, it.kv_len - 1 - kp0);
#pragma unroll 1
      for (int cc = 0; cc < KT / 32; ++cc) {
        if (plo < P && __all_sync(FULL, cm >= 32 * cc + 31)) continue;
        float v[32];
        tmem_ld32(tS + 32 * cc, v);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = 32 * cc + c > cm ? -INFINITY : plo >= P ? 0.f : v[c];
        tmem_st32(tS + 32 * cc, v);
      }
      tmem_st_wait();
    };
    // Step j, its scores in S: from there to P's hand-over.
    auto step = [&](int j, int plan, int plan_next, bool more) {
      if (plan & kSpecial) prepare_scores(j, plan);
      float sc[KT];
#pragma unroll
      for (int cc = 0; cc < KT / 32; ++cc) tmem_ld32(tS + 32 * cc, &sc[32 * cc]);
      tmem_ld_wait();
      if (EARLY) {                             // S may be overwritten
        if (more) tell_next(plan, plan_next);
        tc_fence_before();
        __syncwarp();
        if (more && lane == 0) mbar_arrive(s_left(t));
      }
      // the loaded values are only defined after the wait: keep every use below it
#pragma unroll
      for (int c = 0; c < KT; ++c) asm volatile("" : "+f"(sc[c]));
      // row max, then the exponentials against the (lazily moved) reference
      float mt;
      {
        float a16[16], b6[6];
#pragma unroll
        for (int k = 0; k < 16; ++k)
          a16[k] = max3(max3(sc[8 * k], sc[8 * k + 1], sc[8 * k + 2]), max3(sc[8 * k + 3], sc[8 * k + 4], sc[8 * k + 5]),
                        fmaxf(sc[8 * k + 6], sc[8 * k + 7]));
#pragma unroll
        for (int k = 0; k < 5; ++k) b6[k] = max3(a16[3 * k], a16[3 * k + 1], a16[3 * k + 2]);
        b6[5] = a16[15];
        mt = fmaxf(max3(b6[0], b6[1], b6[2]), max3(b6[3], b6[4], b6[5])) * sl;
      }
      // the reference moves only when the max grew by more than 8 (x256)
      float f = 1.f;
      if (cnt == 0) {
        m_ref = mt;
      } else if (mt > m_ref + 8.f) {
        f = (m_ref == -INFINITY) ? 0.f : ex2_approx(m_ref - mt);
        m_ref = mt;
      }
      // this tile's previous PV has left O (and P) once s_full, or pv_done, says so
      const bool scale_o = cnt > 0 && __any_sync(FULL, f != 1.f);
      if (EARLY && cnt > 0) (void)__all_sync(FULL, mbar_wait_handoff(pv_done(t), (cnt - 1) & 1));
      if (scale_o) {
#pragma unroll 1
        for (int cc = 0; cc < D / 16; ++cc) {
          uint32_t o[16];
          tmem_ld16u(tO + 16 * cc, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tmem_st16u(tO + 16 * cc, o);
        }
      }
      // p, rounded to bf16 (the MMA's operand type); l sums them unrounded
      {
        float nm = (m_ref == -INFINITY) ? 0.f : -m_ref;
        if constexpr (!EARLY) {
          // Warps w and w + 4 share an SM partition and its exponentials.  They take
          // turns, tile 0 first in each step, so that one tile's products run under
          // the other's exponentials (side by side both would wait for both), in
          // the same order on every partition (or a tile waits for its last
          // warp).  The wait is bounded and may be given up: it orders nothing.
          // At D = 64, whose next QK is early, side by side is faster: 1.57 us a step
          // against 1.65.
#pragma unroll 1
          for (int i = 0; i < 256 && turn[warp ^ 4] < (t && !dup ? j + 1 : j); ++i) {}
        }
        asm volatile("" : "+f"(nm));           // no exponential above this
        float acc[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = 0.f;
        uint32_t pk2[KT / 2];
#pragma unroll
        for (int i = 0; i < KT / 2; ++i) {
          float x0, x1;
          fma2(x0, x1, sc[2 * i], sc[2 * i + 1], sl, sl, nm, nm);
          const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
          add2(acc[2 * (i & 3)], acc[2 * (i & 3) + 1], acc[2 * (i & 3)], acc[2 * (i & 3) + 1], e0, e1);
          pk2[i] = pack_bf16x2(e0, e1);
          if (kMost && i == kMost / 2 - 1) {
            tmem_st32u(tP, pk2);
            tmem_st16u(tP + 32, pk2 + 32);
            if (more) tell_next(plan, plan_next);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_most(t));
          }
        }
        if constexpr (EARLY) {
          tmem_st32u(tP, pk2);
          tmem_st32u(tP + 32, pk2 + 32);
        } else {
          tmem_st16u(tP + 48, pk2 + 48);
          if (lane == 0) turn[warp] = j + 1;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(t));
        l_run = l_run * f + (((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7])));
      }
    };
    for (int j = j0; ok && j < steps; j += stride) {
      const bool more = j + stride < steps;
      int plan_next = plan;
      if (quiet > 0) --quiet;
      else if (more) plan_next = plan_step(j + stride);
      if (!__all_sync(FULL, mbar_wait_handoff(s_full(t), cnt & 1))) { ok = false; break; }
      tc_fence_after();
      step(j, plan, plan_next, more);
      ++cnt;
      plan = plan_next;
    }
    if (lane == 0) turn[warp] = 0x7FFFFFFF;

    // ----------------------------------------------------------- epilogue
    (void)__all_sync(FULL, mbar_wait(o_final(t), 0));     // this tile's products have completed
    if (dup) (void)__all_sync(FULL, mbar_wait(o_final(t ^ 1), 0));   // and so has all use of the ring
    tc_fence_after();
    const bool split = it.parts > 1;
    // dup: group 1 hands its half over through the ring, which every MMA has left
    float* half = reinterpret_cast<float*>(smem);            // [D][128 rows]
    float2* half_ml = reinterpret_cast<float2*>(smem + 128 * D * 4);   // (m, l)
    if (dup) {
      if (t == 1) {
        half_ml[r] = make_float2(m_ref, l_run);
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          if (cnt == 0) break;
          float o[32];
          tmem_ld32(tO + 32 * cc, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) half[(32 * cc + e) * 128 + r] = o[e];
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    if (!(dup && t == 1)) {
      float w0 = 1.f, w1 = 0.f;                // weights of this group's O and of the other's
      if (dup) {
        const float2 other = half_ml[r];
        const float M = fmaxf(m_ref, other.x);
        if (M != -INFINITY) {
          w0 = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - M);
          w1 = other.x == -INFINITY ? 0.f : ex2_approx(other.x - M);
        }
        l_run = l_run * w0 + other.y * w1;
        m_ref = M;
      }
      const float inv = l_run != 0.f ? 1.f / l_run : 0.f;   // a NaN stays one, in O and in the parts
      w0 *= inv;
      w1 *= inv;
      const bool both = dup && steps > 1;      // group 1 had a key tile
      const size_t prow = static_cast<size_t>(blockIdx.x) * 256 + t * 128 + r;
      float* po = p.part_o + (static_cast<size_t>(blockIdx.x) * (D / 8) * 256 + t * 128 + r) * 8;
      uint16_t* orow = p.out + qrow * D;
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        float o[32];
        if (cnt > 0) {
          tmem_ld32(tO + 32 * cc, o);
          tmem_ld_wait();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          o[e] = cnt > 0 ? o[e] * w0 : 0.f;
          if (both) o[e] = fmaf(half[(32 * cc + e) * 128 + r], w1, o[e]);
        }
        if (!row_ok) continue;
        if (split) {
#pragma unroll
          for (int c8 = 0; c8 < 4; ++c8) {
            float4* dst = reinterpret_cast<float4*>(po + static_cast<size_t>(4 * cc + c8) * 256 * 8);
            dst[0] = make_float4(o[8 * c8], o[8 * c8 + 1], o[8 * c8 + 2], o[8 * c8 + 3]);
            dst[1] = make_float4(o[8 * c8 + 4], o[8 * c8 + 5], o[8 * c8 + 6], o[8 * c8 + 7]);
          }
        } else {
#pragma unroll
          for (int c8 = 0; c8 < 4; ++c8)
            *reinterpret_cast<uint4*>(orow + 32 * cc + 8 * c8) =
                make_uint4(pack_bf16x2(o[8 * c8], o[8 * c8 + 1]), pack_bf16x2(o[8 * c8 + 2], o[8 * c8 + 3]),
                           pack_bf16x2(o[8 * c8 + 4], o[8 * c8 + 5]), pack_bf16x2(o[8 * c8 + 6], o[8 * c8 + 7]));
        }
      }
      const float l2 = l_run != 0.f ? m_ref + __log2f(l_run) : -INFINITY;
      if (row_ok && split) p.part_l[prow] = l2;
      else if (row_ok && p.lse) p.lse[qrow] = l2 * 0.69314718055994530942f;
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W_MMA) tmem_dealloc(*tmem_slot, 512);
}

// Merge of the parts of one row block: with w_s = 2^(l_s - max l), out = sum_s
// w_s o_s / sum_s w_s.  Block (c, y): rows of CTA c, when it is its row
// block's first part, dims 32 y .. 32 y + 31; a thread per row.
template <int D, int MAXB>
__global__ void __launch_bounds__(256)
prefill_paged_merge_kernel(const __grid_constant__ PrefillPagedParams<MAXB> p) {
  const int c = blockIdx.x;
  const PagedItem it = paged_item(p, c);
  if (it.part != 0) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");      // the parts are there (the kernel before has ended)
  const int t = threadIdx.x >> 7, r = threadIdx.x & 127;
  const int tok = r / p.G;
  if ((it.dup && t == 1) || r >= p.tile_tokens * p.G || tok >= it.ntok[t]) return;
  const int tiles = (it.q_len + p.tile_tokens - 1) / p.tile_tokens;
  const int step = ((tiles + 1) >> 1) * p.Hkv;             // CTAs from one part to the next
  const float* pl = p.part_l + static_cast<size_t>(c) * 256 + threadIdx.x;
  const float* po = p.part_o + ((static_cast<size_t>(c) * (D / 8) + 4 * blockIdx.y) * 256 + threadIdx.x) * 8;
  float M = -INFINITY;
  for (int s = 0; s < it.parts; ++s) M = fmaxf(M, pl[static_cast<size_t>(s) * step * 256]);
  float W = 0.f, acc[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) acc[e] = 0.f;
  for (int s = 0; s < it.parts; ++s) {
    const float ls = pl[static_cast<size_t>(s) * step * 256];
    if (ls == -INFINITY) continue;                         // no key: weight 0
    const float w = ex2_approx(ls - M);
    W += w;
#pragma unroll
    for (int e8 = 0; e8 < 4; ++e8) {
      const float4* src = reinterpret_cast<const float4*>(po + (static_cast<size_t>(s) * step * (D / 8) + e8) * 256 * 8);
      const float4 x = src[0], y = src[1];
      const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[8 * e8 + e] = fmaf(w, v[e], acc[8 * e8 + e]);
    }
  }
  const float inv = W != 0.f ? 1.f / W : 0.f;
  const size_t row = (static_cast<size_t>(it.row0) + it.tok[t] + tok) * p.Hq + static_cast<size_t>(it.kvh) * p.G + r % p.G;
  uint4* dst = reinterpret_cast<uint4*>(p.out + row * D + 32 * blockIdx.y);
#pragma unroll
  for (int e8 = 0; e8 < 4; ++e8) {
    const float* a = acc + 8 * e8;
    dst[e8] = make_uint4(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[2] * inv, a[3] * inv),
                         pack_bf16x2(a[4] * inv, a[5] * inv), pack_bf16x2(a[6] * inv, a[7] * inv));
  }
  if (p.lse && blockIdx.y == 0) p.lse[row] = W != 0.f ? (M + __log2f(W)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace wpattn
