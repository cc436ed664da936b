// What fills and tends a paged KV cache: RoPE with positions along several
// axes, the append of new keys and values, and page maintenance (copy, fork,
// extend, free, compact).
#pragma once

#include "device_util.cuh"
#include "prefill_paged_kernel.cuh"
#include "rope_kernels.cuh"

namespace wpattn {

constexpr int kMaxAxes = 4;

// ------------------------------------------------------------ rotation and append
// One tensor of a launch: token t's H heads at src + t * src_stride.  They go
// to dst + t * H * D, or, when `paged`, to the token's row of the pool dst.
// rotate: pair p turns by the token's position on the pair's axis.
struct AxesSegment {
  const uint16_t* src;
  uint16_t* dst;
  int64_t src_stride;      // elements between tokens
  int H;
  int rotate, paged;
};

template <int MAXB>
struct AxesParams {
  AxesSegment seg[3];
  int nseg;
  int tokens;
  int ways;                // threads that share a token's batches of heads
  int turn;                // some segment is rotated
  const int32_t* pos;      // [axes, pos_stride], or null: the token's row in its sequence
  int64_t pos_stride;
  int axes;
  float sign;              // -1: the inverse rotation
  uint8_t axis[64];        // axis of each pair
  double theta[64];        // base^(-2p/D)
  // paged destinations
  const int32_t* block_table;
  int B, max_pages, page_size, num_pages;
  int start[MAXB + 1];     // first token of each sequence
  int kv_len[MAXB];        // its rows once the tokens are in
};

// One thread per (token, 8 pairs, way): of the segments' heads, taken HB at a time
// one after another, a thread turns every ways-th batch.  It computes its eight
// angles' cosines and sines once, under its first batch's loads, so one way is
// best once the tokens alone fill the GPU (65000 tokens of 14 + 2 heads of 64:
// 50 us with 1 way, 5.3 TB/s, and 65 us with a thread per batch), and a way per
// batch when they are few (64 tokens: one round trip instead of nine).
template <int D, int MAXB>
__global__ void __launch_bounds__(256) rope_axes_kernel(const __grid_constant__ AxesParams<MAXB> p) {
  constexpr int P = D / 2, NC = P / 8, HB = 4;
  const int b0 = (p.seg[0].H + HB - 1) / HB;                                   // batches up to each segment's end
  const int b1 = b0 + (p.nseg > 1 ? (p.seg[1].H + HB - 1) / HB : 0);
  const int b2 = b1 + (p.nseg > 2 ? (p.seg[2].H + HB - 1) / HB : 0);
  const uint64_t items = static_cast<uint64_t>(p.tokens) * NC * p.ways;
  for (uint64_t idx = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; idx < items;
       idx += static_cast<uint64_t>(gridDim.x) * blockDim.x) {
    const int c = static_cast<int>(idx % NC);
    const int way = static_cast<int>(idx / NC % p.ways);
    const int token = static_cast<int>(idx / NC / p.ways);
    uint4 lo[HB], hi[HB];
    int sg = 0, h0 = 0, nb = 0;            // batch in registers
    auto load = [&](int batch) {
      sg = batch < b0 ? 0 : batch < b1 ? 1 : 2;
      const AxesSegment& g = p.seg[sg];
      h0 = (batch - (sg == 0 ? 0 : sg == 1 ? b0 : b1)) * HB;
      nb = min(HB, g.H - h0);
      const uint16_t* src = g.src + token * g.src_stride + static_cast<int64_t>(h0) * D;
#pragma unroll
      for (int u = 0; u < HB; ++u)
        if (u < nb) {
          lo[u] = *reinterpret_cast<const uint4*>(src + u * D + 8 * c);
          hi[u] = *reinterpret_cast<const uint4*>(src + u * D + P + 8 * c);
        }
    };
    load(way);
    int row = token;                       // the token's row in its sequence, and its pool row (-1: none)
    int64_t pool_row = token;
    if (p.block_table) {
      const int b = find_sequence(p.start, p.B, token);
      row = p.kv_len[b] - p.start[b + 1] + token;
      const int pg = p.block_table[static_cast<int64_t>(b) * p.max_pages + row / p.page_size];
      if (pg < 0 || pg >= p.num_pages) record_status(6 /* WPATTN_EINDEX */);
      pool_row = pg < 0 || pg >= p.num_pages ? -1 : static_cast<int64_t>(pg) * p.page_size + row % p.page_size;
    }
    float cs[8], sn[8];
    if (p.turn) {
      int at[kMaxAxes];
#pragma unroll
      for (int a = 0; a < kMaxAxes; ++a) at[a] = !p.pos ? row : a < p.axes ? p.pos[a * p.pos_stride + token] : 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int ax = p.axis[8 * c + e];
        rope_cos_sin(ax == 0 ? at[0] : ax == 1 ? at[1] : ax == 2 ? at[2] : at[3], p.theta[8 * c + e], cs[e], sn[e]);
        sn[e] *= p.sign;
      }
    }
    for (int batch = way; batch < b2; batch += p.ways) {
      if (batch != way) load(batch);
      const AxesSegment& g = p.seg[sg];
      const int64_t to = g.paged ? pool_row : token;
      if (to < 0) continue;                // nowhere to write
      uint16_t* dst = g.dst + (to * g.H + h0) * D;
#pragma unroll
      for (int u = 0; u < HB; ++u)
        if (u < nb) {
          if (g.rotate) {
            uint32_t a[4] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w}, b[4] = {hi[u].x, hi[u].y, hi[u].z, hi[u].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float y0, y1, z0, z1;
              rope_pair_bf16(bf16lo_to_f32(a[k]), bf16lo_to_f32(b[k]), cs[2 * k], sn[2 * k], y0, z0);
              rope_pair_bf16(bf16hi_to_f32(a[k]), bf16hi_to_f32(b[k]), cs[2 * k + 1], sn[2 * k + 1], y1, z1);
              a[k] = pack_bf16x2(y0, y1);
              b[k] = pack_bf16x2(z0, z1);
            }
            lo[u] = make_uint4(a[0], a[1], a[2], a[3]);
            hi[u] = make_uint4(b[0], b[1], b[2], b[3]);
          }
          *reinterpret_cast<uint4*>(dst + u * D + 8 * c) = lo[u];
          *reinterpret_cast<uint4*>(dst + u * D + P + 8 * c) = hi[u];
        }
    }
  }
}

// ------------------------------------------------------------ page maintenance
// refs[i] counts the block-table entries that name page i; 0 = free.
// Allocation takes the lowest free pages in order, so a call's result does
// not depend on how its threads are scheduled.
constexpr int kMaxPools = 256;
constexpr int kPageRows = 1024;     // table rows one call may name
constexpr int kFewRows = 64;        // up to so many take launches with shorter parameters
constexpr int kScanThreads = 1024;

struct PagePools {
  uint8_t* pool[kMaxPools];
  int n;
};

// Exclusive prefix sum of v over the block; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const int before = warp > 0 ? warp_sums[warp - 1] : 0;
  *total = warp_sums[kScanThreads / 32 - 1];
  __syncthreads();                    // warp_sums may be reused
  return before + x - v;
}

// This block's share of a copy of 16-byte units: four loads ahead of their stores
// (compaction of 1965 pages of 64 KB in 4 pools: 174 us, 5.9 TB/s read and
// written; one load at a time and whole pages per block 208 us).
__device__ __forceinline__ void block_copy(uint8_t* __restrict__ dst, const uint8_t* __restrict__ src, int64_t units) {
  uint4* d = reinterpret_cast<uint4*>(dst);
  const uint4* s = reinterpret_cast<const uint4*>(src);
  for (int64_t i = threadIdx.x; i < units; i += 4 * blockDim.x) {
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * blockDim.x < units) x[k] = s[i + k * blockDim.x];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * blockDim.x < units) d[i + k * blockDim.x] = x[k];
  }
}
constexpr int kCopyUnits = 1024;       // 16-byte units (16 KB) of one page that a block copies at a time

// Source rows of a fork, for the look at their pages' refs.
template <int MAXN>
struct ForkSources {
  const int32_t* table;    // [rows, max_pages]
  int num_pages, max_pages, page_size, n;
  int src[MAXN], len[MAXN];
};

// Block 0: the lowest `want` free pages, in order, into list; -1 where there are fewer.
// The others look at the source rows: a page there that is free may be one of those
// handed out, which the fork itself, whose blocks raise counts in any order, cannot
// tell.  Beside the search they take no time of their own.
template <int MAXN>
__global__ void __launch_bounds__(kScanThreads)
find_free_pages_kernel(const int32_t* __restrict__ refs, int num_pages, int32_t* __restrict__ list, int want,
                       const __grid_constant__ ForkSources<MAXN> p) {
  __shared__ int sums[kScanThreads / 32];
  for (int f = blockIdx.x - 1; f >= 0 && f < p.n; f += gridDim.x - 1) {
    const int pages = (p.len[f] + p.page_size - 1) / p.page_size;
    const int32_t* from = p.table + static_cast<int64_t>(p.src[f]) * p.max_pages;
    for (int j = threadIdx.x; j < pages; j += kScanThreads) {
      const int e = from[j];
      if (e >= 0 && e < num_pages && refs[e] <= 0) record_status(6 /* WPATTN_EINDEX */);
    }
  }
  if (blockIdx.x > 0) return;
  int found = 0;
  for (int base = 0; base < num_pages && found < want; base += kScanThreads) {
    const int i = base + threadIdx.x;
    const int mine = i < num_pages && refs[i] == 0 ? 1 : 0;
    int total;
    const int at = found + block_scan(mine, sums, &total);
    if (mine && at < want) list[at] = i;
    found += total;
  }
  for (int i = found + threadIdx.x; i < want; i += kScanThreads) list[i] = -1;
}

template <int MAXN>
struct ForkParams {
  PagePools pools;
  int32_t* table;          // [rows, max_pages]
  int32_t* refs;
  const int32_t* list;     // a free page for each fork with a begun page, in order
  int num_pages, max_pages, page_size, n;
  int64_t row_bytes;       // bytes of one key's heads in a pool
  int src[MAXN], dst[MAXN], len[MAXN];
  int rank[MAXN];          // index into list, -1: the last page is full
};

// Block (x, f): fork f.  Its table row first (x = 0), then its begun page.
template <int MAXN>
__global__ void __launch_bounds__(256) fork_kernel(const __grid_constant__ ForkParams<MAXN> p) {
  const int f = blockIdx.y;
  const int full = p.len[f] / p.page_size, part = p.len[f] % p.page_size;
  const int32_t* from = p.table + static_cast<int64_t>(p.src[f]) * p.max_pages;
  int32_t* to = p.table + static_cast<int64_t>(p.dst[f]) * p.max_pages;
  const int fresh = part ? p.list[p.rank[f]] : -1;
  if (blockIdx.x == 0) {
    for (int j = threadIdx.x; j < p.max_pages; j += blockDim.x) {
      int e = -1;
      if (j < full) {
        e = from[j];
        if (e < 0 || e >= p.num_pages || atomicAdd(p.refs + e, 1) <= 0) record_status(6 /* WPATTN_EINDEX */);
      } else if (j == full && part) {
        e = fresh;
        if (e < 0) record_status(7 /* WPATTN_EPAGES */);
        else p.refs[e] = 1;
      }
      to[j] = e;
    }
  }
  if (!part || fresh < 0) return;
  const int old = from[full];
  if (old < 0 || old >= p.num_pages) {
    if (threadIdx.x == 0) record_status(6 /* WPATTN_EINDEX */);
    return;
  }
  const int64_t page_bytes = p.row_bytes * p.page_size, units = p.row_bytes * part / 16;
  const int64_t pieces = (units + kCopyUnits - 1) / kCopyUnits;
  for (int64_t i = blockIdx.x; i < pieces * p.pools.n; i += gridDim.x) {
    uint8_t* pool = p.pools.pool[i / pieces];
    const int64_t at = i % pieces * kCopyUnits;
    block_copy(pool + fresh * page_bytes + at * 16, pool + old * page_bytes + at * 16,
               min(static_cast<int64_t>(kCopyUnits), units - at));
  }
}

template <int MAXN>
struct RowsParams {
  int32_t* table;
  int32_t* refs;
  int num_pages, max_pages, page_size, n;
  int row[MAXN], len[MAXN];
};

// Block (x, i): row i gives back its pages and its entries become -1; the last block
// of a row goes on to those that it holds behind its length, up to the first
// entry that names none.  A row of no keys is left as it is.
template <int MAXN>
__global__ void __launch_bounds__(256) free_kernel(const __grid_constant__ RowsParams<MAXN> p) {
  __shared__ int stop;
  const int i = blockIdx.y;
  const int pages = (p.len[i] + p.page_size - 1) / p.page_size;
  int32_t* row = p.table + static_cast<int64_t>(p.row[i]) * p.max_pages;
  auto give_back = [&](int j) {
    const int e = row[j];
    row[j] = -1;
    if (e < 0 || e >= p.num_pages) {
      record_status(6 /* WPATTN_EINDEX */);
    } else if (atomicSub(p.refs + e, 1) <= 0) {
      atomicAdd(p.refs + e, 1);           // it was free already
      record_status(6 /* WPATTN_EINDEX */);
    }
  };
  for (int j = blockIdx.x * blockDim.x + threadIdx.x; j < pages; j += gridDim.x * blockDim.x) give_back(j);
  if (blockIdx.x != gridDim.x - 1 || pages == 0) return;
  for (int j0 = pages; j0 < p.max_pages; j0 += blockDim.x) {
    const int j = j0 + threadIdx.x;
    if (threadIdx.x == 0) stop = p.max_pages;
    __syncthreads();
    if (j < p.max_pages && (row[j] < 0 || row[j] >= p.num_pages)) atomicMin(&stop, j);
    __syncthreads();
    const int end = stop;
    if (j < end) give_back(j);
    if (end < j0 + static_cast<int>(blockDim.x)) return;
    __syncthreads();                      // stop is written again
  }
}

struct ExtendParams {
  int32_t* table;
  int32_t* refs;
  int num_pages, max_pages, n;
  int row[kPageRows], first[kPageRows];   // table row, its first new entry
  int start[kPageRows + 1];               // rank of that entry among the call's
};

// The entries that lack a page get the lowest free ones, in their order.  One that names
// a page in use keeps it: the row holds more pages than its length needs (drafts
// that were not kept).  The threads find those that lack one, up to four entries each
// a round, and scan two rows of 1024 counts at once (in 16 bits each); then the pool's
// refs go by, from where the entries before left them.  Bound by the rounds' latency.
// 64 rows by 500 pages each: 49 us; without the next counts' early loads 55, and with one
// entry a thread and round 65.  1000 rows by one: 13 us; without the early loads 14, and
// with four neighbouring entries a thread 19.  The same with the lowest 900000 of 2^20
// pages in use: 479 us; without the early loads 635.
__global__ void __launch_bounds__(kScanThreads) extend_kernel(const __grid_constant__ ExtendParams p) {
  constexpr int kEach = 4;
  __shared__ int sums[kScanThreads / 32];
  __shared__ int32_t* slots[kScanThreads * kEach];   // the entries that lack a page
  const int want = p.start[p.n];
  // until a call of several rounds ends, a page that it hands out has this count: an entry
  // that a later round looks at and that names the page is then still told from its owner's
  const int taken = want > kScanThreads * kEach ? INT32_MIN : 1;
  int base = 0;                              // every page before it is in use
  for (int r0 = 0; r0 < want; r0 += kScanThreads * kEach) {
    int32_t* entry[kEach];
    int e[kEach];
    bool lacks[kEach];
    int n = 0, got = 0;
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int r = r0 + u * kScanThreads + threadIdx.x;
      lacks[u] = r < want;
      if (!lacks[u]) continue;
      const int i = find_sequence(p.start, p.n, r);
      entry[u] = p.table + static_cast<int64_t>(p.row[i]) * p.max_pages + p.first[i] + r - p.start[i];
      e[u] = *entry[u];
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u)
      if (lacks[u] && e[u] >= 0 && e[u] < p.num_pages) {
        const int held = p.refs[e[u]];
        lacks[u] = held <= 0;
        if (held != 1) record_status(6 /* WPATTN_EINDEX */);   // a free page, or one that others read
      }
#pragma unroll
    for (int u = 0; u < kEach; u += 2) {
      if (r0 + u * kScanThreads >= want) break;
      int total;
      const int at = block_scan((lacks[u] ? 1 : 0) | (lacks[u + 1] ? 1 << 16 : 0), sums, &total);
      if (lacks[u]) slots[n + (at & 0xFFFF)] = entry[u];
      n += total & 0xFFFF;
      if (lacks[u + 1]) slots[n + (at >> 16)] = entry[u + 1];
      n += total >> 16;
    }
    __syncthreads();
    auto count_of = [&](int page) { return page < p.num_pages ? p.refs[page] : 1; };
    int count = count_of(base + threadIdx.x);
    while (got < n && base < p.num_pages) {
      const int page = base + threadIdx.x;
      const int next = count_of(page + kScanThreads);   // under the scan's barriers
      const int free = count == 0 ? 1 : 0;
      int found;
      const int k = got + block_scan(free, sums, &found);
      if (free && k < n) {
        p.refs[page] = taken;
        *slots[k] = page;
      }
      if (got + found <= n) {                // else the next entries take the rest of these
        base += kScanThreads;
        count = next;
      }
      got = min(got + found, n);
    }
    if (got < n && threadIdx.x == 0) record_status(7 /* WPATTN_EPAGES */);
    for (int k = got + threadIdx.x; k < n; k += kScanThreads) *slots[k] = -1;
    __syncthreads();                         // slots may be reused
  }
  if (taken == 1) return;
  const int end = min(base + kScanThreads, p.num_pages);
#pragma unroll 4
  for (int page = threadIdx.x; page < end; page += kScanThreads)
    if (p.refs[page] == taken) p.refs[page] = 1;
}

// ws: [0] live pages, [1] moves; then, num_pages of each: the free slot of rank k,
// the moving page of rank k, and each page's rank among those that move (or -1).
// A thread takes four pages at a time and scans both counts at once (each at
// most 4096 a round, in 16 bits).
__global__ void __launch_bounds__(kScanThreads)
compact_plan_kernel(const int32_t* __restrict__ refs, int num_pages, int32_t* __restrict__ ws,
                    int32_t* __restrict__ live_out) {
  __shared__ int sums[kScanThreads / 32];
  int32_t* slot = ws + 2;
  int32_t* from = slot + num_pages;
  int32_t* rank = from + num_pages;
  int total, mine = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < num_pages; i += kScanThreads) mine += refs[i] > 0 ? 1 : 0;
  block_scan(mine, sums, &total);
  const int live = total;
  int holes = 0, moves = 0;
  for (int base = 0; base < num_pages; base += 4 * kScanThreads) {
    const int i0 = base + 4 * threadIdx.x;
    bool hole[4], move[4];
    int both = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool used = i0 + k < num_pages && refs[i0 + k] > 0;
      hole[k] = i0 + k < live && !used;
      move[k] = i0 + k >= live && used;
      both += (hole[k] ? 1 : 0) | (move[k] ? 1 << 16 : 0);
    }
    const int at = block_scan(both, sums, &total);
    int ah = holes + (at & 0xFFFF), am = moves + (at >> 16);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + k < num_pages) {
        if (hole[k]) slot[ah++] = i0 + k;
        rank[i0 + k] = move[k] ? am : -1;
        if (move[k]) from[am++] = i0 + k;
      }
    holes += total & 0xFFFF;
    moves += total >> 16;
  }
  if (threadIdx.x == 0) {
    ws[0] = live;
    ws[1] = moves;
    if (live_out) *live_out = live;
  }
}

struct CompactParams {
  PagePools pools;
  int32_t* table;
  int32_t* refs;
  const int32_t* ws;
  int num_pages;
  int64_t entries;         // of the whole table
  int64_t page_bytes;
};

// Blocks take pieces of the moving pages in turn; then the table's entries and the
// refs follow.
__global__ void __launch_bounds__(256) compact_kernel(const __grid_constant__ CompactParams p) {
  const int32_t* slot = p.ws + 2;
  const int32_t* from = slot + p.num_pages;
  const int32_t* rank = from + p.num_pages;
  const int64_t moves = p.ws[1], units = p.page_bytes / 16, pieces = (units + kCopyUnits - 1) / kCopyUnits;
  for (int64_t i = blockIdx.x; i < moves * p.pools.n * pieces; i += gridDim.x) {
    const int64_t page = i / pieces % moves;
    uint8_t* pool = p.pools.pool[i / pieces / moves];
    const int64_t at = i % pieces * kCopyUnits;
    block_copy(pool + slot[page] * p.page_bytes + at * 16, pool + from[page] * p.page_bytes + at * 16,
               min(static_cast<int64_t>(kCopyUnits), units - at));
  }
  const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t k = first; k < moves; k += stride) {
    p.refs[slot[k]] = p.refs[from[k]];
    p.refs[from[k]] = 0;
  }
  for (int64_t e = first; e < p.entries; e += stride) {
    const int pg = p.table[e];
    if (pg >= 0 && pg < p.num_pages && rank[pg] >= 0) p.table[e] = slot[rank[pg]];
  }
}

struct CopyParams {
  PagePools pools;
  const int32_t* src;      // [n] pages
  const int32_t* dst;
  int n, num_pages;
  int64_t page_bytes;
};

// Block (x, pool): copies pages in turn.
__global__ void __launch_bounds__(256) copy_pages_kernel(const __grid_constant__ CopyParams p) {
  uint8_t* pool = p.pools.pool[blockIdx.y];
  for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
    const int s = p.src[i], d = p.dst[i];
    if (s < 0 || s >= p.num_pages || d < 0 || d >= p.num_pages) {
      if (threadIdx.x == 0) record_status(6 /* WPATTN_EINDEX */);
      continue;
    }
    block_copy(pool + d * p.page_bytes, pool + s * p.page_bytes, p.page_bytes / 16);
  }
}

}  // namespace wpattn
