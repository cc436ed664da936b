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

// One thread per (token, 8 pairs, segment, HB heads): the eight angles are
// turned into cosines and sines once per thread; both 16-byte halves of up to
// HB heads are loaded ahead of them.
template <int D, int MAXB>
__global__ void __launch_bounds__(256) rope_axes_kernel(const __grid_constant__ AxesParams<MAXB> p) {
  constexpr int P = D / 2, NC = P / 8, HB = 4;
  int groups[3], per = 0;                 // head groups of each segment
  for (int s = 0; s < 3; ++s) {
    groups[s] = s < p.nseg ? (p.seg[s].H + HB - 1) / HB : 0;
    per += groups[s];
  }
  const uint64_t items = static_cast<uint64_t>(p.tokens) * NC * per;
  for (uint64_t idx = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; idx < items;
       idx += static_cast<uint64_t>(gridDim.x) * blockDim.x) {
    const int c = static_cast<int>(idx % NC);
    int hg = static_cast<int>(idx / NC % per), sg = 0;
    const int token = static_cast<int>(idx / (static_cast<uint64_t>(NC) * per));
    while (hg >= groups[sg]) hg -= groups[sg++];
    const AxesSegment& g = p.seg[sg];
    const int h0 = hg * HB, nb = min(HB, g.H - h0);
    const uint16_t* src = g.src + token * g.src_stride + static_cast<int64_t>(h0) * D;
    uint4 lo[HB], hi[HB];
#pragma unroll
    for (int u = 0; u < HB; ++u)
      if (u < nb) {
        lo[u] = *reinterpret_cast<const uint4*>(src + u * D + 8 * c);
        hi[u] = *reinterpret_cast<const uint4*>(src + u * D + P + 8 * c);
      }
    int row = token;                      // the token's row in its sequence, and its pool row
    int64_t to = token;
    if (p.block_table) {
      const int b = find_sequence(p.start, p.B, token);
      row = p.kv_len[b] - p.start[b + 1] + token;
      if (g.paged) {
        const int pg = p.block_table[static_cast<int64_t>(b) * p.max_pages + row / p.page_size];
        if (pg < 0 || pg >= p.num_pages) {
          record_status(6 /* WPATTN_EINDEX */);
          continue;                       // nowhere to write
        }
        to = static_cast<int64_t>(pg) * p.page_size + row % p.page_size;
      }
    }
    uint16_t* dst = g.dst + (to * g.H + h0) * D;
    float cs[8], sn[8];
    if (g.rotate) {
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

// ------------------------------------------------------------ page maintenance
// refs[i] counts the block-table entries that name page i; 0 = free.
// Allocation takes the lowest free pages in order, so a call's result does
// not depend on how its threads are scheduled.
constexpr int kMaxPools = 256;
constexpr int kPageRows = 1024;     // table rows one call may name
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

// The lowest `want` free pages, in order, into list; -1 where there are fewer.
__global__ void __launch_bounds__(kScanThreads)
find_free_pages_kernel(const int32_t* __restrict__ refs, int num_pages, int32_t* __restrict__ list, int want) {
  __shared__ int sums[kScanThreads / 32];
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

struct ForkParams {
  PagePools pools;
  int32_t* table;          // [rows, max_pages]
  int32_t* refs;
  const int32_t* list;     // a free page for each fork with a begun page, in order
  int num_pages, max_pages, page_size, n;
  int64_t row_bytes;       // bytes of one key's heads in a pool
  int src[kPageRows], dst[kPageRows], len[kPageRows];
  int rank[kPageRows];     // index into list, -1: the last page is full
};

// Block (x, f): fork f.  Its table row first (x = 0), then its begun page.
__global__ void __launch_bounds__(256) fork_kernel(const __grid_constant__ ForkParams p) {
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
        if (e < 0 || e >= p.num_pages) record_status(6 /* WPATTN_EINDEX */);
        else atomicAdd(p.refs + e, 1);
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
  const int64_t page_bytes = p.row_bytes * p.page_size, chunks = p.row_bytes * part / 16;
  const int64_t all = chunks * p.pools.n;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < all;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    uint8_t* pool = p.pools.pool[i / chunks];
    const int64_t at = i % chunks * 16;
    *reinterpret_cast<uint4*>(pool + fresh * page_bytes + at) =
        *reinterpret_cast<const uint4*>(pool + old * page_bytes + at);
  }
}

struct RowsParams {
  int32_t* table;
  int32_t* refs;
  int num_pages, max_pages, page_size, n;
  int row[kPageRows], len[kPageRows];
};

// Block (x, i): row i gives back its pages and its entries become -1.
__global__ void __launch_bounds__(256) free_kernel(const __grid_constant__ RowsParams p) {
  const int i = blockIdx.y;
  const int pages = (p.len[i] + p.page_size - 1) / p.page_size;
  int32_t* row = p.table + static_cast<int64_t>(p.row[i]) * p.max_pages;
  for (int j = blockIdx.x * blockDim.x + threadIdx.x; j < pages; j += gridDim.x * blockDim.x) {
    const int e = row[j];
    row[j] = -1;
    if (e < 0 || e >= p.num_pages) {
      record_status(6 /* WPATTN_EINDEX */);
    } else if (atomicSub(p.refs + e, 1) <= 0) {
      atomicAdd(p.refs + e, 1);           // it was free already
      record_status(6 /* WPATTN_EINDEX */);
    }
  }
}

struct ExtendParams {
  int32_t* table;
  int32_t* refs;
  int num_pages, max_pages, n;
  int row[kPageRows], first[kPageRows];   // table row, its first new entry
  int start[kPageRows + 1];               // rank of that entry among the call's new pages
};

// Rank r among the call's new pages gets the r-th lowest free page.
__global__ void __launch_bounds__(kScanThreads) extend_kernel(const __grid_constant__ ExtendParams p) {
  __shared__ int sums[kScanThreads / 32];
  const int want = p.start[p.n];
  auto put = [&](int rank, int page) {
    const int i = find_sequence(p.start, p.n, rank);
    p.table[static_cast<int64_t>(p.row[i]) * p.max_pages + p.first[i] + rank - p.start[i]] = page;
  };
  int found = 0;
  for (int base = 0; base < p.num_pages && found < want; base += kScanThreads) {
    const int i = base + threadIdx.x;
    const int mine = i < p.num_pages && p.refs[i] == 0 ? 1 : 0;
    int total;
    const int at = found + block_scan(mine, sums, &total);
    if (mine && at < want) {
      p.refs[i] = 1;
      put(at, i);
    }
    found += total;
  }
  if (found < want && threadIdx.x == 0) record_status(7 /* WPATTN_EPAGES */);
  for (int r = found + threadIdx.x; r < want; r += kScanThreads) put(r, -1);
}

// ws: [0] live pages, [1] moves, then per page: free slot of rank k at
// ws[2 + k], and rank of a page that moves (or -1) at ws[2 + num_pages + page].
__global__ void __launch_bounds__(kScanThreads)
compact_plan_kernel(const int32_t* __restrict__ refs, int num_pages, int32_t* __restrict__ ws,
                    int32_t* __restrict__ live_out) {
  __shared__ int sums[kScanThreads / 32];
  int total, mine = 0;
  for (int i = threadIdx.x; i < num_pages; i += kScanThreads) mine += refs[i] > 0 ? 1 : 0;
  block_scan(mine, sums, &total);
  const int live = total;
  int holes = 0, moves = 0;
  for (int base = 0; base < num_pages; base += kScanThreads) {
    const int i = base + threadIdx.x;
    const bool used = i < num_pages && refs[i] > 0;
    const int hole = i < live && !used ? 1 : 0, move = i >= live && used ? 1 : 0;
    int th, tm;
    const int ah = holes + block_scan(hole, sums, &th), am = moves + block_scan(move, sums, &tm);
    if (hole) ws[2 + ah] = i;
    if (i < num_pages) ws[2 + num_pages + i] = move ? am : -1;
    holes += th;
    moves += tm;
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

// Blocks take pages in turn and move those that the plan moves; then the
// table's entries follow.
__global__ void __launch_bounds__(256) compact_kernel(const __grid_constant__ CompactParams p) {
  const int32_t* slot = p.ws + 2;
  const int32_t* rank = p.ws + 2 + p.num_pages;
  for (int i = blockIdx.x; i < p.num_pages; i += gridDim.x) {
    if (rank[i] < 0) continue;
    const int to = slot[rank[i]];
    for (int n = 0; n < p.pools.n; ++n) {
      const uint8_t* s = p.pools.pool[n] + i * p.page_bytes;
      uint8_t* d = p.pools.pool[n] + to * p.page_bytes;
      for (int64_t at = threadIdx.x * 16; at < p.page_bytes; at += blockDim.x * 16)
        *reinterpret_cast<uint4*>(d + at) = *reinterpret_cast<const uint4*>(s + at);
    }
    if (threadIdx.x == 0) {
      p.refs[to] = p.refs[i];
      p.refs[i] = 0;
    }
  }
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < p.entries;
       e += static_cast<int64_t>(gridDim.x) * blockDim.x) {
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
    for (int64_t at = threadIdx.x * 16; at < p.page_bytes; at += blockDim.x * 16)
      *reinterpret_cast<uint4*>(pool + d * p.page_bytes + at) =
          *reinterpret_cast<const uint4*>(pool + s * p.page_bytes + at);
  }
}

}  // namespace wpattn
