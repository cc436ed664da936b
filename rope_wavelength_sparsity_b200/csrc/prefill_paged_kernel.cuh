// Windowed causal attention of a ragged batch of chunks over a paged KV cache.
//
// "ATFlash: Per-RoPE-Wavelength Attention Windows", Abstract: the window is a
// slice of the query-key contraction axis and the online softmax is left
// untouched.  Query t of sequence b sits at kv_len - q_len + t and attends
// the sequence's keys 0 .. its position, found through the block table.
//
// One warp per (token, query head): a lane scores one key of a block of 32
// over the pairs kept at its distance, then the lanes share the block's
// weights and accumulate D / 32 output dims each.
#pragma once

#include "device_util.cuh"

namespace wpattn {

constexpr int kPagedMaxB = 1024;

struct PrefillPagedParams {
  const uint16_t* q;        // [T, Hq, D]
  const uint16_t* k;        // [num_pages, page_size, Hkv, D]
  const uint16_t* v;
  const int32_t* block_table;  // [B, max_pages]
  uint16_t* out;            // [T, Hq, D]
  float* lse;               // [T, Hq] or null
  int B, Hq, Hkv, G, num_pages, page_size, max_pages;
  float scale_log2;         // softmax scale * log2(e)
  int T[64];                // per-pair thresholds, clamped to int32
  int q_start[kPagedMaxB + 1];  // first row of each sequence in q
  int kv_len[kPagedMaxB];
};

// The sequence whose rows cover `token` (start: B + 1 non-decreasing offsets, token < start[B]).
__device__ __forceinline__ int find_sequence(const int* start, int B, int token) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= token) lo = mid; else hi = mid - 1;
  }
  return lo;
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
__global__ void __launch_bounds__(256)
prefill_paged_kernel(const __grid_constant__ PrefillPagedParams p) {
  constexpr int P = D / 2, E = D / 32;
  constexpr uint32_t FULL = 0xffffffffu;
  __shared__ float sq[8][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + warp;
  if (row >= static_cast<int64_t>(p.q_start[p.B]) * p.Hq) return;
  const int token = static_cast<int>(row / p.Hq), h = static_cast<int>(row % p.Hq);
  const int b = find_sequence(p.q_start, p.B, token);
  const int kvh = h / p.G;
  const int pos = p.kv_len[b] - p.q_start[b + 1] + token;   // kv_len - q_len + t
  for (int e = lane; e < D; e += 32) sq[warp][e] = bf16lo_to_f32(p.q[row * D + e]);
  __syncwarp();
  const int32_t* table = p.block_table + static_cast<size_t>(b) * p.max_pages;
  float m = -INFINITY, l = 0.f, o[E] = {};
  for (int j0 = 0; j0 <= pos; j0 += 32) {
    const int j = j0 + lane;
    size_t at = 0;                          // element offset of this lane's key
    float s = -INFINITY;
    if (j <= pos) {
      const int pg = checked_page(table[j / p.page_size], p.num_pages);
      at = ((static_cast<size_t>(pg) * p.page_size + j % p.page_size) * p.Hkv + kvh) * D;
      s = 0.f;
      for (int pp = 0; pp < P; ++pp)
        if (pos - j <= p.T[pp])
          s = fmaf(sq[warp][pp], bf16lo_to_f32(p.k[at + pp]),
                   fmaf(sq[warp][pp + P], bf16lo_to_f32(p.k[at + pp + P]), s));
      s *= p.scale_log2;
    }
    float bm = s;
    for (int off = 16; off > 0; off >>= 1) bm = fmaxf(bm, __shfl_xor_sync(FULL, bm, off));
    const float mn = fmaxf(m, bm);
    const float f = mn == -INFINITY ? 1.f : ex2_approx(m - mn);
    const float w = mn == -INFINITY ? 0.f : ex2_approx(s - mn);
    m = mn;
    l = l * f + w;
    for (int e = 0; e < E; ++e) o[e] *= f;
    for (int i = 0; i < 32 && j0 + i <= pos; ++i) {
      const float wi = __shfl_sync(FULL, w, i);
      const size_t ai = __shfl_sync(FULL, static_cast<unsigned long long>(at), i);
      for (int e = 0; e < E; ++e) o[e] = fmaf(wi, bf16lo_to_f32(p.v[ai + lane + 32 * e]), o[e]);
    }
  }
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(FULL, l, off);
  for (int e = 0; e < E; ++e) {
    const float val = l > 0.f ? o[e] / l : 0.f;
    p.out[row * D + lane + 32 * e] = static_cast<uint16_t>(pack_bf16x2(val, 0.f) & 0xFFFFu);
  }
  if (p.lse && lane == 0)
    p.lse[row] = l > 0.f ? (m + __log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace wpattn
