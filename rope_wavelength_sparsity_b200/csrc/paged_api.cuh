// C ABI of the paged-cache operators (declarations and contracts in
// include/wpattn.h): argument checks and launches.  Included by api.cu.
#pragma once

#include "paged_kernels.cuh"
#include "prefill_paged_kernel.cuh"

namespace wpattn {
namespace {

int launched() { return cudaGetLastError() == cudaSuccess ? WPATTN_OK : WPATTN_ECUDA; }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// a 32-key block is one page, a part of one page, or a whole number of pages
bool page_size_ok(int page_size) {
  return page_size == 8 || page_size == 16 || (page_size > 0 && page_size % 32 == 0);
}

template <int MAXB>
int launch_rope_axes(AxesParams<MAXB>& p, int D, int num_sms, cudaStream_t st) {
  int batches = 0;
  for (int s = 0; s < p.nseg; ++s) {
    batches += (p.seg[s].H + 3) / 4;
    p.turn |= p.seg[s].rotate;
  }
  // about an eighth of the GPU's threads at least (8100 tokens of 28 + 4 + 4 heads of 128: 27.5 us with one way, 34.5
  // with two, 30.5 with three)
  const uint64_t one = static_cast<uint64_t>(p.tokens) * (D / 16), enough = static_cast<uint64_t>(num_sms) * 256;
  if (one == 0) return WPATTN_OK;
  p.ways = static_cast<int>(std::min<uint64_t>(batches, (enough + one - 1) / one));
  const uint64_t items = one * p.ways;
  const unsigned grid = static_cast<unsigned>(std::min<uint64_t>((items + 255) / 256, static_cast<uint64_t>(num_sms) * 8));
  if (D == 64) rope_axes_kernel<64, MAXB><<<grid, 256, 0, st>>>(p);
  else rope_axes_kernel<128, MAXB><<<grid, 256, 0, st>>>(p);
  return launched();
}

// arguments that the rotating entry points share (positions of no token may be NULL, as an empty tensor's are)
bool axes_ok(int D, int64_t tokens, const int32_t* positions, int64_t pos_stride, int32_t axes,
             const uint8_t* pair_axis, double base) {
  if (!(base > 1.0) || std::isinf(base) || axes < 1 || axes > kMaxAxes) return false;
  if (!positions && axes != 1 && tokens > 0) return false;
  if (positions && (!aligned4(positions) || (axes > 1 && pos_stride < tokens))) return false;
  for (int i = 0; pair_axis && i < D / 2; ++i)
    if (pair_axis[i] >= axes) return false;
  return true;
}

template <int MAXB>
void set_axes(AxesParams<MAXB>& p, int D, const int32_t* positions, int64_t pos_stride, int32_t axes,
              const uint8_t* pair_axis, double base) {
  for (int i = 0; i < D / 2; ++i) p.axis[i] = pair_axis ? pair_axis[i] : 0;
  p.pos = positions;
  p.pos_stride = pos_stride;
  p.axes = axes;
  rope_thetas(base, D, p.theta);
}

// pools of a page operator: every pointer present and 16-byte aligned, a page a multiple of 16 bytes
int set_pools(PagePools* out, void* const* pools, int32_t n_pools, int64_t page_bytes) {
  if (n_pools < 0 || (n_pools > 0 && !pools) || page_bytes <= 0 || page_bytes % 16 != 0) return WPATTN_EINVAL;
  if (n_pools > kMaxPools) return WPATTN_EUNSUPPORTED;
  std::memset(out, 0, sizeof *out);
  out->n = n_pools;
  for (int i = 0; i < n_pools; ++i) {
    if (!pools[i] || !aligned16(pools[i])) return WPATTN_EINVAL;
    out->pool[i] = static_cast<uint8_t*>(pools[i]);
  }
  return WPATTN_OK;
}

// what the page kernels' 32-bit loops and the rounding up to whole pages can take
bool page_counts_ok(int32_t num_pages, int32_t page_size, int32_t max_pages) {
  return num_pages <= (1 << 30) && int64_t(max_pages) * page_size <= (int64_t(1) << 30);
}

// 1 <= n <= kPageRows rows named once each, inside the table; sorted into `sorted`
bool rows_ok(const int32_t* rows, int32_t n, int32_t num_rows, int32_t (&sorted)[kPageRows]) {
  std::copy(rows, rows + n, sorted);
  std::sort(sorted, sorted + n);
  return sorted[0] >= 0 && sorted[n - 1] < num_rows && std::adjacent_find(sorted, sorted + n) == sorted + n;
}

template <int MAXB>
int append_impl(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const void* q,
                int64_t q_stride, void* q_out, void* k_pages, void* v_pages, int32_t num_pages,
                int32_t page_size, const int32_t* block_table, int32_t max_pages, const int32_t* new_len,
                const int32_t* kv_len, int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t tokens,
                const int32_t* positions, int64_t pos_stride, int32_t axes, const uint8_t* pair_axis,
                double base, int num_sms, cudaStream_t st) {
  AxesParams<MAXB> p;
  std::memset(&p, 0, sizeof p);
  p.tokens = tokens;
  p.sign = 1.f;
  p.seg[0] = AxesSegment{static_cast<const uint16_t*>(k), static_cast<uint16_t*>(k_pages), k_stride, Hkv, base != 0.0, 1};
  p.seg[1] = AxesSegment{static_cast<const uint16_t*>(v), static_cast<uint16_t*>(v_pages), v_stride, Hkv, 0, 1};
  p.nseg = 2;
  if (q) p.seg[p.nseg++] = AxesSegment{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(q_out), q_stride, Hq, 1, 0};
  if (base != 0.0) set_axes(p, D, positions, pos_stride, axes, pair_axis, base);
  p.block_table = block_table;
  p.B = B;
  p.max_pages = max_pages;
  p.page_size = page_size;
  p.num_pages = num_pages;
  for (int b = 0; b < B; ++b) {
    p.start[b + 1] = p.start[b] + new_len[b];
    p.kv_len[b] = kv_len[b];
  }
  return launch_rope_axes(p, D, num_sms, st);
}

// sum of B lengths of at least 0; -1 when one is negative or the sum passes int32
int64_t sum_lengths(const int32_t* len, int32_t B) {
  int64_t sum = 0;
  for (int b = 0; b < B; ++b) {
    if (len[b] < 0) return -1;
    sum += len[b];
  }
  return sum <= INT32_MAX ? sum : -1;
}

// tokens of a prefill: rounded up to whole row tiles (of at most 128) they still fit 32 bits
constexpr int64_t kMaxTokens = INT32_MAX - 127;

template <int MAXN>
int launch_fork(const PagePools& pools, int num_pages, int page_size, int64_t row_bytes, int32_t* table,
                int max_pages, int32_t* refs, const int32_t* src, const int32_t* dst, const int32_t* len, int n,
                int32_t* list, int num_sms, cudaStream_t st) {
  ForkParams<MAXN> p;
  p.pools = pools;
  int begun = 0, most = 0;
  for (int i = 0; i < n; ++i) {
    p.src[i] = src[i];
    p.dst[i] = dst[i];
    p.len[i] = len[i];
    p.rank[i] = len[i] % page_size ? begun++ : -1;
    most = std::max(most, len[i] % page_size);
  }
  if (begun > 0) {
    ForkSources<MAXN> from;
    from.table = table;
    from.num_pages = num_pages; from.max_pages = max_pages; from.page_size = page_size; from.n = n;
    std::copy(src, src + n, from.src);
    std::copy(len, len + n, from.len);
    find_free_pages_kernel<MAXN><<<1 + n, kScanThreads, 0, st>>>(refs, num_pages, list, begun, from);
    const int rc = launched();
    if (rc != WPATTN_OK) return rc;
  }
  p.table = table; p.refs = refs; p.list = list;
  p.num_pages = num_pages; p.max_pages = max_pages; p.page_size = page_size; p.n = n;
  p.row_bytes = row_bytes;
  // 16 KB of copies a block, at most about eight blocks an SM
  const int64_t per_fork = row_bytes * most * pools.n;
  const int64_t x = std::max<int64_t>(1, std::min<int64_t>((per_fork + 16383) / 16384, int64_t(num_sms) * 8 / n + 1));
  fork_kernel<MAXN><<<dim3(static_cast<unsigned>(x), n), 256, 0, st>>>(p);
  return launched();
}

template <int MAXN>
int launch_free(int num_pages, int page_size, int32_t* table, int max_pages, int32_t* refs, const int32_t* rows,
                const int32_t* len, int n, int most_pages, cudaStream_t st) {
  RowsParams<MAXN> p;
  std::copy(rows, rows + n, p.row);
  std::copy(len, len + n, p.len);
  p.table = table; p.refs = refs;
  p.num_pages = num_pages; p.max_pages = max_pages; p.page_size = page_size; p.n = n;
  free_kernel<MAXN><<<dim3((most_pages + 255) / 256, n), 256, 0, st>>>(p);
  return launched();
}

// ------------------------------------------------------------ prefill_paged: plan and launch
// Which CTAs run a call: sequences in order, each with the parts its row
// blocks' key ranges are cut into; those with several parts come first.
struct PagedPlan {
  int n = 0, ctas = 0, split_ctas = 0;
  uint16_t seq[kPagedMaxB], parts[kPagedMaxB], lead[kPagedMaxB];
  int item0[kPagedMaxB + 1];
  size_t bytes(int D) const { return static_cast<size_t>(split_ctas) * 256 * (D + 1) * sizeof(float); }
};

// Time of `count[i]` CTAs of cost[i] each, in that order, on `slots` SMs that each
// take the next CTA when free.  SMs that are free at the same time are kept
// together, so the work is in the number of distinct times.
float wave_time(const int* count, const float* cost, int n, int slots) {
  struct Level { float t; int k; };
  Level lv[64];
  int m = 1;
  lv[0] = Level{0.f, slots};
  float rest = 0.f;                       // work beyond the bookkeeping's bound, spread evenly
  int turns = 0;
  for (int i = 0; i < n; ++i) {
    int left = count[i];
    while (left > 0) {
      if (++turns > 400 || m >= 63) { rest += left * cost[i] / slots; break; }
      const int k = std::min(left, lv[0].k);
      left -= k;
      const float t = lv[0].t + cost[i];
      if ((lv[0].k -= k) == 0) { --m; std::copy(lv + 1, lv + 1 + m, lv); }
      int at = m;
      while (at > 0 && lv[at - 1].t > t) --at;
      if (at > 0 && lv[at - 1].t == t) { lv[at - 1].k += k; continue; }
      std::copy_backward(lv + at, lv + m, lv + m + 1);
      lv[at] = Level{t, k};
      ++m;
    }
  }
  return lv[m - 1].t + rest;
}

// Measured costs in microseconds, [row tiles of a block - 1]: a key tile of 128
// keys (D = 64, 128), a CTA's start and end, each threshold that the walk
// passes (most lie within kLeadKeys of the diagonal, so the part of the last
// keys is made shorter by them), and the merge pass.
constexpr float kTileUs[2][2] = {{0.95f, 1.75f}, {1.4f, 2.1f}};
constexpr float kCtaUs[2] = {7.f, 10.f}, kPairUs[2] = {0.8f, 1.5f}, kMergeUs = 5.f;
constexpr int kMinPartTiles = 2, kMaxParts = 64, kLeadKeys = 1024;

// The length of a part is the one whose grid these costs say is done first, out
// of some that make a fraction of a wave to a dozen waves of the whole work, and
// no split at all.
bool plan_paged(const int32_t* q_len, const int32_t* kv_len, int B, int G, int Hkv, const WindowPlan& window,
                int num_sms, PagedPlan* out) {
  const int tile_tokens = 128 / G;
  struct Work { int b, blocks, nkt, lead; float tile, us, cta; };
  Work w[kPagedMaxB];
  int n = 0;
  double total = 0;
  for (int b = 0; b < B; ++b) {
    if (q_len[b] == 0) continue;
    const int tiles = (q_len[b] + tile_tokens - 1) / tile_tokens, two = tiles > 1 ? 1 : 0;
    const float tile = kTileUs[window.D == 128][two];
    int passed = 0;
    for (int i = 0; i < window.P; i += window.g)
      passed += window.T[i] < std::min(kv_len[b], kLeadKeys) ? 1 : 0;
    Work& x = w[n++];
    x = Work{b, (tiles + 1) / 2, (kv_len[b] + 127) / 128, static_cast<int>(passed * kPairUs[two] / tile), tile, 0.f,
             kCtaUs[two]};
    x.us = (x.nkt + x.lead) * tile;
    total += static_cast<double>(x.blocks) * Hkv * x.us;
  }
  // longest rows first
  std::sort(w, w + n, [](const Work& a, const Work& b) { return a.us != b.us ? a.us > b.us : a.b < b.b; });
  auto parts_of = [&](const Work& x, double us) {   // parts of about `us` each
    const int tiles = static_cast<int>(std::max<double>(kMinPartTiles, std::min(us / x.tile, 1e9)));
    const int parts = std::min(kMaxParts, (x.nkt + x.lead + tiles - 1) / tiles);
    return std::max(1, std::min(parts, x.nkt / kMinPartTiles));
  };
  // tiles that the last part is shorter by, at most so many that it keeps one
  auto lead_of = [&](const Work& x, int parts) {
    return parts < 2 ? 0 : std::max(0, std::min(x.lead, (x.nkt - 1) / (parts - 1) * parts - x.nkt));
  };
  auto cta_us = [&](const Work& x, int parts) {   // of a row block's longest part
    const int per = (x.nkt + lead_of(x, parts) + parts - 1) / parts;
    return std::max(per, x.nkt - (parts - 1) * per + x.lead) * x.tile + x.cta;
  };
  int count[kPagedMaxB];
  float cost[kPagedMaxB];
  double best_us = 1e12;
  float best = 0;
  constexpr float kWaves[] = {0.f, 0.4f, 0.5f, 0.6f, 0.7f, 0.8f, 0.9f, 1.f, 1.2f, 1.5f, 1.8f, 2.f, 2.5f, 3.f, 4.f, 5.f, 7.f, 9.f, 12.f};
  for (const float k : kWaves) {
    const double us = k == 0 ? 1e12 : total / (static_cast<double>(num_sms) * k);
    if (k > 0 && n > 0 && us >= w[0].us) continue;  // nothing would be split
    int m = 0;
    bool split = false;
    for (int i = 0; i < n; ++i) {
      const int parts = parts_of(w[i], us);
      const float c = cta_us(w[i], parts);
      const int64_t ctas = int64_t(w[i].blocks) * Hkv * parts;
      split |= parts > 1;
      if (ctas > INT32_MAX / 2) return false;
      if (m > 0 && cost[m - 1] == c && count[m - 1] < INT32_MAX / 2) count[m - 1] += static_cast<int>(ctas);
      else { cost[m] = c; count[m++] = static_cast<int>(ctas); }
    }
    const float t = wave_time(count, cost, m, num_sms) + (split ? kMergeUs : 0.f);
    if (k == 0 || t < best) { best = t; best_us = us; }
  }
  // split sequences first: only their CTAs have room in the workspace
  int64_t ctas = 0;
  out->n = 0;
  for (int pass = 0; pass < 2; ++pass) {
    for (int i = 0; i < n; ++i) {
      const int parts = parts_of(w[i], best_us);
      if ((parts > 1) != (pass == 0)) continue;
      out->item0[out->n] = static_cast<int>(ctas);
      out->seq[out->n] = static_cast<uint16_t>(w[i].b);
      out->lead[out->n] = static_cast<uint16_t>(lead_of(w[i], parts));
      out->parts[out->n++] = static_cast<uint16_t>(parts);
      ctas += int64_t(w[i].blocks) * Hkv * parts;
      if (ctas > INT32_MAX) return false;
    }
    if (pass == 0) out->split_ctas = static_cast<int>(ctas);
  }
  out->item0[out->n] = out->ctas = static_cast<int>(ctas);
  return true;
}

struct PagedCall {
  DeviceInfo* dev;
  PagedPlan plan;
  const WindowPlan* window;
  const void *q, *k, *v;
  void *out, *workspace;
  float* lse;
  const int32_t *block_table, *q_len, *kv_len;
  int num_pages, page_size, max_pages, B, Hq, Hkv;
  float scale;
  cudaStream_t st;
};

template <int D, bool G8, int MAXB>
int launch_paged(const PagedCall& c) {
  using L = PagedSmem<D>;
  PrefillPagedParams<MAXB> p;
  std::memset(&p, 0, sizeof p);
  p.q = static_cast<const uint16_t*>(c.q);
  p.block_table = c.block_table;
  p.out = static_cast<uint16_t*>(c.out);
  p.lse = c.lse;
  p.part_o = static_cast<float*>(c.workspace);
  p.part_l = p.part_o + static_cast<size_t>(c.plan.split_ctas) * 256 * D;
  p.B = c.plan.n; p.Hq = c.Hq; p.Hkv = c.Hkv; p.G = c.Hq / c.Hkv;
  p.num_pages = c.num_pages; p.page_size = c.page_size; p.max_pages = c.max_pages;
  p.unit = std::min(128, c.page_size & -c.page_size);
  p.tile_tokens = 128 / p.G;
  p.scale_log2 = c.scale * 1.44269504088896340736f;
  for (int i = 0; i < 64; ++i)
    p.T[i] = c.window->T[i] > INT32_MAX ? INT32_MAX : static_cast<int>(c.window->T[i]);
  std::copy(c.plan.item0, c.plan.item0 + c.plan.n + 1, p.item0);
  std::copy(c.plan.seq, c.plan.seq + c.plan.n, p.seq);
  std::copy(c.plan.parts, c.plan.parts + c.plan.n, p.parts);
  std::copy(c.plan.lead, c.plan.lead + c.plan.n, p.lead);
  for (int b = 0; b < c.B; ++b) {
    p.q_start[b + 1] = p.q_start[b] + c.q_len[b];
    p.kv_len[b] = c.kv_len[b];
  }
  // pools as groups of 8 keys: (64 dims, 8 keys, panels of every head, groups)
  const cuuint64_t row = static_cast<cuuint64_t>(c.Hkv) * D * 2;
  const cuuint64_t dims[4] = {64, 8, static_cast<cuuint64_t>(c.Hkv) * (D / 64),
                              static_cast<cuuint64_t>(c.num_pages) * c.page_size / 8};
  const cuuint64_t strides[3] = {row, 128, 8 * row};
  const cuuint32_t box[4] = {64, 8, D / 64, static_cast<cuuint32_t>(p.unit / 8)}, estr[4] = {1, 1, 1, 1};
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return WPATTN_ECUDA;
  CUtensorMap maps[2];
  for (int i = 0; i < 2; ++i)
    if (enc(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(i ? c.v : c.k), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return WPATTN_ECUDA;
  const auto kernel = prefill_paged_kernel<D, G8, MAXB>;
  static std::atomic<bool> attr_set[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return WPATTN_ECUDA;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC) != cudaSuccess)
      return WPATTN_ECUDA;
    attr_set[dev].store(true, std::memory_order_release);
  }
  kernel<<<c.plan.ctas, 384, L::ALLOC, c.st>>>(maps[0], maps[1], p);
  const int rc = launched();
  if (rc != WPATTN_OK || c.plan.split_ctas == 0) return rc;
  // launched while the parts' kernel runs; it waits for that kernel's end by itself
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c.plan.split_ctas, D / 32);
  cfg.blockDim = dim3(256);
  cfg.stream = c.st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_paged_merge_kernel<D, MAXB>, p) == cudaSuccess ? launched() : WPATTN_ECUDA;
}

template <int D, bool G8>
int run_paged(const PagedCall& c) {
  // a launch copies its parameters: 17 KB for 1024 sequences, 1.5 KB for 64
  return c.B <= 64 ? launch_paged<D, G8, 64>(c) : launch_paged<D, G8, kPagedMaxB>(c);
}

}  // namespace
}  // namespace wpattn

extern "C" {

int wpattn_rope_axes(const void* q, int64_t q_stride, void* q_out, const void* k, int64_t k_stride,
                     void* k_out, int32_t tokens, int32_t Hq, int32_t Hkv, int32_t head_dim,
                     const int32_t* positions, int64_t pos_stride, int32_t axes, const uint8_t* pair_axis_host,
                     double rope_base, int32_t inverse, void* cuda_stream) {
  if (tokens < 0 || Hq <= 0 || (k && Hkv <= 0) || (!k != !k_out)) return WPATTN_EINVAL;
  if (head_dim != 64 && head_dim != 128) return WPATTN_EUNSUPPORTED;
  if ((!positions && tokens > 0) || (inverse != 0 && inverse != 1) ||
      !axes_ok(head_dim, tokens, positions, pos_stride, axes, pair_axis_host, rope_base))
    return WPATTN_EINVAL;
  if (tokens == 0) return WPATTN_OK;
  if (!q || !q_out || !aligned16(q) || !aligned16(q_out) || q_stride < int64_t(Hq) * head_dim || q_stride % 8)
    return WPATTN_EINVAL;
  if (k && (!aligned16(k) || !aligned16(k_out) || k_stride < int64_t(Hkv) * head_dim || k_stride % 8))
    return WPATTN_EINVAL;
  DeviceInfo* dev = nullptr;
  int rc;
  if ((rc = device_info(&dev)) != WPATTN_OK) return rc;
  AxesParams<1> p;
  std::memset(&p, 0, sizeof p);
  p.tokens = tokens;
  p.sign = inverse ? -1.f : 1.f;
  set_axes(p, head_dim, positions, pos_stride, axes, pair_axis_host, rope_base);
  p.seg[0] = AxesSegment{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(q_out), q_stride, Hq, 1, 0};
  p.nseg = 1;
  if (k) p.seg[p.nseg++] = AxesSegment{static_cast<const uint16_t*>(k), static_cast<uint16_t*>(k_out), k_stride, Hkv, 1, 0};
  return launch_rope_axes(p, head_dim, dev->num_sms, static_cast<cudaStream_t>(cuda_stream));
}

int wpattn_append_paged(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const void* q,
                        int64_t q_stride, void* q_out, void* k_pages, void* v_pages, int32_t num_pages,
                        int32_t page_size, const int32_t* block_table, int32_t max_pages_per_seq,
                        const int32_t* new_len_host, const int32_t* kv_len_host, int32_t B, int32_t Hq,
                        int32_t Hkv, int32_t head_dim, const int32_t* positions, int64_t pos_stride,
                        int32_t axes, const uint8_t* pair_axis_host, double rope_base, void* cuda_stream) {
  if (B < 0 || Hkv <= 0 || (!q != !q_out) || (q && Hq <= 0)) return WPATTN_EINVAL;
  if (head_dim != 64 && head_dim != 128) return WPATTN_EUNSUPPORTED;
  if (rope_base == 0.0 && (q || positions || pair_axis_host)) return WPATTN_EINVAL;  // nothing would turn them
  if (!page_size_ok(page_size) || B > kPagedMaxB) return WPATTN_EUNSUPPORTED;
  if (B == 0) return WPATTN_OK;
  if (!new_len_host || !kv_len_host || num_pages <= 0 || max_pages_per_seq <= 0) return WPATTN_EINVAL;
  const int64_t tokens = sum_lengths(new_len_host, B), cap = int64_t(max_pages_per_seq) * page_size;
  if (tokens < 0) return WPATTN_EINVAL;
  for (int b = 0; b < B; ++b)
    if (kv_len_host[b] < new_len_host[b] || kv_len_host[b] > cap) return WPATTN_EINVAL;
  if (rope_base != 0.0 && !axes_ok(head_dim, tokens, positions, pos_stride, axes, pair_axis_host, rope_base))
    return WPATTN_EINVAL;
  if (tokens == 0) return WPATTN_OK;
  if (!k || !v || !k_pages || !v_pages || !block_table || !aligned4(block_table)) return WPATTN_EINVAL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages) ||
      (q && (!aligned16(q) || !aligned16(q_out))))
    return WPATTN_EINVAL;
  const int64_t kv_row = int64_t(Hkv) * head_dim, q_row = int64_t(Hq) * head_dim;
  if (k_stride < kv_row || v_stride < kv_row || (k_stride | v_stride) % 8 || (q && (q_stride < q_row || q_stride % 8)))
    return WPATTN_EINVAL;
  DeviceInfo* dev = nullptr;
  int rc;
  if ((rc = device_info(&dev)) != WPATTN_OK) return rc;
  const auto impl = B <= 64 ? append_impl<64> : append_impl<kPagedMaxB>;
  return impl(k, k_stride, v, v_stride, q, q_stride, q_out, k_pages, v_pages, num_pages, page_size, block_table,
              max_pages_per_seq, new_len_host, kv_len_host, B, Hq, Hkv, head_dim, static_cast<int32_t>(tokens),
              positions, pos_stride, axes, pair_axis_host, rope_base, dev->num_sms,
              static_cast<cudaStream_t>(cuda_stream));
}

size_t wpattn_prefill_paged_workspace_size(const wpattn_window* w, const int32_t* q_len_host,
                                           const int32_t* kv_len_host, int32_t B, int32_t Hq, int32_t Hkv) {
  WindowPlan plan;
  if (make_window_plan(w, &plan) != WPATTN_OK || (plan.D != 64 && plan.D != 128)) return 0;
  if (B <= 0 || B > kPagedMaxB || Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hq / Hkv > 128 || !q_len_host || !kv_len_host)
    return 0;
  const int64_t tokens = sum_lengths(q_len_host, B);
  if (tokens < 0 || tokens > kMaxTokens) return 0;
  for (int b = 0; b < B; ++b)
    if (kv_len_host[b] < 0 || kv_len_host[b] > (1 << 30)) return 0;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev) != WPATTN_OK) return 0;
  PagedPlan pp;
  return plan_paged(q_len_host, kv_len_host, B, Hq / Hkv, Hkv, plan, dev->num_sms, &pp) ? pp.bytes(plan.D) : 0;
}

int wpattn_prefill_paged(const wpattn_window* w, const void* q, const void* k_pages, const void* v_pages,
                         int32_t num_pages, int32_t page_size, const int32_t* block_table,
                         int32_t max_pages_per_seq, const int32_t* q_len_host, const int32_t* kv_len_host,
                         int32_t B, int32_t Hq, int32_t Hkv, float softmax_scale, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* cuda_stream) {
  WindowPlan plan;
  int rc = make_window_plan(w, &plan);
  if (rc != WPATTN_OK) return rc;
  if (B < 0 || Hq <= 0 || Hkv <= 0 || (Hq % Hkv) != 0 || num_pages <= 0 || max_pages_per_seq <= 0)
    return WPATTN_EINVAL;
  if (!(softmax_scale == softmax_scale)) return WPATTN_EINVAL;  // NaN
  if ((plan.D != 64 && plan.D != 128) || !page_size_ok(page_size) || B > kPagedMaxB || Hq / Hkv > 128)
    return WPATTN_EUNSUPPORTED;
  if (B == 0) return WPATTN_OK;
  if (!q_len_host || !kv_len_host) return WPATTN_EINVAL;
  const int64_t tokens = sum_lengths(q_len_host, B), cap = int64_t(max_pages_per_seq) * page_size;
  if (tokens < 0) return WPATTN_EINVAL;
  for (int b = 0; b < B; ++b)
    if (kv_len_host[b] < 0 || kv_len_host[b] > cap) return WPATTN_EINVAL;
  if (tokens == 0) return WPATTN_OK;
  if (!q || !out || !k_pages || !v_pages || !block_table || !aligned4(block_table) || !aligned4(lse))
    return WPATTN_EINVAL;
  if (!aligned16(q) || !aligned16(out) || !aligned16(k_pages) || !aligned16(v_pages)) return WPATTN_EINVAL;
  if (cap > (int64_t(1) << 30) || int64_t(num_pages) * page_size >= (int64_t(1) << 31) ||
      tokens > kMaxTokens)
    return WPATTN_EUNSUPPORTED;
  PagedCall c;
  if ((rc = device_info(&c.dev)) != WPATTN_OK) return rc;
  if (!plan_paged(q_len_host, kv_len_host, B, Hq / Hkv, Hkv, plan, c.dev->num_sms, &c.plan))
    return WPATTN_EUNSUPPORTED;
  if (c.plan.split_ctas > 0) {
    if (!workspace || workspace_bytes < c.plan.bytes(plan.D)) return WPATTN_EWORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return WPATTN_EINVAL;
  }
  c.window = &plan;
  c.q = q; c.k = k_pages; c.v = v_pages; c.out = out; c.lse = lse; c.workspace = workspace;
  c.block_table = block_table; c.q_len = q_len_host; c.kv_len = kv_len_host;
  c.num_pages = num_pages; c.page_size = page_size; c.max_pages = max_pages_per_seq;
  c.B = B; c.Hq = Hq; c.Hkv = Hkv;
  c.scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt(static_cast<float>(plan.D));
  c.st = static_cast<cudaStream_t>(cuda_stream);
  if (plan.D == 64) return plan.g == 8 ? run_paged<64, true>(c) : run_paged<64, false>(c);
  return plan.g == 8 ? run_paged<128, true>(c) : run_paged<128, false>(c);
}

int wpattn_pages_copy(void* const* pools_host, int32_t n_pools, int32_t num_pages, int64_t page_bytes,
                      const int32_t* src, const int32_t* dst, int32_t n, void* cuda_stream) {
  CopyParams p;
  int rc = set_pools(&p.pools, pools_host, n_pools, page_bytes);
  if (rc != WPATTN_OK) return rc;
  if (n < 0 || num_pages <= 0) return WPATTN_EINVAL;
  if (n > (1 << 30)) return WPATTN_EUNSUPPORTED;
  if (n == 0 || n_pools == 0) return WPATTN_OK;
  if (!src || !dst || !aligned4(src) || !aligned4(dst)) return WPATTN_EINVAL;
  DeviceInfo* dev = nullptr;
  if ((rc = device_info(&dev)) != WPATTN_OK) return rc;
  p.src = src; p.dst = dst; p.n = n; p.num_pages = num_pages; p.page_bytes = page_bytes;
  const dim3 grid(std::min(n, std::max(1, dev->num_sms * 8 / n_pools)), n_pools);
  copy_pages_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(cuda_stream)>>>(p);
  return launched();
}

size_t wpattn_pages_workspace_size(int32_t num_pages) {
  return num_pages > 0 ? (static_cast<size_t>(num_pages) * 3 + 2) * 4 + 4 * kPageRows : 0;
}

int wpattn_pages_fork(void* const* pools_host, int32_t n_pools, int32_t num_pages, int32_t page_size,
                      int64_t row_bytes, int32_t* block_table, int32_t num_rows, int32_t max_pages,
                      int32_t* refs, const int32_t* src_rows_host, const int32_t* dst_rows_host,
                      const int32_t* len_host, int32_t n, void* workspace, size_t workspace_bytes,
                      void* cuda_stream) {
  if (page_size <= 0 || row_bytes <= 0 || row_bytes % 16) return WPATTN_EINVAL;
  PagePools pools;
  int rc = set_pools(&pools, pools_host, n_pools, row_bytes * page_size);
  if (rc != WPATTN_OK) return rc;
  if (n < 0 || num_pages <= 0 || num_rows <= 0 || max_pages <= 0) return WPATTN_EINVAL;
  if (n > kPageRows || !page_counts_ok(num_pages, page_size, max_pages)) return WPATTN_EUNSUPPORTED;
  if (n == 0) return WPATTN_OK;
  if (!block_table || !refs || !src_rows_host || !dst_rows_host || !len_host || !aligned4(block_table) ||
      !aligned4(refs))
    return WPATTN_EINVAL;
  int32_t dsts[kPageRows];
  if (!rows_ok(dst_rows_host, n, num_rows, dsts)) return WPATTN_EINVAL;
  for (int i = 0; i < n; ++i)
    if (src_rows_host[i] < 0 || src_rows_host[i] >= num_rows || len_host[i] < 0 ||
        len_host[i] > int64_t(max_pages) * page_size || std::binary_search(dsts, dsts + n, src_rows_host[i]))
      return WPATTN_EINVAL;
  if (!workspace || workspace_bytes < wpattn_pages_workspace_size(num_pages)) return WPATTN_EWORKSPACE;
  if (!aligned16(workspace)) return WPATTN_EINVAL;
  DeviceInfo* dev = nullptr;
  if ((rc = device_info(&dev)) != WPATTN_OK) return rc;
  const auto fork = n <= kFewRows ? launch_fork<kFewRows> : launch_fork<kPageRows>;
  return fork(pools, num_pages, page_size, row_bytes, block_table, max_pages, refs, src_rows_host, dst_rows_host,
              len_host, n, static_cast<int32_t*>(workspace), dev->num_sms, static_cast<cudaStream_t>(cuda_stream));
}

int wpattn_pages_free(int32_t num_pages, int32_t page_size, int32_t* block_table, int32_t num_rows,
                      int32_t max_pages, int32_t* refs, const int32_t* rows_host, const int32_t* len_host,
                      int32_t n, void* cuda_stream) {
  if (n < 0 || num_pages <= 0 || page_size <= 0 || num_rows <= 0 || max_pages <= 0) return WPATTN_EINVAL;
  if (n > kPageRows || !page_counts_ok(num_pages, page_size, max_pages)) return WPATTN_EUNSUPPORTED;
  if (n == 0) return WPATTN_OK;
  int32_t sorted[kPageRows];
  if (!block_table || !refs || !rows_host || !len_host || !aligned4(block_table) || !aligned4(refs) ||
      !rows_ok(rows_host, n, num_rows, sorted))
    return WPATTN_EINVAL;
  int longest = 0;
  for (int i = 0; i < n; ++i) {
    if (len_host[i] < 0 || len_host[i] > int64_t(max_pages) * page_size) return WPATTN_EINVAL;
    longest = std::max(longest, len_host[i]);
  }
  if (longest == 0) return WPATTN_OK;
  DeviceInfo* dev = nullptr;
  const int rc = device_info(&dev);
  if (rc != WPATTN_OK) return rc;
  const auto give_back = n <= kFewRows ? launch_free<kFewRows> : launch_free<kPageRows>;
  return give_back(num_pages, page_size, block_table, max_pages, refs, rows_host, len_host, n,
                   (longest + page_size - 1) / page_size, static_cast<cudaStream_t>(cuda_stream));
}

int wpattn_pages_extend(int32_t num_pages, int32_t page_size, int32_t* block_table, int32_t num_rows,
                        int32_t max_pages, int32_t* refs, const int32_t* rows_host, const int32_t* len_host,
                        const int32_t* new_len_host, int32_t n, void* cuda_stream) {
  if (n < 0 || num_pages <= 0 || page_size <= 0 || num_rows <= 0 || max_pages <= 0) return WPATTN_EINVAL;
  if (n > kPageRows || !page_counts_ok(num_pages, page_size, max_pages)) return WPATTN_EUNSUPPORTED;
  if (n == 0) return WPATTN_OK;
  int32_t sorted[kPageRows];
  if (!block_table || !refs || !rows_host || !len_host || !new_len_host || !aligned4(block_table) ||
      !aligned4(refs) || !rows_ok(rows_host, n, num_rows, sorted))
    return WPATTN_EINVAL;
  ExtendParams p;
  std::memset(&p, 0, sizeof p);
  int64_t want = 0;
  for (int i = 0; i < n; ++i) {
    if (len_host[i] < 0 || new_len_host[i] < len_host[i] || new_len_host[i] > int64_t(max_pages) * page_size)
      return WPATTN_EINVAL;
    p.row[i] = rows_host[i];
    p.first[i] = (len_host[i] + page_size - 1) / page_size;
    want += (new_len_host[i] + page_size - 1) / page_size - p.first[i];
    if (want > (1 << 30)) return WPATTN_EUNSUPPORTED;   // the kernel's loops step past it by a block of threads
    p.start[i + 1] = static_cast<int>(want);
  }
  if (want == 0) return WPATTN_OK;
  DeviceInfo* dev = nullptr;
  const int rc = device_info(&dev);
  if (rc != WPATTN_OK) return rc;
  p.table = block_table; p.refs = refs;
  p.num_pages = num_pages; p.max_pages = max_pages; p.n = n;
  extend_kernel<<<1, kScanThreads, 0, static_cast<cudaStream_t>(cuda_stream)>>>(p);
  return launched();
}

int wpattn_pages_compact(void* const* pools_host, int32_t n_pools, int32_t num_pages, int64_t page_bytes,
                         int32_t* block_table, int64_t entries, int32_t* refs, int32_t* live,
                         void* workspace, size_t workspace_bytes, void* cuda_stream) {
  CompactParams p;
  int rc = set_pools(&p.pools, pools_host, n_pools, page_bytes);
  if (rc != WPATTN_OK) return rc;
  if (num_pages <= 0 || entries < 0 || (entries > 0 && !block_table) || !refs || !aligned4(block_table) ||
      !aligned4(refs) || !aligned4(live))
    return WPATTN_EINVAL;
  if (num_pages > (1 << 30)) return WPATTN_EUNSUPPORTED;
  if (!workspace || workspace_bytes < wpattn_pages_workspace_size(num_pages)) return WPATTN_EWORKSPACE;
  if (!aligned16(workspace)) return WPATTN_EINVAL;
  DeviceInfo* dev = nullptr;
  if ((rc = device_info(&dev)) != WPATTN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  int32_t* ws = static_cast<int32_t*>(workspace);
  compact_plan_kernel<<<1, kScanThreads, 0, st>>>(refs, num_pages, ws, live);
  if ((rc = launched()) != WPATTN_OK) return rc;
  p.table = block_table; p.refs = refs; p.ws = ws; p.num_pages = num_pages;
  p.entries = entries; p.page_bytes = page_bytes;
  compact_kernel<<<std::min(num_pages, dev->num_sms * 8), 256, 0, st>>>(p);
  return launched();
}

}  // extern "C"
