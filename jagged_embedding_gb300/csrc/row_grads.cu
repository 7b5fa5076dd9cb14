// Gradient of the (scaled) embedding lookup by sorted IDs:
//   rows = the distinct IDs, ascending;  G[u] = scale * sum over p with ids[p] = rows[u] of dout[p]
// -- FreeScale (arXiv 2604.24073) Algorithm 2 lines 7, 18 and 20 without the
// optimizer: what update_embedding receives, for callers that clip, average or
// apply an optimizer of their own.
//
//   1. sort of (row, position): counting passes over one range of entries a block;
//   2. heads: numbers the distinct rows of the sorted entries, over the same ranges;
//   3. reduce: a group of lanes per tile of `chunk` sorted entries sums dout
//      rows in fp32 in entry order; a row inside the tile is written out, a row
//      that crosses a tile's edge leaves partial sums;
//   4. join: adds the partial sums of the rows that cross edges, in tile order
//      (a hot row crosses thousands of tiles: a whole block adds those).
// A small batch (at most 8192 entries) takes two launches instead of seven to sixteen: one block sorts and
// numbers in shared memory, then a warp sums each distinct row.
// The order of every sum follows from the sorted order and T alone: results are
// the same bits from run to run.
//
// Bound by HBM: 8 B of ID and one row of dout per position, one row of G per
// distinct ID; the sort moves about 20 B per ID and pass beside that.  2M Zipf IDs
// over 10M rows, bf16 rows of 128 into fp32 rows: 252 us a call -- sort 77, numbering
// 19, reduce 138 (0.79 GB, 5.7 TB/s), join 14 -- of which those bytes alone would take 124.
// 2000 IDs: 18 us, half of it the one block that sorts.
#include <atomic>

#include "convert.cuh"
#include "fs_common.cuh"
#include "range_sort.cuh"

namespace fs {
namespace {

// ------------------------------------------------------------- numbering the rows

struct Numbering {
  int64_t* rows;    // [cap] out
  int64_t cap;
  int64_t* count;   // [1] out
  uint32_t* start;  // [T + 1]: first sorted entry of distinct row u; start[count] = n
  uint32_t* before; // [tiles]: distinct rows that begin before tile t
  int chunk_log2;
};

// Distinct rows that begin in each block's range of the sorted entries, then their numbers:
// a block adds up the counts of the blocks before it (two launches, 8 B read per entry).
constexpr int kHeadThreads = range_sort::kThreads, kHeadItems = 8, kHeadTile = kHeadThreads * kHeadItems;

__global__ void __launch_bounds__(kHeadThreads) head_count_kernel(const uint32_t* keys, const int64_t* n_dev,
                                                                  uint32_t* __restrict__ counts) {
  __shared__ uint32_t scratch[32];
  range_sort::launch_next();
  range_sort::wait_previous();
  const range_sort::Range r = range_sort::range_of(__ldcg(n_dev));
  uint32_t mine = 0, total;
  for (int64_t j = threadIdx.x; j < r.count; j += kHeadTile) {
    uint32_t k[kHeadItems], p[kHeadItems];
#pragma unroll
    for (int q = 0; q < kHeadItems; ++q)
      if (j + q * kHeadThreads < r.count) {
        const int64_t i = r.first + j + q * kHeadThreads;
        k[q] = __ldcg(keys + i);
        p[q] = i ? __ldcg(keys + i - 1) : ~k[q];
      }
#pragma unroll
    for (int q = 0; q < kHeadItems; ++q) mine += j + q * kHeadThreads < r.count && k[q] != p[q];
  }
  block_exclusive_scan<uint32_t>(mine, scratch, &total);
  if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kHeadThreads) number_kernel(const uint32_t* keys, const int64_t* n_dev, Numbering N,
                                                              const uint32_t* counts, int32_t* err) {
  __shared__ uint32_t scratch[32];
  range_sort::wait_previous();
  const int64_t n = __ldcg(n_dev);
  const range_sort::Range r = range_sort::range_of(n);
  uint32_t part = 0, run;
  for (int b = threadIdx.x; b < int(blockIdx.x); b += kHeadThreads) part += __ldcg(counts + b);
  block_exclusive_scan<uint32_t>(part, scratch, &run);
  for (int64_t t0 = 0; t0 < r.count; t0 += kHeadTile) {
    const int64_t i0 = r.first + t0 + int64_t(threadIdx.x) * kHeadItems, end = r.first + r.count;
    uint32_t k[kHeadItems], prev = 0;
    if (i0 < end) {  // (begins at a multiple of 8; the array ends at one of 64)
      const uint4 a = __ldcg(reinterpret_cast<const uint4*>(keys + i0)), b = __ldcg(reinterpret_cast<const uint4*>(keys + i0) + 1);
      k[0] = a.x, k[1] = a.y, k[2] = a.z, k[3] = a.w, k[4] = b.x, k[5] = b.y, k[6] = b.z, k[7] = b.w;
      if (i0 > 0) prev = __ldcg(keys + i0 - 1);
    }
    uint32_t heads = 0, mine = 0;
#pragma unroll
    for (int q = 0; q < kHeadItems; ++q) {
      const bool h = i0 + q < end && (i0 + q == 0 || k[q] != (q ? k[q - 1] : prev));
      heads |= uint32_t(h) << q;
      mine += h;
    }
    uint32_t total;
    uint32_t u = run + block_exclusive_scan<uint32_t>(mine, scratch, &total);
    run += total;
#pragma unroll
    for (int q = 0; q < kHeadItems; ++q) {
      const int64_t i = i0 + q;
      if (i < end && (i & ((int64_t(1) << N.chunk_log2) - 1)) == 0) N.before[i >> N.chunk_log2] = u;
      if ((heads >> q) & 1u) {
        N.start[u] = uint32_t(i);
        if (int64_t(u) < N.cap) N.rows[u] = int64_t(k[q]);
        else set_err(err, FS_ERR_CAPACITY);
        ++u;
      }
    }
  }
  if (threadIdx.x == 0 && (r.count > 0 ? r.first + r.count == n : n == 0 && blockIdx.x == 0)) {
    *N.count = int64_t(run);
    N.start[run] = uint32_t(n);
  }
}

// ------------------------------------------------------------- small batches

// Sort, numbering and the count of a batch of at most 1024 * ITEMS entries by
// one block: keys in registers, stable counting passes of at most 10
// bits over shared memory.  An ID out of range takes the key 2^kb - 1 >= R,
// sorts last and is dropped.
constexpr int kSmallThreads = 1024, kSmallWarps = kSmallThreads / 32, kSmallBins = 1024;
constexpr int64_t kSmallMax = kSmallThreads * 8;
template <int ITEMS>
constexpr size_t small_smem() {
  return (size_t(kSmallThreads) * ITEMS * 2 + size_t(kSmallWarps + 1) * kSmallBins + 64) * sizeof(uint32_t);
}

template <int ITEMS>
__global__ void __launch_bounds__(kSmallThreads, 1) small_sort_kernel(const int64_t* __restrict__ ids, int32_t T, int64_t R,
                                                                      int kb, uint32_t* out_v, Numbering N,
                                                                      int32_t* err) {
  extern __shared__ uint32_t sm[];
  range_sort::launch_next();
  uint32_t* keys = sm;
  uint32_t* vals = keys + kSmallThreads * ITEMS;
  uint32_t* hist = vals + kSmallThreads * ITEMS;  // [warps][digits]
  uint32_t* dstart = hist + kSmallWarps * kSmallBins;  // [digits]
  uint32_t* red = dstart + kSmallBins;                 // [64]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto slot = [&](int i) { return warp * 32 * ITEMS + i * 32 + lane; };  // slot order = item order
  const uint32_t bad = uint32_t((uint64_t(1) << kb) - 1);
  uint32_t k[ITEMS], v[ITEMS], rank[ITEMS], valid = 0;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int g = slot(i);
    k[i] = bad;
    v[i] = uint32_t(g);
    if (g < T) {
      const int64_t id = __ldcs(ids + g);
      if (uint64_t(id) < uint64_t(R)) {
        k[i] = uint32_t(id);
        ++valid;
      } else {
        set_err(err, FS_ERR_ID_RANGE);
      }
    }
  }
  const int passes = (kb + 9) / 10, bits = (kb + passes - 1) / passes, nb = 1 << bits;
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = bits * pass;
    for (int j = threadIdx.x; j < kSmallWarps * nb; j += kSmallThreads) hist[j] = 0u;
    __syncthreads();
    uint32_t* wh = hist + warp * nb;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const bool live = slot(i) < T;
      const uint32_t d = (k[i] >> shift) & uint32_t(nb - 1);
      const unsigned lv = __ballot_sync(0xffffffffu, live);
      const unsigned same = __match_any_sync(0xffffffffu, d);
      const unsigned peers = same & (live ? lv : ~lv);
      const unsigned lt = __popc(peers & lanemask_lt());
      const uint32_t base = live ? wh[d] : 0u;
      rank[i] = base + lt;
      __syncwarp();
      if (live && lt == 0) wh[d] = base + __popc(peers);
      __syncwarp();
    }
    __syncthreads();
    // thread d: digit d's entries, exclusive over the warps (all read before any is
    // written: one latency instead of 32), then over the digits
    uint32_t tot = 0;
    if (int(threadIdx.x) < nb) {
      uint32_t c[kSmallWarps];
#pragma unroll
      for (int w = 0; w < kSmallWarps; ++w) c[w] = hist[w * nb + threadIdx.x];
#pragma unroll
      for (int w = 0; w < kSmallWarps; ++w) {
        hist[w * nb + threadIdx.x] = tot;
        tot += c[w];
      }
    }
    uint32_t all;
    const uint32_t first = block_exclusive_scan<uint32_t>(tot, red, &all);
    if (int(threadIdx.x) < nb) dstart[threadIdx.x] = first;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (slot(i) < T) {
        const uint32_t d = (k[i] >> shift) & uint32_t(nb - 1);
        const uint32_t at = dstart[d] + hist[warp * nb + d] + rank[i];
        keys[at] = k[i];
        vals[at] = v[i];
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (slot(i) < T) {
        k[i] = keys[slot(i)];
        v[i] = vals[slot(i)];
      }
    __syncthreads();
  }
  // the sorted entries are in `keys` / `vals`; the valid ones come first
  uint32_t n, total;
  block_exclusive_scan<uint32_t>(valid, red, &n);
  uint32_t mine = 0, heads = 0;
  // consecutive entries per thread for the numbering
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t p = threadIdx.x * ITEMS + i;
    const bool h = p < n && (p == 0 || keys[p] != keys[p - 1]);
    heads |= uint32_t(h) << i;
    mine += h;
  }
  uint32_t u = block_exclusive_scan<uint32_t>(mine, red, &total);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t p = threadIdx.x * ITEMS + i;
    if (p >= n) break;
    if ((heads >> i) & 1u) {
      N.start[u] = p;
      if (int64_t(u) < N.cap) N.rows[u] = int64_t(keys[p]);
      else set_err(err, FS_ERR_CAPACITY);
      ++u;
    }
    out_v[p] = vals[p];
  }
  if (threadIdx.x == 0) {
    *N.count = total;
    N.start[total] = n;
  }
}

// Sums of a small batch: a warp per distinct row, LPR lanes (VEC columns each) a dout row, 32 / LPR
// rows beside one another, kRedRows of them in flight per lane; their sums meet by
// shuffles.  A row of more than kLongRow entries is taken by the block's eight warps.
// blockIdx.y picks LPR * VEC columns of wider rows.
// The blocks may be in place while the sort still writes vals, start and count: those are read
// after the wait and past L1, and are not declared constant for this kernel's lifetime.
constexpr int kSmallRowThreads = 256, kSmallRowWarps = kSmallRowThreads / 32, kLongRow = 48;

template <class EI, class EO, int VEC, int LPR>
__global__ void __launch_bounds__(kSmallRowThreads) grad_small_kernel(const uint32_t* vals, const uint32_t* start,
                                                                      const int64_t* count,
                                                                      const void* __restrict__ dout, int32_t dim,
                                                                      float scale, void* __restrict__ grads, int64_t cap) {
  constexpr int SUB = 32 / LPR;
  constexpr int SV = VEC * EO::kBytes > 16 ? VEC / 2 : VEC;  // columns of one store
  __shared__ uint32_t long_row[kSmallRowWarps];
  __shared__ float sums[kSmallRowWarps][LPR * VEC];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / LPR, c = (int(blockIdx.y) * LPR + lane % LPR) * VEC;
  range_sort::wait_previous();
  const int64_t found = __ldcg(count), distinct = found < cap ? found : cap;
  auto add = [&](float (&acc)[VEC], uint32_t e, uint32_t end, uint32_t step) {
    for (; e < end; e += 8 * step) {
      Raw<EI, VEC> g[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (e + q * step < end && c < dim) fetch<true>(g[q], dout, int64_t(__ldcg(vals + e + q * step)) * dim + c);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (e + q * step < end && c < dim) {
          float x[VEC];
          unpack(g[q], x);
#pragma unroll
          for (int k = 0; k < VEC; ++k) acc[k] += x[k];
        }
    }
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < VEC; ++k) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
  };
  auto put = [&](int64_t u, float (&acc)[VEC]) {
#pragma unroll
    for (int k = 0; k < VEC; k += SV) {
      float y[SV];
#pragma unroll
      for (int i = 0; i < SV; ++i) y[i] = acc[k + i] * scale;
      store_vec<EO, SV, true>(grads, u * dim + c + k, y);
    }
  };
  const int64_t u = int64_t(blockIdx.x) * kSmallRowWarps + warp;
  bool is_long = false;
  if (u < distinct) {
    const uint32_t s = __ldcg(start + u), e = __ldcg(start + u + 1);
    is_long = e - s > uint32_t(kLongRow);
    if (!is_long) {
      float acc[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
      add(acc, s + sub, e, SUB);
      if (sub == 0 && c < dim) put(u, acc);
    }
  }
  if (lane == 0) long_row[warp] = is_long ? 1u : 0u;
  __syncthreads();
  for (int w = 0; w < kSmallRowWarps; ++w) {
    if (!long_row[w]) continue;  // (the same for every thread)
    const int64_t ul = int64_t(blockIdx.x) * kSmallRowWarps + w;
    float acc[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
    add(acc, __ldcg(start + ul) + warp * SUB + sub, __ldcg(start + ul + 1), SUB * kSmallRowWarps);
    if (sub == 0)
#pragma unroll
      for (int k = 0; k < VEC; ++k) sums[warp][(lane % LPR) * VEC + k] = acc[k];
    __syncthreads();
    if (warp == 0 && sub == 0 && c < dim) {
      for (int q = 1; q < kSmallRowWarps; ++q)
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[k] += sums[q][(lane % LPR) * VEC + k];
      put(ul, acc);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------- reduce

constexpr int kRedThreads = 128, kRedRows = 8;  // dout rows in flight per lane

// LPR lanes (VEC columns each) per tile of 2^chunk_log2 sorted entries;
// blockIdx.y picks LPR * VEC columns of wider rows.  kRedRows dout rows are in
// flight per lane, held as loaded; the next step's keys and positions are
// loaded before this step's rows.  (The key and position arrays are padded to
// 64 entries, so a step's vector loads stay inside them.)
template <class EI, class EO, int VEC, int LPR>
__global__ void __launch_bounds__(kRedThreads, 6) grad_reduce_kernel(
    const uint32_t* __restrict__ keys, const uint32_t* __restrict__ vals, const int64_t* __restrict__ n_dev,
    const uint32_t* __restrict__ before, int chunk_log2, const void* __restrict__ dout, int32_t dim, float scale,
    void* __restrict__ grads, int64_t cap, float* __restrict__ part_head, float* __restrict__ part_tail) {
  constexpr int SV = VEC * EO::kBytes > 16 ? VEC / 2 : VEC;  // columns of one store of a finished row
  constexpr int PV = VEC > 4 ? 4 : VEC;                      // and of a partial one
  const int64_t n = *n_dev;
  const int chunk = 1 << chunk_log2;
  const int64_t t = (int64_t(blockIdx.x) * kRedThreads + threadIdx.x) / LPR;
  const int64_t s0 = t << chunk_log2;
  if (s0 >= n) return;
  const int c = (int(blockIdx.y) * LPR + int(threadIdx.x % LPR)) * VEC;
  if (c >= dim) return;
  const int m = n - s0 < chunk ? int(n - s0) : chunk;
  struct Eight {
    uint32_t x[8];
  };
  auto load8 = [](const uint32_t* p) {
    Eight e;
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    e.x[0] = a.x, e.x[1] = a.y, e.x[2] = a.z, e.x[3] = a.w, e.x[4] = b.x, e.x[5] = b.y, e.x[6] = b.z, e.x[7] = b.w;
    return e;
  };
  Eight nk = load8(keys + s0), nv = load8(vals + s0);
  int64_t u = before[t];
  bool from_prev = s0 > 0 && keys[s0 - 1] == nk.x[0];  // the tile's first row began in an earlier tile
  if (from_prev) --u;
  float acc[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
  auto partial = [&](float* part) {
#pragma unroll
    for (int k = 0; k < VEC; k += PV) {
      float x[PV];
#pragma unroll
      for (int i = 0; i < PV; ++i) x[i] = acc[k + i];
      store_vec<F32, PV, false>(part, t * dim + c + k, x);
    }
  };
  bool open = false;
  for (int j = 0; j < m; j += kRedRows) {
    const Eight key = nk, val = nv;
    Raw<EI, VEC> g[kRedRows];
#pragma unroll
    for (int q = 0; q < kRedRows; ++q)
      if (j + q < m) fetch<true>(g[q], dout, int64_t(val.x[q]) * dim + c);
    if (s0 + j + kRedRows < n) {
      nk = load8(keys + s0 + j + kRedRows);  // (past the tile: its first key tells whether the last row goes on)
      if (j + kRedRows < m) nv = load8(vals + s0 + j + kRedRows);
    }
#pragma unroll
    for (int q = 0; q < kRedRows; ++q) {
      if (j + q < m) {
        float x[VEC];
        unpack(g[q], x);
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[k] += x[k];
        open = true;
        const uint32_t after = q + 1 < kRedRows ? key.x[(q + 1) % kRedRows] : nk.x[0];
        if (s0 + j + q + 1 == n || after != key.x[q]) {  // the row's last entry
          if (from_prev) {
            partial(part_head);
          } else if (uint64_t(u) < uint64_t(cap)) {
#pragma unroll
            for (int k = 0; k < VEC; k += SV) {
              float y[SV];
#pragma unroll
              for (int i = 0; i < SV; ++i) y[i] = acc[k + i] * scale;
              store_vec<EO, SV, true>(grads, u * dim + c + k, y);
            }
          }
          from_prev = false;
          open = false;
          ++u;
#pragma unroll
          for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
        }
      }
    }
  }
  if (open) partial(from_prev ? part_head : part_tail);  // the row goes on: it began before this tile, or here
}

// The rows that begin in a tile and go on in the next: a row's sum is its tile's
// tail plus the heads of the following tiles up to the row's last.  A block takes
// one contiguous range of tiles: a thread per tile finds its row and its last
// tile (a chain of dependent loads, walked for the whole range together), then
// a warp per row adds.  Rows over more than kLongTiles tiles are added by the whole
// block: warp w takes every 16th tile, then the warps' sums in warp order.
// VEC columns a lane.  (A warp per tile that walked the chain itself took 39 us
// for 2M entries of 128, this 18.)
constexpr int kJoinThreads = 512, kJoinWarps = kJoinThreads / 32, kLongTiles = 16, kJoinPerSm = 2;

template <class EO, int VEC>
__global__ void __launch_bounds__(kJoinThreads, kJoinPerSm) grad_join_kernel(
    const uint32_t* __restrict__ keys, const int64_t* __restrict__ n_dev, const uint32_t* __restrict__ start,
    const uint32_t* __restrict__ before, int chunk_log2, int32_t dim, float scale, void* __restrict__ grads, int64_t cap,
    const float* __restrict__ part_head, const float* __restrict__ part_tail) {
  __shared__ uint32_t row[kJoinThreads];           // rows to join, in tile order
  __shared__ int32_t from[kJoinThreads], to[kJoinThreads];  // their first and last tiles
  __shared__ float sums[kJoinWarps][32 * VEC];
  __shared__ uint32_t scratch[32];
  const int64_t n = *n_dev;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t ntiles = (n + (int64_t(1) << chunk_log2) - 1) >> chunk_log2;
  // heads of tiles first, first + step, ... up to last, added to a
  auto sum_tiles = [&](float (&a)[VEC], int64_t first, int64_t last, int64_t step, int c) {
    int64_t v = first;
    for (; v + 7 * step <= last; v += 8 * step) {
      float x[8][VEC];
#pragma unroll
      for (int q = 0; q < 8; ++q) load_vec<F32, VEC, true>(part_head, (v + q * step) * dim + c, x[q]);
#pragma unroll
      for (int q = 0; q < 8; ++q)
#pragma unroll
        for (int k = 0; k < VEC; ++k) a[k] += x[q][k];
    }
    for (; v <= last; v += step) {
      float x[VEC];
      load_vec<F32, VEC, true>(part_head, v * dim + c, x);
#pragma unroll
      for (int k = 0; k < VEC; ++k) a[k] += x[k];
    }
  };
  auto put = [&](int64_t u, int c, float (&a)[VEC]) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) a[k] *= scale;
    store_vec<EO, VEC, false>(grads, u * dim + c, a);
  };
  const int64_t per = (ntiles + gridDim.x - 1) / gridDim.x;
  const int64_t begin = per * blockIdx.x, end = begin + per < ntiles ? begin + per : ntiles;
  for (int64_t t0 = begin; t0 < end; t0 += kJoinThreads) {
    const int64_t t = t0 + threadIdx.x, edge = (t + 1) << chunk_log2;
    uint32_t u = 0;
    int64_t last = 0;
    bool joins = false;
    if (t < end && edge < n) {
      const uint32_t k0 = keys[edge - 1], k1 = keys[edge], after = before[t + 1];  // (one latency for the three)
      if (k0 == k1) {
        u = after - 1;
        if (int64_t(u) < cap) {
          const uint32_t s = start[u], e = start[u + 1];
          joins = int64_t(s) >= (t << chunk_log2);  // it begins in this tile
          last = int64_t(e - 1) >> chunk_log2;
        }
      }
    }
    uint32_t rows;
    const uint32_t at = block_exclusive_scan<uint32_t>(joins ? 1u : 0u, scratch, &rows);
    if (joins) {
      row[at] = u;
      from[at] = int32_t(t);
      to[at] = int32_t(last);
    }
    __syncthreads();
    for (uint32_t i = warp; i < rows; i += kJoinWarps) {
      const int64_t tt = from[i], last_t = to[i];
      if (last_t - tt > kLongTiles) continue;
      for (int c = lane * VEC; c < dim; c += 32 * VEC) {
        float a[VEC];
        load_vec<F32, VEC, true>(part_tail, tt * dim + c, a);
        sum_tiles(a, tt + 1, last_t, 1, c);
        put(row[i], c, a);
      }
    }
    for (uint32_t i = 0; i < rows; ++i) {
      const int64_t tt = from[i], last_t = to[i];
      if (last_t - tt <= kLongTiles) continue;  // (the same for every thread)
      for (int c0 = 0; c0 < dim; c0 += 32 * VEC) {
        const int c = c0 + lane * VEC;
        float a[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) a[k] = 0.f;
        if (c < dim) sum_tiles(a, tt + 1 + warp, last_t, kJoinWarps, c);
#pragma unroll
        for (int k = 0; k < VEC; ++k) sums[warp][lane * VEC + k] = a[k];
        __syncthreads();
        if (warp == 0 && c < dim) {
          load_vec<F32, VEC, true>(part_tail, tt * dim + c, a);
          for (int q = 0; q < kJoinWarps; ++q)
#pragma unroll
            for (int k = 0; k < VEC; ++k) a[k] += sums[q][lane * VEC + k];
          put(row[i], c, a);
        }
        __syncthreads();
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------- host side

// Entries per reduce tile: 8 for the smallest batches (one step of loads),
// doubled while more than 8192 tiles remain, at most 64: enough groups of lanes to
// fill the GPU, few edges, each of which costs a partial row written and read
// (2M entries of 128 bf16: 64 was 10 us a call faster than 128 and 18 than 32).
int chunk_log2_for(int64_t T) {
  int c = 3;
  while (c < 6 && (T >> c) > 8192) ++c;
  return c;
}

struct GradLayout {
  int chunk_log2 = 3;
  int64_t tiles = 0;
};

GradLayout grad_layout(int64_t T) {
  GradLayout L;
  L.chunk_log2 = chunk_log2_for(T);
  L.tiles = (T + (int64_t(1) << L.chunk_log2) - 1) >> L.chunk_log2;
  return L;
}

struct GradWs {
  range_sort::Ws sort;
  uint32_t *start = nullptr, *before = nullptr;
  uint32_t* heads = nullptr;  // distinct rows that begin in each block's range
  float *part_head = nullptr, *part_tail = nullptr;
};

template <class Cursor>
void take_grad(const GradLayout& L, int64_t T, int32_t dim, Cursor& ws, GradWs& G) {
  range_sort::take(T, ws, G.sort);
  G.start = ws.template take<uint32_t>(size_t(T) + 1);
  G.before = ws.template take<uint32_t>(size_t(L.tiles) + 1);
  G.heads = ws.template take<uint32_t>(range_sort::kMaxBlocks);
  G.part_head = ws.template take<float>(size_t(L.tiles) * dim);
  G.part_tail = ws.template take<float>(size_t(L.tiles) * dim);
}

template <class EI, class EO, int VEC, int LPR>
void launch_reduce_lpr(const GradLayout& L, const GradWs& G, const uint32_t* sk, const uint32_t* sv, const void* dout,
                       int32_t dim, float scale, void* grads, int64_t cap, cudaStream_t st) {
  const int64_t threads = L.tiles * LPR;
  const dim3 grid(unsigned((threads + kRedThreads - 1) / kRedThreads), unsigned((dim + LPR * VEC - 1) / (LPR * VEC)));
  grad_reduce_kernel<EI, EO, VEC, LPR><<<grid, kRedThreads, 0, st>>>(sk, sv, G.sort.n, G.before, L.chunk_log2,
                                                                     dout, dim, scale, grads, cap, G.part_head,
                                                                     G.part_tail);
}

template <class EI, class EO, int VEC>
void launch_small_vec(int64_t most_rows, const GradWs& G, const uint32_t* sv, const int64_t* count, const void* dout,
                      int32_t dim, float scale, void* grads, int64_t cap, cudaStream_t st) {
  const int chunks = (dim + VEC - 1) / VEC;
  const int lpr = chunks <= 8 ? 8 : (chunks <= 16 ? 16 : 32);
  const dim3 grid(unsigned((most_rows + kSmallRowWarps - 1) / kSmallRowWarps), unsigned((chunks + lpr - 1) / lpr));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kSmallRowThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto go = [&](auto kern) {
    cudaLaunchKernelEx(&cfg, kern, sv, static_cast<const uint32_t*>(G.start), count, dout, dim, scale, grads, cap);
  };
  if (lpr == 8) go(grad_small_kernel<EI, EO, VEC, 8>);
  else if (lpr == 16) go(grad_small_kernel<EI, EO, VEC, 16>);
  else go(grad_small_kernel<EI, EO, VEC, 32>);
}

// The sort of a small batch: ITEMS entries a thread.  Its shared memory is allowed once per device.
template <int ITEMS>
bool launch_small_sort(const int64_t* ids, int64_t T, int64_t R, uint32_t* sv, const Numbering& N, int32_t* err,
                       cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
  if (!bit || !(ready.load(std::memory_order_relaxed) & bit)) {
    if (cudaFuncSetAttribute(small_sort_kernel<ITEMS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(small_smem<ITEMS>())) != cudaSuccess)
      return false;
    ready.fetch_or(bit);
  }
  const int kb = range_sort::bits_for(uint64_t(R));  // room for a key past every row
  small_sort_kernel<ITEMS><<<1, kSmallThreads, small_smem<ITEMS>(), st>>>(ids, int32_t(T), R, kb, sv, N, err);
  return true;
}

template <class EI, class EO, int VEC>
void launch_reduce_vec(const GradLayout& L, const GradWs& G, const uint32_t* sk, const uint32_t* sv, const void* dout,
                       int32_t dim, float scale, void* grads, int64_t cap, cudaStream_t st) {
  const int chunks = (dim + VEC - 1) / VEC;
  if (chunks <= 8) launch_reduce_lpr<EI, EO, VEC, 8>(L, G, sk, sv, dout, dim, scale, grads, cap, st);
  else if (chunks <= 16) launch_reduce_lpr<EI, EO, VEC, 16>(L, G, sk, sv, dout, dim, scale, grads, cap, st);
  else launch_reduce_lpr<EI, EO, VEC, 32>(L, G, sk, sv, dout, dim, scale, grads, cap, st);
}

}  // namespace
}  // namespace fs

using namespace fs;

extern "C" size_t fs_emb_grad_rows_workspace_size(int64_t T, int64_t num_rows, int32_t dim) {
  if (T < 0 || T > INT32_MAX || num_rows < 1 || num_rows >= (int64_t(1) << 32) || dim < 1) return 0;
  const GradLayout L = grad_layout(T);
  WsCounter c;
  GradWs G;
  take_grad(L, T, dim, c, G);
  return c.used + 256;
}

extern "C" fs_status fs_emb_grad_rows(int64_t num_rows, int32_t dim, const int64_t* ids, int64_t T, const void* dout,
                                      fs_dtype dout_dtype, float scale, int64_t* rows, void* row_grads,
                                      fs_dtype grad_dtype, int64_t cap_rows, int64_t* count, int32_t* err, void* ws,
                                      size_t ws_bytes, fs_stream_t stream) {
  FS_NVTX_RANGE();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T < 0 || T > INT32_MAX || num_rows < 1 || num_rows >= (int64_t(1) << 32) || dim < 1 || cap_rows < 0 || !count ||
      !err)
    return FS_ERR_INVALID_ARG;
  if ((dout_dtype != FS_F32 && dout_dtype != FS_BF16) || (grad_dtype != FS_F32 && grad_dtype != FS_BF16))
    return FS_ERR_INVALID_ARG;
  if (!aligned(count, 8)) return FS_ERR_ALIGNMENT;
  if (T == 0) return cudaMemsetAsync(count, 0, sizeof(int64_t), st) == cudaSuccess ? FS_OK : FS_ERR_CUDA;
  if (!ids || !dout || (cap_rows > 0 && (!rows || !row_grads))) return FS_ERR_INVALID_ARG;
  const size_t ib = dout_dtype == FS_F32 ? 4 : 2, ob = grad_dtype == FS_F32 ? 4 : 2;
  if (!aligned(ids, 8) || !aligned(rows, 8) || !aligned(dout, ib) || !aligned(row_grads, ob)) return FS_ERR_ALIGNMENT;
  if (!ws || ws_bytes < fs_emb_grad_rows_workspace_size(T, num_rows, dim)) return FS_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return FS_ERR_ALIGNMENT;  // (sorted entries and partial sums move in 16-byte accesses)

  const GradLayout L = grad_layout(T);
  WsCursor cur(ws, ws_bytes);
  GradWs G;
  take_grad(L, T, dim, cur, G);
  if (!cur.ok) return FS_ERR_WORKSPACE;
  const Numbering N{rows, cap_rows, count, G.start, G.before, L.chunk_log2};
  int launches = 0;
  uint32_t *sk = G.sort.k[0], *sv = G.sort.v[0];
  const bool small = T <= kSmallMax;
  if (small) {
    bool ok;
    if (T <= kSmallThreads) ok = launch_small_sort<1>(ids, T, num_rows, sv, N, err, st);
    else if (T <= kSmallThreads * 2) ok = launch_small_sort<2>(ids, T, num_rows, sv, N, err, st);
    else if (T <= kSmallThreads * 3) ok = launch_small_sort<3>(ids, T, num_rows, sv, N, err, st);
    else if (T <= kSmallThreads * 4) ok = launch_small_sort<4>(ids, T, num_rows, sv, N, err, st);
    else if (T <= kSmallThreads * 6) ok = launch_small_sort<6>(ids, T, num_rows, sv, N, err, st);
    else ok = launch_small_sort<8>(ids, T, num_rows, sv, N, err, st);
    if (!ok) return FS_ERR_CUDA;
    launches += 1;
  } else {
    int side = 0;
    const fs_status s = range_sort::sort(ids, T, num_rows, range_sort::bits_for(uint64_t(num_rows - 1)), G.sort, err, st, &side,
                                         &launches);
    if (s != FS_OK) return s;
    sk = G.sort.k[side];
    sv = G.sort.v[side];
    const int blocks = range_sort::blocks_for(T);
    if (range_sort::launch_after(head_count_kernel, blocks, kHeadThreads, st, sk, G.sort.n, G.heads) != cudaSuccess ||
        range_sort::launch_after(number_kernel, blocks, kHeadThreads, st, sk, G.sort.n, N, G.heads, err) != cudaSuccess)
      return FS_ERR_CUDA;
    launches += 2;
  }
  const int vec = ib == 4 ? 4 : 8;
  // 16-byte loads of dout where rows and addresses allow them, element by element otherwise
  const bool wide = dim % vec == 0 && aligned(dout, 16) && aligned(row_grads, 16);
  const int64_t most_rows = T < num_rows ? T : num_rows;
#define FS_GRAD(EI, EO, V)                                                                                        \
  do {                                                                                                            \
    if (small && wide) launch_small_vec<EI, EO, V>(most_rows, G, sv, count, dout, dim, scale, row_grads, cap_rows, st); \
    else if (small) launch_small_vec<EI, EO, 1>(most_rows, G, sv, count, dout, dim, scale, row_grads, cap_rows, st);    \
    else if (wide) launch_reduce_vec<EI, EO, V>(L, G, sk, sv, dout, dim, scale, row_grads, cap_rows, st);         \
    else launch_reduce_vec<EI, EO, 1>(L, G, sk, sv, dout, dim, scale, row_grads, cap_rows, st);                   \
  } while (0)
  if (ib == 4 && ob == 4) FS_GRAD(F32, F32, 4);
  else if (ib == 4) FS_GRAD(F32, Bf16, 4);
  else if (ob == 4) FS_GRAD(Bf16, F32, 8);
  else FS_GRAD(Bf16, Bf16, 8);
#undef FS_GRAD
  if (small) {
    count_launch(launches + 1);
    return launch_status();
  }
  const int64_t want = (L.tiles + kJoinWarps - 1) / kJoinWarps, most = int64_t(sm_count()) * kJoinPerSm;
  auto join = [&](auto kern) {
    kern<<<unsigned(want < most ? want : most), kJoinThreads, 0, st>>>(sk, G.sort.n, G.start, G.before,
                                                                       L.chunk_log2, dim, scale, row_grads, cap_rows,
                                                                       G.part_head, G.part_tail);
  };
  const bool wide4 = dim % 4 == 0 && aligned(row_grads, 4 * ob);
  if (ob == 4) wide4 ? join(grad_join_kernel<F32, 4>) : join(grad_join_kernel<F32, 1>);
  else wide4 ? join(grad_join_kernel<Bf16, 4>) : join(grad_join_kernel<Bf16, 1>);
  count_launch(launches + 2);
  return launch_status();
}
