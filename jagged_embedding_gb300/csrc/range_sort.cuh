// Stable counting sort of (ID, position) for batches of up to a few million
// entries, where a pass is bound by its launches and latencies, not by bytes
// (LSD radix sort over digits of at most 8 bits).
//
// The entries are cut into one contiguous range per block, as many blocks as
// fit on the GPU together.  A pass is three launches, each waiting for the one
// before it on the device (programmatic dependent launch), so that blocks are
// in place when their inputs are:
//   count:   a block's entries per digit, counts[digit][block];
//   scan:    a warp per digit: exclusive prefix over the blocks, digit totals;
//   scatter: the block walks its range in tiles: rank of every entry among the
//            tile's entries of its digit (ballots in a warp, warps in order),
//            staged in digit order in shared memory, written in runs.
// No block waits on another inside a launch.  What an earlier launch wrote is read past L1 (a block may be
// in place before its inputs are).  The first pass reads the IDs
// themselves and drops those out of range.
//
// 2M IDs of 24 bits: 77 us for three passes; the library's sort for large tables, four
// launches a pass over fixed tiles, takes 106 us here.  A row gradient call (rows of 32 bf16)
// with this sort and that one: 20,000 IDs 63 and 91 us, 200,000 81 and 106, 2M 193 and 245,
// 10M 735 and 794, 50M 3.69 and 3.51 ms: not worth a second way.
#pragma once

#include "fs_common.cuh"

namespace fs {
namespace range_sort {

// Block shape: 256 x 16 entries in 64 registers, 4 blocks per SM: the entries in registers of all
// blocks together are 2.5M, and fewer, larger tiles mean fewer barriers (a row gradient call of 2M entries 252 us;
// 512 x 8 in 32 registers 262, 1024 x 7 265, 5 blocks per SM 271, 3 264; match.any in place of the ballots 261).
constexpr int kThreads = 256, kWarps = kThreads / 32, kItems = 16, kTile = kThreads * kItems;
constexpr int kBits = 8, kBins = 1 << kBits;
constexpr int kPerSm = 4;            // resident blocks per SM
constexpr int kMaxBlocks = 1024;     // of one launch; sizes the counts
constexpr int64_t kLeast = 1024;     // entries a block is worth

struct Entries {
  const int64_t* ids;    // first pass
  int64_t R;
  const uint32_t* keys;  // later passes
  const uint32_t* vals;
};

struct Range {
  int64_t first;
  int64_t count;
};

// Block b's entries of n: equal shares, begun at multiples of 32.
__device__ __forceinline__ Range range_of(int64_t n) {
  const int64_t per = ((n + gridDim.x - 1) / gridDim.x + 31) / 32 * 32;
  const int64_t first = per * blockIdx.x;
  if (first >= n) return {n, 0};
  return {first, n - first < per ? n - first : per};
}

__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <bool FIRST>
__global__ void __launch_bounds__(kThreads, kPerSm) count_kernel(Entries in, int64_t T, const int64_t* n_dev, int shift,
                                                                 uint32_t mask, uint32_t* __restrict__ counts,
                                                                 int32_t* err) {
  __shared__ uint32_t bins[kBins];
  launch_next();
  for (int d = threadIdx.x; d < kBins; d += kThreads) bins[d] = 0u;
  wait_previous();
  __syncthreads();
  const Range r = range_of(FIRST ? T : __ldcg(n_dev));
  for (int64_t j = threadIdx.x; j < r.count; j += kTile) {
    if constexpr (FIRST) {
      int64_t id[kItems];
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if (j + i * kThreads < r.count) id[i] = __ldg(in.ids + r.first + j + i * kThreads);
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if (j + i * kThreads < r.count) {
          if (uint64_t(id[i]) < uint64_t(in.R)) atomicAdd(bins + ((uint32_t(id[i]) >> shift) & mask), 1u);
          else set_err(err, FS_ERR_ID_RANGE);
        }
    } else {
      uint32_t k[kItems];
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if (j + i * kThreads < r.count) k[i] = __ldcg(in.keys + r.first + j + i * kThreads);
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if (j + i * kThreads < r.count) atomicAdd(bins + ((k[i] >> shift) & mask), 1u);
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < kBins; d += kThreads) counts[int64_t(d) * gridDim.x + blockIdx.x] = bins[d];
}

constexpr int kScanThreads = 256, kScanBlocks = kBins / (kScanThreads / 32), kScanItems = 20;  // counts in flight per lane (8: 8 us more a sort)

static __global__ void __launch_bounds__(kScanThreads) scan_kernel(uint32_t* __restrict__ counts, int blocks,
                                                                   uint32_t* __restrict__ totals) {
  const int lane = threadIdx.x & 31, d = int(blockIdx.x) * (kScanThreads / 32) + int(threadIdx.x >> 5);
  launch_next();
  wait_previous();
  uint32_t* row = counts + int64_t(d) * blocks;
  uint32_t carry = 0;
  for (int b = lane; b - lane < blocks; b += 32 * kScanItems) {
    uint32_t c[kScanItems], x[kScanItems];
#pragma unroll
    for (int q = 0; q < kScanItems; ++q) x[q] = c[q] = b + q * 32 < blocks ? __ldcg(row + b + q * 32) : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int q = 0; q < kScanItems; ++q) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x[q], o);
        if (lane >= o) x[q] += y;
      }
#pragma unroll
    for (int q = 0; q < kScanItems; ++q) {
      if (b + q * 32 < blocks) row[b + q * 32] = carry + x[q] - c[q];
      carry += __shfl_sync(0xffffffffu, x[q], 31);
    }
  }
  if (lane == 0) totals[d] = carry;
}

template <bool FIRST>
__global__ void __launch_bounds__(kThreads, kPerSm) scatter_kernel(Entries in, int64_t T, int64_t* n_dev, int shift,
                                                                   uint32_t mask, const uint32_t* counts,
                                                                   const uint32_t* totals,
                                                                   uint32_t* __restrict__ out_k,
                                                                   uint32_t* __restrict__ out_v) {
  union Stage {
    uint32_t hist[kWarps][kBins];  // while ranking
    struct {
      uint32_t key[kTile];
      uint32_t val[kTile];
    } out;
  };
  __shared__ Stage sm;
  __shared__ uint32_t local_start[kBins], out_off[kBins], scratch[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  launch_next();
  wait_previous();
  uint32_t run = 0;  // thread d: where the next entry of digit d goes
  {
    const bool mine = int(threadIdx.x) < kBins;
    const uint32_t before = mine ? __ldcg(counts + int64_t(threadIdx.x) * gridDim.x + blockIdx.x) : 0u;
    uint32_t all;
    run = block_exclusive_scan<uint32_t>(mine ? __ldcg(totals + threadIdx.x) : 0u, scratch, &all) + before;
    if (FIRST && blockIdx.x == 0 && threadIdx.x == 0) *n_dev = all;
  }
  const Range r = range_of(FIRST ? T : __ldcg(n_dev));
  const int64_t tiles = (r.count + kTile - 1) / kTile;
  const int64_t per = tiles ? (r.count + tiles - 1) / tiles : 1;
  for (int64_t t0 = 0; t0 < r.count; t0 += per) {
    const int64_t base = r.first + t0;
    const int cnt = int(r.count - t0 < per ? r.count - t0 : per);
    const int items = (cnt + kThreads - 1) / kThreads;  // slots a thread has in this tile
    auto place = [&](int i) { return (warp * items + i) * 32 + lane; };  // slot order = entry order
    uint32_t key[kItems], rank[kItems];  // rank: ~0 = no entry
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      rank[i] = ~0u;
      key[i] = 0u;
      if (i < items && place(i) < cnt) {
        if constexpr (FIRST) {
          const int64_t id = __ldg(in.ids + base + place(i));
          key[i] = uint32_t(id);
          if (uint64_t(id) < uint64_t(in.R)) rank[i] = 0u;
        } else {
          key[i] = __ldcg(in.keys + base + place(i));
          rank[i] = 0u;
        }
      }
    }
    for (int j = threadIdx.x; j < kWarps * kBins; j += kThreads) (&sm.hist[0][0])[j] = 0u;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      if (i >= items) break;
      const bool live = rank[i] != ~0u;
      const uint32_t d = (key[i] >> shift) & mask;
      const unsigned lv = __ballot_sync(0xffffffffu, live);
      unsigned peers = live ? lv : ~lv;
#pragma unroll
      for (int b = 0; b < kBits; ++b) {
        const bool on = (d >> b) & 1u;
        const unsigned m = __ballot_sync(0xffffffffu, on);
        peers &= on ? m : ~m;
      }
      const unsigned lt = __popc(peers & lanemask_lt());
      const uint32_t before = live ? sm.hist[warp][d] : 0u;
      __syncwarp();
      if (live) {
        rank[i] = before + lt;
        if (lt == 0) sm.hist[warp][d] = before + __popc(peers);
      }
      __syncwarp();
    }
    __syncthreads();
    uint32_t val[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      if (rank[i] != ~0u) val[i] = FIRST ? uint32_t(base + place(i)) : __ldcg(in.vals + base + place(i));
    uint32_t tot = 0, all;
    if (int(threadIdx.x) < kBins) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const uint32_t c = sm.hist[w][threadIdx.x];
        sm.hist[w][threadIdx.x] = tot;
        tot += c;
      }
    }
    const uint32_t start = block_exclusive_scan<uint32_t>(tot, scratch, &all);
    if (int(threadIdx.x) < kBins) {
      local_start[threadIdx.x] = start;
      out_off[threadIdx.x] = run - start;  // staged entry j of digit d goes to out_off[d] + j (modulo 2^32)
      run += tot;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      if (rank[i] != ~0u) {
        const uint32_t d = (key[i] >> shift) & mask;
        rank[i] += local_start[d] + sm.hist[warp][d];
      }
    __syncthreads();  // the counts are read: their space becomes the staging area
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      if (rank[i] != ~0u) {
        sm.out.key[rank[i]] = key[i];
        sm.out.val[rank[i]] = val[i];
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const uint32_t j = threadIdx.x + i * kThreads;
      if (j < all) {
        const uint32_t k = sm.out.key[j];
        const uint32_t at = out_off[(k >> shift) & mask] + j;
        out_k[at] = k;
        out_v[at] = sm.out.val[j];
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host side

struct Ws {
  uint32_t *counts = nullptr, *totals = nullptr;
  int64_t* n = nullptr;  // valid entries, on the device
  uint32_t* k[2] = {nullptr, nullptr};
  uint32_t* v[2] = {nullptr, nullptr};
};

// The key and position arrays end on multiples of 64 entries.
template <class Cursor>
void take(int64_t T, Cursor& ws, Ws& W) {
  const int64_t most = (T + kLeast - 1) / kLeast;  // (at least blocks_for(T))
  W.counts = ws.template take<uint32_t>(size_t(kBins) * size_t(most < kMaxBlocks ? most : kMaxBlocks));
  W.totals = ws.template take<uint32_t>(kBins);
  W.n = ws.template take<int64_t>(1);
  const size_t padded = (size_t(T) + 63) / 64 * 64;
  for (int i = 0; i < 2; ++i) {
    W.k[i] = ws.template take<uint32_t>(padded);
    W.v[i] = ws.template take<uint32_t>(padded);
  }
}

inline int blocks_for(int64_t T) {
  int64_t b = int64_t(sm_count()) * kPerSm;
  if (b > kMaxBlocks) b = kMaxBlocks;
  if (b > (T + kLeast - 1) / kLeast) b = (T + kLeast - 1) / kLeast;
  return int(b < 1 ? 1 : b);
}

// A launch that may begin before the one in front of it ends (its kernel waits on the device).
template <class... P, class... A>
cudaError_t launch_after(void (*kern)(P...), int grid, int threads, cudaStream_t st, A... a) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(a)...);
}

inline int bits_for(uint64_t max_key) {
  int b = 1;
  while (b < 64 && (max_key >> b) != 0) ++b;
  return b;
}

// Sorts ids[0 .. T) (those below R) with their positions; *side: which of W.k / W.v holds the result.
inline fs_status sort(const int64_t* ids, int64_t T, int64_t R, int key_bits, const Ws& W, int32_t* err,
                      cudaStream_t st, int* side, int* launches) {
  const int blocks = blocks_for(T);
  const int passes = (key_bits + kBits - 1) / kBits, bits = (key_bits + passes - 1) / passes;
  const uint32_t mask = (1u << bits) - 1u;
  for (int p = 0; p < passes; ++p) {
    const int shift = p * bits, o = p & 1;
    const Entries in{ids, R, W.k[o ^ 1], W.v[o ^ 1]};
    cudaError_t e = cudaSuccess;
    if (p == 0) count_kernel<true><<<blocks, kThreads, 0, st>>>(in, T, W.n, shift, mask, W.counts, err);
    else e = launch_after(count_kernel<false>, blocks, kThreads, st, in, T, W.n, shift, mask, W.counts, err);
    if (e == cudaSuccess) e = launch_after(scan_kernel, kScanBlocks, kScanThreads, st, W.counts, blocks, W.totals);
    if (e == cudaSuccess)
      e = launch_after(p == 0 ? scatter_kernel<true> : scatter_kernel<false>, blocks, kThreads, st, in, T, W.n, shift,
                       mask, W.counts, W.totals, W.k[o], W.v[o]);
    if (e != cudaSuccess) return FS_ERR_CUDA;
    *launches += 3;
    *side = o;
  }
  return FS_OK;
}

}  // namespace range_sort
}  // namespace fs
