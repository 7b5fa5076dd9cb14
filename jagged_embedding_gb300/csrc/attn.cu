// Attention inside each sample of a jagged batch, and its backward pass, on
// the fifth-generation tensor cores.
//
// Row i of a sample of L positions, the last L - uih of them candidates, sees
// key j iff (j <= i or not causal) and (j < uih or j == i).
//   x = scale * q.k,  lse = log sum_j exp(x_j),  o = sum_j exp(x_j - lse) v_j
// backward, recomputing p = exp(x - lse):
//   delta = do.o,  ds = p * (do.v - delta)
//   dq = scale * sum_j ds k_j,  dk = scale * sum_i ds q_i,  dv = sum_i p do_i
//
// A sample is cut into tiles of 128 positions, the same for queries and keys.
// A planning kernel lists the tiles of all samples, those with the most work
// first, so that blocks taken in order leave no long tail.  One block per tile
// and head then walks the tiles that its rows (or, for dk and dv, its keys)
// meet: whole tiles that nothing of which is visible are never loaded.
//
// The backward pass is two kernels: one block per query tile for dq, one per
// key tile for dk and dv, each summing in its own accumulators, so every sum
// has a fixed order and nothing is added atomically; it recomputes x and do.v
// twice (7 products where a pass with atomic sums of dq needs 5).
#include <cuda_bf16.h>

#include <atomic>
#include <mutex>

#include "fs_common.cuh"
#include "tcgen.cuh"

namespace fs {
namespace {

constexpr int kTile = 128;                   // positions per tile
constexpr int kBox = kTile * 128;            // bytes of a TMA box: 128 rows of 64 bf16
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------- planning

struct Tile {
  int32_t begin;  // first position of the sample
  int32_t L, uih;
  int32_t t;      // tile index inside the sample
};

// Key tiles that query tile t meets: the first n (those of the history up to
// the causal limit), then, where its rows are all candidates, its own.
__device__ __forceinline__ int key_tiles(const Tile& x, bool causal, int& own) {
  const int end = min((x.t + 1) * kTile, x.L);
  const int lim = causal ? min(x.uih, end) : x.uih;
  const int n = (lim + kTile - 1) / kTile;
  own = x.t >= n ? 1 : 0;
  return n;
}

// Query tiles that key tile t meets: [first, first + n).
__device__ __forceinline__ int query_tiles(const Tile& x, bool causal, int& first) {
  const int all = (x.L + kTile - 1) / kTile;
  if (x.t * kTile >= x.uih) {  // candidates only: seen by themselves
    first = x.t;
    return 1;
  }
  first = causal ? x.t : 0;
  return all - first;
}

constexpr int kPlanThreads = 1024, kBuckets = 1024;

// Lists the tiles of all samples twice, by descending number of key tiles (for
// queries; an entry stands for `span` neighbouring tiles, and its t counts such
// groups) and of query tiles (for keys; only where by_key is given, span 1): a
// counting sort over the tile counts by one block.  The order among equals
// does not matter to any result.
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const int64_t* __restrict__ offsets, int64_t S, int64_t T,
                                                                 const int32_t* __restrict__ cand, bool causal,
                                                                 int span, int32_t* ntiles, Tile* by_query,
                                                                 Tile* by_key, int32_t* err) {
  __shared__ int32_t hist[2][kBuckets];
  __shared__ int32_t scan[32];
  for (int i = threadIdx.x; i < 2 * kBuckets; i += kPlanThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  auto bucket = [](int cost) { return kBuckets - min(cost, kBuckets); };  // most work first
  auto each = [&](bool report, auto f) {
    for (int64_t s = threadIdx.x; s < S; s += kPlanThreads) {
      const int64_t b = offsets[s], e = offsets[s + 1];
      if (b < 0 || e < b || e > T) {
        if (report) set_err(err, FS_ERR_BAD_OFFSETS);
        continue;
      }
      const int32_t L = int32_t(e - b);
      int32_t c = cand ? cand[s] : 0;
      if (c < 0 || c > L) {
        if (report) set_err(err, FS_ERR_INVALID_ARG);
        c = c < 0 ? 0 : L;
      }
      Tile x{int32_t(b), L, L - c, 0};
      for (; x.t * span * kTile < L; ++x.t) {
        int own, first;
        Tile last = x;  // the entry's last tile has the most key tiles
        last.t = min(x.t * span + span - 1, (L - 1) / kTile);
        const int nk = key_tiles(last, causal, own) + own;
        f(x, bucket(nk), bucket(query_tiles(x, causal, first)));
      }
    }
  };
  // Offsets that are not in order can describe more tiles than the lists hold:
  // then nothing is listed (the error word says so).
  int64_t total = 0;
  each(true, [&](const Tile&, int bq, int bk) {
    atomicAdd(&hist[0][bq], 1);
    if (by_key) atomicAdd(&hist[1][bk], 1);
  });
  __syncthreads();
  for (int w = 0; w < (by_key ? 2 : 1); ++w) {
    int32_t n;
    const int32_t mine = hist[w][threadIdx.x];
    const int32_t at = block_exclusive_scan<int32_t>(mine, scan, &n);
    hist[w][threadIdx.x] = at;
    total = n;
  }
  __syncthreads();
  const int64_t most = T / kTile + (S < T ? S : T);
  if (total > most) {
    if (threadIdx.x == 0) {
      set_err(err, FS_ERR_BAD_OFFSETS);
      *ntiles = 0;
    }
    return;
  }
  if (threadIdx.x == 0) *ntiles = int32_t(total);
  each(false, [&](const Tile& x, int bq, int bk) {
    by_query[atomicAdd(&hist[0][bq], 1)] = x;
    if (by_key) by_key[atomicAdd(&hist[1][bk], 1)] = x;
  });
}

// ------------------------------------------------------------- shared pieces

struct AttnArgs {
  const int32_t* ntiles;
  const Tile* tiles;
  int32_t heads, kv_heads;
  int64_t T;
  bool causal;
  float scale;
  __nv_bfloat16* o;        // forward: out
  const __nv_bfloat16* out;   // backward: out and dout
  const __nv_bfloat16* dout;
  float* lse;
  float* delta;            // [heads, T]: written by the dq kernel, read by the dk / dv kernel
  __nv_bfloat16 *dq, *dk, *dv;
  int64_t dq_stride, dk_stride, dv_stride;
  int32_t* err;
  uint64_t wait_ns;
};

// Wait of a whole warp for a barrier's phase, with a limit; sets the error word when it gives up.
// The hand-overs between the warps of a block come every few hundred cycles, so it polls without
// asking to sleep and looks at the clock only now and then.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t phase, const AttnArgs& a) {
  uint64_t t0 = 0;
  for (uint32_t polls = 1;; ++polls) {
    if (__all_sync(0xffffffffu, bulk::try_wait(bar, phase & 1u))) return true;
    if ((polls & 1023u) == 0) {
      const uint64_t now = bulk::global_ns();
      if (t0 == 0) t0 = now;
      if (__any_sync(0xffffffffu, now - t0 > a.wait_ns)) break;
    }
  }
  if ((threadIdx.x & 31) == 0) set_err(a.err, FS_ERR_TIMEOUT);
  return false;
}

// Tile of `rows` DH columns from position y of head h, as DH / 64 boxes (one thread).
template <int DH>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int h, int y, uint32_t bar) {
#pragma unroll
  for (int b = 0; b < DH / 64; ++b) tc::load_box(dst + b * kBox, map, h * DH + b * 64, y, bar);
}

// Rows [from, 128) of a loaded tile become zero (whole warp): they belong to
// another sample or to none, and a NaN there must not meet a zero weight.
template <int DH>
__device__ __forceinline__ void zero_rows(unsigned char* tile, int from) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int b = 0; b < DH / 64; ++b) {
    uint4* p = reinterpret_cast<uint4*>(tile + b * kBox);
    for (int i = from * 8 + lane; i < kTile * 8; i += 32) p[i] = make_uint4(0, 0, 0, 0);
  }
  bulk::fence_async_shared();
  __syncwarp();
}

// D[128 x 128] = A B^T over DH columns, both tiles K-major.  Called by a whole warp; lane 0 issues.
template <int DH>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t id = tc::idesc(kTile, kTile, false);
  d = tc::uni(d);
  const uint32_t da = tc::uni(tc::desc_k(a)), db = tc::uni(tc::desc_k(b));
  if ((threadIdx.x & 31) == 0) {
    tc::mma_ss<true>(d, tc::at(da, 0), tc::at(db, 0), id, false);
#pragma unroll
    for (int k = 1; k < DH / 16; ++k) {
      const uint32_t off = (k / 4) * kBox + (k % 4) * 32;
      tc::mma_ss<false>(d, tc::at(da, off), tc::at(db, off), id, true);
    }
  }
}

// D[128 x DH] (+)= A B, A [128 x 128] bf16 in tensor memory, its first 64 columns at a0, the
// others at a1, B a tile of 128 rows.  Called by a whole warp; lane 0 issues.
template <int DH>
__device__ __forceinline__ void mma_cols(uint32_t d, uint32_t a0, uint32_t a1, uint32_t b, bool acc) {
  constexpr uint32_t id = tc::idesc(kTile, DH, true);
  d = tc::uni(d), a0 = tc::uni(a0), a1 = tc::uni(a1);
  const uint32_t db = tc::uni(tc::desc_mn(b, kBox));
  const bool on = tc::uni(uint32_t(acc)) != 0;
  if ((threadIdx.x & 31) == 0) {
    tc::mma_ts<true>(d, a0, tc::at(db, 0), id, on);
#pragma unroll
    for (int k = 1; k < kTile / 16; ++k)
      tc::mma_ts<false>(d, (k < 4 ? a0 + 8 * k : a1 + 8 * (k - 4)), tc::at(db, k * 2048), id, true);
  }
}

// Commit by the lane that issues the products.
__device__ __forceinline__ void commit(uint32_t bar) {
  bar = tc::uni(bar);
  if ((threadIdx.x & 31) == 0) tc::commit(bar);
}

// 32 fp32 columns, scaled, as bf16 to 64 contiguous bytes.
__device__ __forceinline__ void store32(__nv_bfloat16* p, const float* x, float f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 v;
    v.x = tc::pack2(x[8 * i] * f, x[8 * i + 1] * f);
    v.y = tc::pack2(x[8 * i + 2] * f, x[8 * i + 3] * f);
    v.z = tc::pack2(x[8 * i + 4] * f, x[8 * i + 5] * f);
    v.w = tc::pack2(x[8 * i + 6] * f, x[8 * i + 7] * f);
    reinterpret_cast<uint4*>(p)[i] = v;
  }
}

template <int DH>
constexpr int tile_bytes() { return DH / 64 * kBox; }

__device__ __forceinline__ unsigned char* align_smem(unsigned char* p) {
  return p + ((1024u - (bulk::smem_addr(p) & 1023u)) & 1023u);
}

// ------------------------------------------------------------- forward

// One block per SM works through units: two query tiles that read the same
// keys and values, so each loaded tile serves two products.  They are the same
// positions of two query heads that share a key/value head, or, where the
// number of sharing heads is odd, neighbouring tiles of one head.  A warpgroup
// per query tile, one row a thread, does the softmax; one warp issues the
// products, one the loads, which run ahead into the next unit.  Products of one
// query tile run under the softmax of the other.  Tensor memory: x of each tile in 128
// columns, p (bf16) over it, o beside them.
// A softmax thread holds a row of 128 scores: the third warpgroup (loads,
// products, two idle warps) gives registers to the other two.  384 threads are
// launched with kFwdRegs each; 2 * 128 * 208 + 128 * 88 is that total.
constexpr int kFwdThreads = 384, kFwdRegs = 168;
template <int DH> constexpr int fwd_slots() { return DH == 64 ? 8 : 4; }
template <int DH> constexpr int fwd_smem() { return tile_bytes<DH>() * (2 + fwd_slots<DH>()) + 1024; }

struct FwdUnit {
  Tile x;
  int head[2], row[2];  // query head and tile index of each query tile
  int nk[2], own[2];    // key tiles of the history, and whether its own tile follows
  int kv_head, common, n;
  bool by_head, both;

  __device__ __forceinline__ FwdUnit(const Tile& tile, int part, const AttnArgs& a) : x(tile) {
    const int group = a.heads / a.kv_heads;
    by_head = group % 2 == 0;
    if (by_head) {
      head[0] = 2 * part, head[1] = 2 * part + 1;
      row[0] = row[1] = x.t;
    } else {
      head[0] = head[1] = part;
      row[0] = 2 * x.t, row[1] = 2 * x.t + 1;
    }
    kv_head = head[0] / group;
    both = row[1] * kTile < x.L;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      Tile y = x;
      y.t = row[i];
      nk[i] = key_tiles(y, a.causal, own[i]);
    }
    if (!both) nk[1] = own[1] = 0;
    common = max(nk[0], nk[1]);
    n = common + own[0] + (by_head ? 0 : own[1]);
  }
  // The unit's j-th key tile, and whether query tile i meets it.
  __device__ __forceinline__ int key_tile(int j) const {
    return j < common ? j : ((j == common && own[0]) || by_head ? row[0] : row[1]);
  }
  __device__ __forceinline__ bool meets(int i, int j) const {
    if (by_head) return true;
    return i ? j < nk[1] || (own[1] && j == common + own[0]) : j < nk[0] || (own[0] && j == common);
  }
};

// Units of this block: dealt out in rounds, back and forth, most work first.
struct Deal {
  int64_t units;
  int64_t round = 0;
  __device__ __forceinline__ int64_t next() {
    const int64_t g = gridDim.x, b = blockIdx.x;
    const int64_t u = round * g + ((round & 1) ? g - 1 - b : b);
    ++round;
    return u < units ? u : -1;
  }
};

template <int DH>
__global__ void __launch_bounds__(kFwdThreads, 1) attn_fwd_kernel(const __grid_constant__ CUtensorMap mq,
                                                                  const __grid_constant__ CUtensorMap mk,
                                                                  const __grid_constant__ CUtensorMap mv, AttnArgs a,
                                                                  int parts) {
  constexpr int TB = tile_bytes<DH>(), NS = fwd_slots<DH>();
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t bars[8 + 2 * NS];
  __shared__ uint32_t tmem_at;
  const int64_t units = int64_t(*a.ntiles) * parts;
  if (int64_t(blockIdx.x) >= units) return;
  unsigned char* smem = align_smem(raw);
  const uint32_t q_at = bulk::smem_addr(smem), kv_at = q_at + 2 * TB;
  const uint32_t bar = bulk::smem_addr(bars);
  const uint32_t q_full = bar, q_free = bar + 8, s_full = bar + 16, p_ready = bar + 32, o_full = bar + 48, drain = bar + 56,
                 full = bar + 64, free = bar + 64 + 8 * NS;
  const int warp = int(tc::uni(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (warp == 8) {
    if (lane == 0) {
      for (int i = 0; i < 8 + 2 * NS; ++i) bulk::mbar_init(bar + 8 * i, i == 4 || i == 5 ? 4 : 1);
      bulk::fence_init();
    }
    __syncwarp();
    tc::alloc(&tmem_at, 512);
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t s_at = tmem_at, o_at = tmem_at + 256;  // of query tile 0; tile 1's follow
  Deal deal{units};
  bool ok = true;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 9) {
    // loads: the two query tiles of a unit, then its key and value tiles, in order, through NS slots
    int64_t slot = 0;
    for (int k = 0;; ++k) {
      const int64_t u = deal.next();
      if (u < 0) break;
      const FwdUnit f(a.tiles[u / parts], int(u % parts), a);
      if (k > 0 && !(ok = wait(q_free, k - 1, a))) break;
      if (lane == 0) {
        bulk::arrive_expect_tx(q_full, f.both ? 2 * TB : TB);
        load_tile<DH>(q_at, &mq, f.head[0], f.x.begin + f.row[0] * kTile, q_full);
        if (f.both) load_tile<DH>(q_at + TB, &mq, f.head[1], f.x.begin + f.row[1] * kTile, q_full);
      }
      for (int j = 0; ok && j < 2 * f.n; ++j, ++slot) {
        const int s = int(slot % NS);
        if (slot >= NS && !(ok = wait(free + 8 * s, uint32_t(slot / NS - 1), a))) break;
        if (lane == 0) {
          bulk::arrive_expect_tx(full + 8 * s, TB);
          load_tile<DH>(kv_at + s * TB, j & 1 ? &mv : &mk, f.kv_head, f.x.begin + f.key_tile(j >> 1) * kTile,
                        full + 8 * s);
        }
      }
      if (!ok) break;
    }
    if (!ok)  // gave up: let what is in flight land
      for (int64_t s = slot > NS ? slot - NS : 0; s < slot; ++s)
        bulk::warp_wait(full + 8 * int(s % NS), uint32_t(s / NS) & 1u, a.wait_ns);
    } else if (warp == 8) {
    // products: at step j, o += p v of key tile j - 1 and x of key tile j, of query tile 0, then of 1
    int64_t slot = 0;           // of the unit's first key tile
    uint32_t done[2] = {0, 0};  // p's consumed
    for (int k = 0; ok; ++k) {
      const int64_t u = deal.next();
      if (u < 0) break;
      const FwdUnit f(a.tiles[u / parts], int(u % parts), a);
      if (!(ok = wait(q_full, k, a))) break;
      uint32_t acc[2] = {0, 0};
      for (int j = 0; j <= f.n; ++j) {
        const int64_t ks = slot + 2 * j, vs = ks - 1;  // slots of key tile j and value tile j - 1
        const uint32_t k_tile = kv_at + uint32_t(ks % NS) * TB, v_tile = kv_at + uint32_t(vs % NS + NS) % NS * TB;
        if (j > 0) {
          if (!(ok = wait(full + 8 * int(vs % NS), uint32_t(vs / NS), a))) break;
          const int valid = f.x.L - f.key_tile(j - 1) * kTile;
          if (valid < kTile) zero_rows<DH>(smem + 2 * TB + int(vs % NS) * TB, valid);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 1 && !f.both) continue;
          if (j > 0 && f.meets(i, j - 1)) {
            if (!(ok = wait(p_ready + 8 * i, done[i], a))) break;
            ++done[i];
            tc::fence_after();
            mma_cols<DH>(o_at + i * DH, s_at + 128 * i, s_at + 128 * i + 32, v_tile, acc[i] != 0);
            acc[i] = 1;
          }
          if (j < f.n && f.meets(i, j)) {
            // x overwrites p: the products execute in the order they are issued
            if (!(ok = wait(full + 8 * int(ks % NS), uint32_t(ks / NS), a))) break;
            mma_rows<DH>(s_at + 128 * i, q_at + i * TB, k_tile);
            commit(s_full + 8 * i);
          }
        }
        if (!ok) break;
        if (j > 0) commit(free + 8 * int(vs % NS));
        if (j < f.n) commit(free + 8 * int(ks % NS));
        if (j == f.n - 1) commit(q_free);
        if (j == f.n) commit(o_full);
      }
      slot += 2 * f.n;
    }
    if (!ok) {
      if (lane == 0) tc::commit(drain);
      bulk::warp_wait(drain, 0, a.wait_ns);
    }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int i = warp >> 2;  // query tile of this warpgroup
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t x_at = s_at + 128 * i + lanes, acc_at = o_at + DH * i + lanes;
    const float c = a.scale * kLog2e;
    uint32_t seen = 0;
    for (int k = 0; ok; ++k) {
      const int64_t u = deal.next();
      if (u < 0) break;
      const FwdUnit f(a.tiles[u / parts], int(u % parts), a);
      const int tile = i ? f.row[1] : f.row[0];
      const int row = tile * kTile + int(threadIdx.x & 127);  // position inside the sample
      float m = -INFINITY, l = 0.f;
      bool first = true;
      for (int j = 0; j < f.n; ++j) {
        if ((i == 1 && !f.both) || !f.meets(i, j)) continue;
        if (!(ok = wait(s_full + 8 * i, seen, a))) break;
        ++seen;
        tc::fence_after();
        float s[128];
#pragma unroll
        for (int b = 0; b < 4; ++b) tc::ld32(x_at + 32 * b, s + 32 * b);
        tc::wait_ld();
#pragma unroll
        for (int b = 0; b < 4; ++b) tc::tie32(s + 32 * b);
        const int k0 = f.key_tile(j) * kTile;
        if (k0 + kTile > f.x.uih || (a.causal && k0 + kTile > tile * kTile)) {
          const int lim = (a.causal ? min(f.x.uih, row + 1) : f.x.uih) - k0, self = row - k0;
#pragma unroll
          for (int q = 0; q < 128; ++q) s[q] = (q < lim || q == self) ? s[q] : -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int q = 4; q < 124; q += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], fmaxf(s[q + e], s[q + 4 + e]));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[124 + e]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (first) {
          m = top;
          first = false;
        } else {
          // the sums keep an older maximum until a row's has grown by 2^8: p stays
          // below 2^8, its rounding relative, and o is rescaled only then
          const bool grow = (top - m) * c > 8.f;
          if (__any_sync(0xffffffffu, grow)) {
            const float mn = grow ? top : m, g = tc::ex2((m - mn) * c);
            m = mn;
            l *= g;
#pragma unroll
            for (int b = 0; b < DH / 32; ++b) {
              float o[32];
              tc::ld32(acc_at + 32 * b, o);
              tc::wait_ld();
              tc::tie32(o);
#pragma unroll
              for (int q = 0; q < 32; q += 2) tc::mul2(o + q, g, g);
              tc::st32(acc_at + 32 * b, reinterpret_cast<const uint32_t*>(o));
            }
          }
        }
        const float mc = -m * c;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t p[64];
#pragma unroll
        for (int q = 0; q < 128; q += 4) {
          tc::fma2(s + q, c, c, mc, mc);
          tc::fma2(s + q + 2, c, c, mc, mc);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[q + e] = tc::ex2(s[q + e]);
          tc::add2(sum, s[q], s[q + 1]);
          tc::add2(sum + 2, s[q + 2], s[q + 3]);
          p[q / 2] = tc::pack2(s[q], s[q + 1]);
          p[q / 2 + 1] = tc::pack2(s[q + 2], s[q + 3]);
          if (q == 60) tc::st32(x_at, p);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tc::st32(x_at + 32, p + 32);
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::arrive(p_ready + 8 * i);
      }
      if (!ok || !(ok = wait(o_full, k, a))) break;
      tc::fence_after();
      if (i == 1 && !f.both) continue;
      const int64_t pos = int64_t(f.x.begin) + row;
      const int head = i ? f.head[1] : f.head[0];
      const float inv = 1.f / l;
#pragma unroll
      for (int b = 0; b < DH / 32; ++b) {
        float o[32];
        tc::ld32(acc_at + 32 * b, o);
        tc::wait_ld();
        tc::tie32(o);
        if (row < f.x.L) store32(a.o + (pos * a.heads + head) * DH + 32 * b, o, inv);
      }
      if (row < f.x.L) a.lse[int64_t(head) * a.T + pos] = (m * c + log2f(l)) * (1.f / kLog2e);
      tc::fence_before();
    }
  }
  __syncthreads();
  if (warp == 8) {
    tc::fence_after();
    tc::dealloc(tmem_at, 512);
  }
}

// ------------------------------------------------------------- backward

constexpr int kBwdThreads = 288;  // eight warps for the elementwise part, one for loads and products
template <int DH> constexpr int bwd_smem() { return tile_bytes<DH>() * 6 + 1024; }

// dq of one query tile and head.  A thread holds one query row and 64 of the
// 128 keys.  Per key tile: x = q k^T and do v^T into 128 columns each; p = exp(x - lse)
// stays in registers and frees x, so the next tile's x is computed while
// ds = p * (do v^T - delta) is formed; ds (bf16) goes over do v^T and multiplies k.
template <int DH>
__global__ void __launch_bounds__(kBwdThreads, 1) attn_dq_kernel(const __grid_constant__ CUtensorMap mq,
                                                                 const __grid_constant__ CUtensorMap mk,
                                                                 const __grid_constant__ CUtensorMap mv,
                                                                 const __grid_constant__ CUtensorMap mdo, AttnArgs a) {
  constexpr int TB = tile_bytes<DH>();
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t bars[12];
  __shared__ uint32_t tmem_at;
  __shared__ float half_delta[2][kTile];
  const int head = int(blockIdx.x % unsigned(a.heads));
  const int64_t at = blockIdx.x / unsigned(a.heads);
  if (at >= *a.ntiles) return;
  const Tile x = a.tiles[at];
  const int kv_head = head / (a.heads / a.kv_heads);
  int own;
  const int nk = key_tiles(x, a.causal, own);
  const int n = nk + own;
  unsigned char* smem = align_smem(raw);
  const uint32_t q_at = bulk::smem_addr(smem), do_at = q_at + TB, k_at = do_at + TB, v_at = k_at + 2 * TB;
  const uint32_t bar = bulk::smem_addr(bars);
  const uint32_t q_full = bar, k_full = bar + 8, v_full = bar + 24, s_full = bar + 40, dp_full = bar + 48,
                 s_read = bar + 56, ds_ready = bar + 64, dq_done = bar + 72, drain = bar + 80, fin = bar + 88;
  const int warp = int(tc::uni(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (warp == 8) {
    if (lane == 0) {
      tc::prefetch_map(&mq), tc::prefetch_map(&mk), tc::prefetch_map(&mv), tc::prefetch_map(&mdo);
      for (int i = 0; i < 12; ++i) bulk::mbar_init(bar + 8 * i, i == 7 || i == 8 ? 8 : 1);
      bulk::fence_init();
    }
    __syncwarp();
    tc::alloc(&tmem_at, 512);
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t s_at = tmem_at, dp_at = tmem_at + 128, dq_at = tmem_at + 256;
  auto key_tile = [&](int j) { return j < nk ? j : x.t; };

  if (warp == 8) {
    int loaded_k = 0, loaded_v = 0;
    auto load_k = [&](int j) {
      if (lane == 0) {
        bulk::arrive_expect_tx(k_full + 8 * (j & 1), TB);
        load_tile<DH>(k_at + (j & 1) * TB, &mk, kv_head, x.begin + key_tile(j) * kTile, k_full + 8 * (j & 1));
      }
      loaded_k = j + 1;
    };
    auto load_v = [&](int j) {
      if (lane == 0) {
        bulk::arrive_expect_tx(v_full + 8 * (j & 1), TB);
        load_tile<DH>(v_at + (j & 1) * TB, &mv, kv_head, x.begin + key_tile(j) * kTile, v_full + 8 * (j & 1));
      }
      loaded_v = j + 1;
    };
    auto key_ready = [&](int j) {
      if (!wait(k_full + 8 * (j & 1), j >> 1, a)) return false;
      const int valid = x.L - key_tile(j) * kTile;
      if (valid < kTile) zero_rows<DH>(smem + TB * (2 + (j & 1)), valid);
      return true;
    };
    if (lane == 0) {
      bulk::arrive_expect_tx(q_full, 2 * TB);
      load_tile<DH>(q_at, &mq, head, x.begin + x.t * kTile, q_full);
      load_tile<DH>(do_at, &mdo, head, x.begin + x.t * kTile, q_full);
    }
    for (int j = 0; j < 2 && j < n; ++j) {
      load_k(j);
      load_v(j);
    }
    bool ok = wait(q_full, 0, a) && key_ready(0) && wait(v_full, 0, a);
    if (ok) {
      mma_rows<DH>(s_at, q_at, k_at);
      commit(s_full);
      mma_rows<DH>(dp_at, do_at, v_at);
      commit(dp_full);
    }
    for (int j = 0; ok && j < n; ++j) {
      const int st = j & 1, nx = st ^ 1;
      if (j + 1 < n) {
        if (!(ok = key_ready(j + 1) && wait(s_read, j, a))) break;
        tc::fence_after();
        mma_rows<DH>(s_at, q_at, k_at + nx * TB);
        commit(s_full);
      }
      if (!(ok = wait(ds_ready, j, a))) break;
      tc::fence_after();
      mma_cols<DH>(dq_at, dp_at, dp_at + 64, k_at + st * TB, j != 0);
      commit(j + 1 < n ? dq_done : fin);
      if (j + 1 < n) {
        if (!(ok = wait(v_full + 8 * nx, (j + 1) >> 1, a))) break;
        // do v^T overwrites ds: the products execute in the order they are issued
        mma_rows<DH>(dp_at, do_at, v_at + nx * TB);
        commit(dp_full);
      }
      if (j + 2 < n) {
        load_v(j + 2);  // (ds_ready: the product that read this stage is done)
        if (!(ok = wait(dq_done, j, a))) break;
        load_k(j + 2);
      }
    }
    if (!ok) {
      if (lane == 0) tc::commit(drain);
      bulk::warp_wait(drain, 0, a.wait_ns);
      bulk::warp_wait(q_full, 0, a.wait_ns);
      for (int s = 0; s < 2; ++s) {
        if (loaded_k > s) bulk::warp_wait(k_full + 8 * s, ((loaded_k - 1 - s) >> 1) & 1, a.wait_ns);
        if (loaded_v > s) bulk::warp_wait(v_full + 8 * s, ((loaded_v - 1 - s) >> 1) & 1, a.wait_ns);
      }
    }
  } else {
    const int r = threadIdx.x & 127, half = threadIdx.x >> 7;
    const int row = x.t * kTile + r;
    const bool live = row < x.L;
    const int64_t pos = int64_t(x.begin) + row;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t cols = 64 * half;
    const float c = a.scale * kLog2e;
    // delta = dout.out of the row, half of the columns each
    float d = 0.f;
    if (live) {
      const uint4* po = reinterpret_cast<const uint4*>(a.out + (pos * a.heads + head) * DH + half * (DH / 2));
      const uint4* pg = reinterpret_cast<const uint4*>(a.dout + (pos * a.heads + head) * DH + half * (DH / 2));
#pragma unroll
      for (int i = 0; i < DH / 16; ++i) {
        const uint4 u = __ldg(po + i), w = __ldg(pg + i);
        const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          d = fmaf(__uint_as_float(uu[q] << 16), __uint_as_float(ww[q] << 16), d);
          d = fmaf(__uint_as_float(uu[q] & 0xFFFF0000u), __uint_as_float(ww[q] & 0xFFFF0000u), d);
        }
      }
    }
    half_delta[half][r] = d;
    asm volatile("bar.sync 1, 256;" ::: "memory");
    const float delta = half_delta[0][r] + half_delta[1][r];
    if (live && half == 0) a.delta[int64_t(head) * a.T + pos] = delta;
    const float lse2 = live ? a.lse[int64_t(head) * a.T + pos] * kLog2e : 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (!(ok = wait(s_full, j, a))) break;
      tc::fence_after();
      float p[64];
      tc::ld32(s_at + lanes + cols, p);
      tc::ld32(s_at + lanes + cols + 32, p + 32);
      tc::wait_ld();
      tc::tie32(p);
      tc::tie32(p + 32);
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::arrive(s_read);
      const int k0 = key_tile(j) * kTile + int(cols);
      const bool masked = k0 - int(cols) + kTile > x.uih || (a.causal && k0 - int(cols) + kTile > x.t * kTile);
      const int lim = (a.causal ? min(x.uih, row + 1) : x.uih) - k0, self = row - k0;
#pragma unroll
      for (int i = 0; i < 64; i += 2) {
        tc::fma2(p + i, c, c, -lse2, -lse2);
        p[i] = tc::ex2(p[i]);
        p[i + 1] = tc::ex2(p[i + 1]);
      }
      if (!(ok = wait(dp_full, j, a))) break;
      tc::fence_after();
      uint32_t w[32];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float g[32];
        tc::ld32(dp_at + lanes + cols + 32 * b, g);
        tc::wait_ld();
        tc::tie32(g);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          tc::add2(g + i, -delta, -delta);
          tc::mul2(g + i, p[32 * b + i], p[32 * b + i + 1]);
        }
        if (masked) {
#pragma unroll
          for (int i = 0; i < 32; ++i) g[i] = (32 * b + i < lim || 32 * b + i == self) ? g[i] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 32; i += 2) w[16 * b + i / 2] = tc::pack2(g[i], g[i + 1]);
      }
      tc::st32(dp_at + lanes + cols, w);
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::arrive(ds_ready);
    }
    if (ok && wait(fin, 0, a)) {
      tc::fence_after();
#pragma unroll
      for (int b = 0; b < DH / 64; ++b) {
        const int col = half * (DH / 2) + 32 * b;
        float g[32];
        tc::ld32(dq_at + lanes + col, g);
        tc::wait_ld();
        tc::tie32(g);
        if (live) store32(a.dq + pos * a.dq_stride + head * DH + col, g, a.scale);
      }
      tc::fence_before();
    }
  }
  __syncthreads();
  if (warp == 8) {
    tc::fence_after();
    tc::dealloc(tmem_at, 512);
  }
}

// dk and dv of one key tile and key/value head, over the query heads that
// share it and the query tiles that see it.  A thread holds one key and 64 of
// the 128 queries (everything transposed: x^T = k q^T, v do^T).  p^T (bf16)
// goes over x^T and multiplies do, then the next x^T is computed while
// ds^T = p^T * (v do^T - delta) is formed; ds^T goes over v do^T and multiplies q.
template <int DH>
__global__ void __launch_bounds__(kBwdThreads, 1) attn_dkv_kernel(const __grid_constant__ CUtensorMap mq,
                                                                  const __grid_constant__ CUtensorMap mk,
                                                                  const __grid_constant__ CUtensorMap mv,
                                                                  const __grid_constant__ CUtensorMap mdo, AttnArgs a) {
  constexpr int TB = tile_bytes<DH>();
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t bars[10];
  __shared__ uint32_t tmem_at;
  __shared__ __align__(16) float row_lse[2][kTile], row_delta[2][kTile];
  const int kv_head = int(blockIdx.x % unsigned(a.kv_heads));
  const int64_t at = blockIdx.x / unsigned(a.kv_heads);
  if (at >= *a.ntiles) return;
  const Tile x = a.tiles[at];
  const int group = a.heads / a.kv_heads;
  int first;
  const int nq = query_tiles(x, a.causal, first);
  const int n = nq * group;
  unsigned char* smem = align_smem(raw);
  const uint32_t k_at = bulk::smem_addr(smem), v_at = k_at + TB, q_at = v_at + TB;  // then two stages of (q, do)
  const uint32_t bar = bulk::smem_addr(bars);
  const uint32_t k_full = bar, q_full = bar + 8, s_full = bar + 24, dp_full = bar + 32, p_ready = bar + 40,
                 ds_ready = bar + 48, done = bar + 56, drain = bar + 64, fin = bar + 72;
  const int warp = int(tc::uni(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (warp == 8) {
    if (lane == 0) {
      tc::prefetch_map(&mq), tc::prefetch_map(&mk), tc::prefetch_map(&mv), tc::prefetch_map(&mdo);
      for (int i = 0; i < 10; ++i) bulk::mbar_init(bar + 8 * i, i == 5 || i == 6 ? 8 : 1);
      bulk::fence_init();
    }
    __syncwarp();
    tc::alloc(&tmem_at, 512);
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t s_at = tmem_at, dp_at = tmem_at + 128, dv_at = tmem_at + 256, dk_at = tmem_at + 256 + DH;
  auto query_tile = [&](int j) { return first + j % nq; };
  auto query_head = [&](int j) { return kv_head * group + j / nq; };

  if (warp == 8) {
    int loaded = 0;
    auto load_q = [&](int j) {
      if (lane == 0) {
        const uint32_t b = q_full + 8 * (j & 1), to = q_at + (j & 1) * 2 * TB;
        const int y = x.begin + query_tile(j) * kTile;
        bulk::arrive_expect_tx(b, 2 * TB);
        load_tile<DH>(to, &mq, query_head(j), y, b);
        load_tile<DH>(to + TB, &mdo, query_head(j), y, b);
      }
      loaded = j + 1;
    };
    auto query_ready = [&](int j) {
      if (!wait(q_full + 8 * (j & 1), j >> 1, a)) return false;
      const int valid = x.L - query_tile(j) * kTile;
      if (valid < kTile) {
        zero_rows<DH>(smem + TB * (2 + 2 * (j & 1)), valid);
        zero_rows<DH>(smem + TB * (3 + 2 * (j & 1)), valid);
      }
      return true;
    };
    if (lane == 0) {
      bulk::arrive_expect_tx(k_full, 2 * TB);
      load_tile<DH>(k_at, &mk, kv_head, x.begin + x.t * kTile, k_full);
      load_tile<DH>(v_at, &mv, kv_head, x.begin + x.t * kTile, k_full);
    }
    for (int j = 0; j < 2 && j < n; ++j) load_q(j);
    bool ok = wait(k_full, 0, a) && query_ready(0);
    if (ok) {
      mma_rows<DH>(s_at, k_at, q_at);
      commit(s_full);
      mma_rows<DH>(dp_at, v_at, q_at + TB);
      commit(dp_full);
    }
    for (int j = 0; ok && j < n; ++j) {
      const uint32_t cur = q_at + (j & 1) * 2 * TB, nxt = q_at + ((j + 1) & 1) * 2 * TB;
      if (j + 1 < n && !(ok = query_ready(j + 1))) break;
      if (!(ok = wait(p_ready, j, a))) break;
      tc::fence_after();
      mma_cols<DH>(dv_at, s_at, s_at + 64, cur + TB, j != 0);
      if (j + 1 < n) {  // x^T overwrites p^T: the products execute in the order they are issued
        mma_rows<DH>(s_at, k_at, nxt);
        commit(s_full);
      }
      if (!(ok = wait(ds_ready, j, a))) break;
      tc::fence_after();
      mma_cols<DH>(dk_at, dp_at, dp_at + 64, cur, j != 0);
      commit(j + 1 < n ? done : fin);
      if (j + 1 < n) {
        mma_rows<DH>(dp_at, v_at, nxt + TB);
        commit(dp_full);
      }
      if (j + 2 < n) {
        if (!(ok = wait(done, j, a))) break;
        load_q(j + 2);
      }
    }
    if (!ok) {
      if (lane == 0) tc::commit(drain);
      bulk::warp_wait(drain, 0, a.wait_ns);
      bulk::warp_wait(k_full, 0, a.wait_ns);
      for (int s = 0; s < 2; ++s)
        if (loaded > s) bulk::warp_wait(q_full + 8 * s, ((loaded - 1 - s) >> 1) & 1, a.wait_ns);
    }
  } else {
    const int r = threadIdx.x & 127, half = threadIdx.x >> 7;
    const int key = x.t * kTile + r;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t cols = 64 * half;
    const float c = a.scale * kLog2e;
    // lse (in powers of two) or delta of query r of tile j; queries past the sample's end weigh nothing
    auto row_value = [&](int j) {
      const int i = query_tile(j) * kTile + r;
      const int64_t at = int64_t(query_head(j)) * a.T + x.begin + i;
      if (half == 0) return i < x.L ? a.lse[at] * kLog2e : INFINITY;
      return i < x.L ? a.delta[at] : 0.f;
    };
    auto put_value = [&](int j, float v) { (half == 0 ? row_lse : row_delta)[j & 1][r] = v; };
    put_value(0, row_value(0));
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      // one barrier a tile: this tile's values are in, and the last tile's are read
      asm volatile("bar.sync 1, 256;" ::: "memory");
      float next = 0.f;
      if (j + 1 < n) next = row_value(j + 1);
      ok = ok && wait(s_full, j, a);
      if (!ok) continue;  // every warp keeps meeting the barrier
      tc::fence_after();
      float p[64];
      tc::ld32(s_at + lanes + cols, p);
      tc::ld32(s_at + lanes + cols + 32, p + 32);
      tc::wait_ld();
      tc::tie32(p);
      tc::tie32(p + 32);
      const float4* ls = reinterpret_cast<const float4*>(&row_lse[j & 1][cols]);
#pragma unroll
      for (int i = 0; i < 64; i += 4) {
        const float4 z = ls[i / 4];
        tc::fma2(p + i, c, c, -z.x, -z.y);
        tc::fma2(p + i + 2, c, c, -z.z, -z.w);
#pragma unroll
        for (int q = 0; q < 4; ++q) p[i + q] = tc::ex2(p[i + q]);
      }
      const int i0 = query_tile(j) * kTile;
      if (x.t * kTile + kTile > x.uih || (a.causal && i0 < x.t * kTile + kTile)) {
        // query i0 + cols + i sees this key from `from` on, or only where it is the key's own position
        const int self = key - i0 - int(cols);
        const int from = key >= x.uih ? 128 : (a.causal ? self : -1);
#pragma unroll
        for (int i = 0; i < 64; ++i) p[i] = (i >= from || i == self) ? p[i] : 0.f;
      }
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 64; i += 2) w[i / 2] = tc::pack2(p[i], p[i + 1]);
      tc::st32(s_at + lanes + cols, w);
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::arrive(p_ready);
      if (j + 1 < n) put_value(j + 1, next);
      ok = wait(dp_full, j, a);
      if (!ok) continue;
      tc::fence_after();
      const float4* dl = reinterpret_cast<const float4*>(&row_delta[j & 1][cols]);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float g[32];
        tc::ld32(dp_at + lanes + cols + 32 * b, g);
        tc::wait_ld();
        tc::tie32(g);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 z = dl[8 * b + i / 4];
          tc::add2(g + i, -z.x, -z.y);
          tc::add2(g + i + 2, -z.z, -z.w);
          tc::mul2(g + i, p[32 * b + i], p[32 * b + i + 1]);
          tc::mul2(g + i + 2, p[32 * b + i + 2], p[32 * b + i + 3]);
          w[16 * b + i / 2] = tc::pack2(g[i], g[i + 1]);
          w[16 * b + i / 2 + 1] = tc::pack2(g[i + 2], g[i + 3]);
        }
      }
      tc::st32(dp_at + lanes + cols, w);
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::arrive(ds_ready);
    }
    if (ok && wait(fin, 0, a)) {
      tc::fence_after();
      const int64_t pos = int64_t(x.begin) + key;
      __nv_bfloat16* to = half == 0 ? a.dv + pos * a.dv_stride : a.dk + pos * a.dk_stride;
      const uint32_t from = half == 0 ? dv_at : dk_at;
      const float f = half == 0 ? 1.f : a.scale;
#pragma unroll
      for (int b = 0; b < DH / 32; ++b) {
        float g[32];
        tc::ld32(from + lanes + 32 * b, g);
        tc::wait_ld();
        tc::tie32(g);
        if (key < x.L) store32(to + kv_head * DH + 32 * b, g, f);
      }
      tc::fence_before();
    }
  }
  __syncthreads();
  if (warp == 8) {
    tc::fence_after();
    tc::dealloc(tmem_at, 512);
  }
}

// ------------------------------------------------------------- host side

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult got;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &got) == cudaSuccess &&
        got == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
    else
      cudaGetLastError();
  });
  return fn;
}

// Map of [T, width] bf16 with rows `stride` elements apart, in boxes of 128 rows of 64 columns.
bool encode(CUtensorMap* map, const void* base, int64_t T, int64_t width, int64_t stride) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cuuint64_t(width), cuuint64_t(T)}, strides[1] = {cuuint64_t(stride) * 2};
  const cuuint32_t box[2] = {64, kTile}, ones[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

fs_status check_attn(int64_t S, int64_t T, int32_t Hq, int32_t Hkv, int32_t Dh, float scale, const int64_t* offsets,
                     const int32_t* cand, const float* lse, const int32_t* err) {
  if (S < 0 || S > INT32_MAX || T < 0 || T > INT32_MAX || Hkv < 1 || Hq < Hkv || Hq > 1024 || Hq % Hkv != 0 || !err)
    return FS_ERR_INVALID_ARG;
  if ((Dh != 64 && Dh != 128) || !(scale > 0.f) || !(scale <= 3.4e38f)) return FS_ERR_INVALID_ARG;
  if (S > 0 && !offsets) return FS_ERR_INVALID_ARG;
  if (S > 0 && T > 0 && !lse) return FS_ERR_INVALID_ARG;
  if (!aligned(offsets, 8) || !aligned(cand, 4) || !aligned(lse, 4)) return FS_ERR_ALIGNMENT;
  return FS_OK;
}

// Rows of q, k, v and their gradients: bf16, `heads * Dh` elements each, rows
// `stride` elements apart, 16-byte aligned.
fs_status check_rows(const void* p, int64_t stride, int32_t heads, int32_t Dh) {
  if (!p || stride < int64_t(heads) * Dh || stride >= (int64_t(1) << 36)) return FS_ERR_INVALID_ARG;
  return aligned(p, 16) && stride % 8 == 0 ? FS_OK : FS_ERR_ALIGNMENT;
}

int64_t most_tiles(int64_t T, int64_t S) { return T / kTile + (S < T ? S : T); }

struct AttnWs {
  int32_t* ntiles = nullptr;
  Tile *by_query = nullptr, *by_key = nullptr;
  float* delta = nullptr;
};

template <class Ws>
void take_attn(int64_t T, int64_t S, int32_t Hq, Ws& ws, AttnWs& W) {
  W.ntiles = ws.template take<int32_t>(1);
  W.by_query = ws.template take<Tile>(size_t(most_tiles(T, S)));
  W.by_key = ws.template take<Tile>(size_t(most_tiles(T, S)));
  W.delta = ws.template take<float>(size_t(Hq) * size_t(T));
}

// Allows a kernel its shared memory, once per device (`done` holds a bit for each).  A kernel
// that moves registers between its warps (regs > 0) must have been built with that many a
// thread: with fewer, the warps that ask for more would wait for ever.
template <class K>
bool prepare_kernel(K kern, int bytes, int regs, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return true;
  cudaFuncAttributes f;
  if (cudaFuncGetAttributes(&f, kern) != cudaSuccess || f.numRegs < regs) return false;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.fetch_or(bit);
  return true;
}

std::atomic<uint64_t> g_fwd_ready[2], g_bwd_ready[2][2];

}  // namespace
}  // namespace fs

using namespace fs;

extern "C" size_t fs_jagged_attn_workspace_size(int64_t T, int64_t S, int32_t heads, int32_t kv_heads,
                                                int32_t head_dim) {
  if (T < 0 || S < 0 || heads < 1 || kv_heads < 1 || (head_dim != 64 && head_dim != 128)) return 0;
  WsCounter c;
  AttnWs W;
  take_attn(T, S, heads, c, W);
  return c.used;
}

extern "C" fs_status fs_jagged_attn(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                    int64_t v_stride, const int64_t* offsets, int64_t S, int64_t T, int32_t heads,
                                    int32_t kv_heads, int32_t head_dim, const int32_t* cand_len, int32_t causal,
                                    float scale, void* out, float* lse, int32_t* err, void* ws, size_t ws_bytes,
                                    fs_stream_t stream) {
  FS_NVTX_RANGE();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  fs_status s = check_attn(S, T, heads, kv_heads, head_dim, scale, offsets, cand_len, lse, err);
  if (s != FS_OK) return s;
  if (S == 0 || T == 0) return FS_OK;
  if ((s = check_rows(q, q_stride, heads, head_dim)) != FS_OK || (s = check_rows(k, k_stride, kv_heads, head_dim)) != FS_OK ||
      (s = check_rows(v, v_stride, kv_heads, head_dim)) != FS_OK ||
      (s = check_rows(out, int64_t(heads) * head_dim, heads, head_dim)) != FS_OK)
    return s;
  if (!ws || ws_bytes < fs_jagged_attn_workspace_size(T, S, heads, kv_heads, head_dim)) return FS_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return FS_ERR_ALIGNMENT;
  if (most_tiles(T, S) * heads > INT32_MAX) return FS_ERR_INVALID_ARG;
  WsCursor cur(ws, ws_bytes);
  AttnWs W;
  take_attn(T, S, heads, cur, W);
  CUtensorMap mq, mk, mv;
  if (!encode(&mq, q, T, int64_t(heads) * head_dim, q_stride) || !encode(&mk, k, T, int64_t(kv_heads) * head_dim, k_stride) ||
      !encode(&mv, v, T, int64_t(kv_heads) * head_dim, v_stride))
    return FS_ERR_CUDA;
  AttnArgs a{};
  a.ntiles = W.ntiles, a.tiles = W.by_query;
  a.heads = heads, a.kv_heads = kv_heads, a.T = T, a.causal = causal != 0, a.scale = scale;
  a.o = static_cast<__nv_bfloat16*>(out), a.lse = lse, a.err = err;
  a.wait_ns = uint64_t(spin_limit()) * 256u;
  const bool by_head = heads / kv_heads % 2 == 0;  // two heads of one tile share a block, else two tiles of one head
  const int parts = by_head ? heads / 2 : heads;
  attn_plan_kernel<<<1, kPlanThreads, 0, st>>>(offsets, S, T, cand_len, a.causal, by_head ? 1 : 2, W.ntiles, W.by_query,
                                               nullptr, err);
  const int64_t units = most_tiles(T, S) * parts;
  const unsigned grid = unsigned(units < sm_count() ? units : sm_count());
  if (head_dim == 64) {
    if (!prepare_kernel(attn_fwd_kernel<64>, fwd_smem<64>(), kFwdRegs, g_fwd_ready[0])) return FS_ERR_CUDA;
    attn_fwd_kernel<64><<<grid, kFwdThreads, fwd_smem<64>(), st>>>(mq, mk, mv, a, parts);
  } else {
    if (!prepare_kernel(attn_fwd_kernel<128>, fwd_smem<128>(), kFwdRegs, g_fwd_ready[1])) return FS_ERR_CUDA;
    attn_fwd_kernel<128><<<grid, kFwdThreads, fwd_smem<128>(), st>>>(mq, mk, mv, a, parts);
  }
  count_launch(2);
  return launch_status();
}

extern "C" fs_status fs_jagged_attn_backward(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                             const void* v, int64_t v_stride, const void* out, const float* lse,
                                             const void* dout, const int64_t* offsets, int64_t S, int64_t T,
                                             int32_t heads, int32_t kv_heads, int32_t head_dim, const int32_t* cand_len,
                                             int32_t causal, float scale, void* dq, int64_t dq_stride, void* dk,
                                             int64_t dk_stride, void* dv, int64_t dv_stride, int32_t* err, void* ws,
                                             size_t ws_bytes, fs_stream_t stream) {
  FS_NVTX_RANGE();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  fs_status s = check_attn(S, T, heads, kv_heads, head_dim, scale, offsets, cand_len, lse, err);
  if (s != FS_OK) return s;
  if (S == 0 || T == 0) return FS_OK;
  const int64_t ow = int64_t(heads) * head_dim, kw = int64_t(kv_heads) * head_dim;
  if ((s = check_rows(q, q_stride, heads, head_dim)) != FS_OK || (s = check_rows(k, k_stride, kv_heads, head_dim)) != FS_OK ||
      (s = check_rows(v, v_stride, kv_heads, head_dim)) != FS_OK || (s = check_rows(out, ow, heads, head_dim)) != FS_OK ||
      (s = check_rows(dout, ow, heads, head_dim)) != FS_OK || (s = check_rows(dq, dq_stride, heads, head_dim)) != FS_OK ||
      (s = check_rows(dk, dk_stride, kv_heads, head_dim)) != FS_OK ||
      (s = check_rows(dv, dv_stride, kv_heads, head_dim)) != FS_OK)
    return s;
  if (!ws || ws_bytes < fs_jagged_attn_workspace_size(T, S, heads, kv_heads, head_dim)) return FS_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return FS_ERR_ALIGNMENT;
  if (most_tiles(T, S) * heads > INT32_MAX) return FS_ERR_INVALID_ARG;
  WsCursor cur(ws, ws_bytes);
  AttnWs W;
  take_attn(T, S, heads, cur, W);
  CUtensorMap mq, mk, mv, mdo;
  if (!encode(&mq, q, T, ow, q_stride) || !encode(&mk, k, T, kw, k_stride) || !encode(&mv, v, T, kw, v_stride) ||
      !encode(&mdo, dout, T, ow, ow))
    return FS_ERR_CUDA;
  AttnArgs a{};
  a.ntiles = W.ntiles;
  a.heads = heads, a.kv_heads = kv_heads, a.T = T, a.causal = causal != 0, a.scale = scale;
  a.out = static_cast<const __nv_bfloat16*>(out), a.dout = static_cast<const __nv_bfloat16*>(dout);
  a.lse = const_cast<float*>(lse), a.delta = W.delta, a.err = err;
  a.dq = static_cast<__nv_bfloat16*>(dq), a.dk = static_cast<__nv_bfloat16*>(dk), a.dv = static_cast<__nv_bfloat16*>(dv);
  a.dq_stride = dq_stride, a.dk_stride = dk_stride, a.dv_stride = dv_stride;
  a.wait_ns = uint64_t(spin_limit()) * 256u;
  attn_plan_kernel<<<1, kPlanThreads, 0, st>>>(offsets, S, T, cand_len, a.causal, 1, W.ntiles, W.by_query, W.by_key, err);
  const unsigned gq = unsigned(most_tiles(T, S) * heads), gk = unsigned(most_tiles(T, S) * kv_heads);
  AttnArgs b = a;
  a.tiles = W.by_query, b.tiles = W.by_key;
  if (head_dim == 64) {
    if (!prepare_kernel(attn_dq_kernel<64>, bwd_smem<64>(), 0, g_bwd_ready[0][0])) return FS_ERR_CUDA;
    if (!prepare_kernel(attn_dkv_kernel<64>, bwd_smem<64>(), 0, g_bwd_ready[0][1])) return FS_ERR_CUDA;
    attn_dq_kernel<64><<<gq, kBwdThreads, bwd_smem<64>(), st>>>(mq, mk, mv, mdo, a);
    attn_dkv_kernel<64><<<gk, kBwdThreads, bwd_smem<64>(), st>>>(mq, mk, mv, mdo, b);
  } else {
    if (!prepare_kernel(attn_dq_kernel<128>, bwd_smem<128>(), 0, g_bwd_ready[1][0])) return FS_ERR_CUDA;
    if (!prepare_kernel(attn_dkv_kernel<128>, bwd_smem<128>(), 0, g_bwd_ready[1][1])) return FS_ERR_CUDA;
    attn_dq_kernel<128><<<gq, kBwdThreads, bwd_smem<128>(), st>>>(mq, mk, mv, mdo, a);
    attn_dkv_kernel<128><<<gk, kBwdThreads, bwd_smem<128>(), st>>>(mq, mk, mv, mdo, b);
  }
  count_launch(3);
  return launch_status();
}
