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
// first; one block per SM then takes units (a tile and a head) from the list as
// it gets free, and walks the tiles that the unit's rows (or, for dk and dv,
// its keys) meet: tiles nothing of which is visible are never loaded.
//
// Roles inside a block: one warp takes units and loads tiles by TMA through a
// ring of shared-memory slots, running ahead into the next unit; one thread
// issues the products; two warpgroups do the elementwise part
// with the scores in tensor memory.  They meet at mbarriers only.  Every wait has a
// limit, after which the error word is set, copies and products in flight are
// waited for and the block ends.
//
// The backward pass is two kernels: one block per query tile for dq, one per
// key tile for dk and dv, each summing in its own accumulators, so every sum
// has a fixed order and nothing is added atomically; it recomputes x and do.v
// twice (7 products where a pass with atomic sums of dq needs 5).
//
// Scores, softmax statistics, sums and accumulators are fp32.  p and ds are rounded to bf16, since the tensor cores
// take both operands in the type of q, k and v: each error is 2^-9 of its own term and they are as many as the
// terms, so a result is off by about as much again as by its own rounding to bf16 (relative norms against 64 bits:
// out 2.0e-3, gradients 2.4e-3, where rounding alone leaves 1.7e-3).  A backward pass over a small batch, in which
// each unit has an SM of its own, takes p and ds as pairs of bf16 (FINE: 2^-17, a second product for the rests, in the
// half of the columns that the rounded values leave free): with few terms the errors may come together
// by chance (1 batch in 250 had half as much again), and the products are not what such a batch waits for.  8 samples of up
// to 511 positions: gradients 2.4e-3 -> 1.7e-3, 19.1 -> 21.7 us; 22,000 positions of long histories would pay 323 -> 423 us.
//
// Bound on long samples by the tensor cores and the hand-overs between products
// and elementwise warps, on short ones by the chain of latencies inside one unit.
// 22,000 positions of causal samples up to 4096, 8 query and 2 key/value heads of 128:
// forward 93 us (1070 TFLOP/s over visible pairs, tensor pipe 55% active), backward
// 291 us (850 TFLOP/s over 5 products, 55 and 61% active over the 7 that run).  350,000 positions in 256 such
// samples: 1.7 ms (1210 TFLOP/s) and 5.7 ms (900); with heads of 64 1.1 ms (920) and 3.7 ms (690).
#include <cuda_bf16.h>

#include <atomic>
#include <mutex>
#include <type_traits>
#include <utility>

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
  int32_t part;   // which half of a key tile's work (only where split >= 0)
  int32_t split;  // number of the halved key tile, -1: in one piece
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

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32, kBuckets = 1024;

struct Plan {
  int32_t ntiles[2];  // entries of the two lists: queries, keys
  int32_t next[2];    // units handed out beyond the first of each block
};

// At most this many (key tile, key/value head) units are cut in half: each takes over half of
// an SM's share of all the work.
constexpr int64_t most_split(int64_t sms) { return 2 * sms; }

// Lists the tiles of all samples twice, by descending number of key tiles (for
// queries; an entry stands for `span` neighbouring tiles, and its t counts such
// groups) and of query tiles (for keys; only where by_key is given, span 1): a
// counting sort over the tile counts by one block.  The order among equals
// does not matter to any result.  A warp takes up to 32 samples at a time and
// spreads their tiles over its lanes.
// A key tile whose units (one per key/value head, over `group` query heads) each take more than half of
// an SM's share of the whole work is listed as two halves: in a batch with a few long samples
// one such unit would otherwise set the time.
__global__ void __launch_bounds__(kPlanThreads, 1) attn_plan_kernel(const int64_t* __restrict__ offsets, int64_t S, int64_t T,
                                                                 const int32_t* __restrict__ cand, bool causal,
                                                                 int span, int kv_heads, int group, int sms, Plan* plan,
                                                                 Tile* by_query, Tile* by_key, int32_t* flags,
                                                                 int32_t* err) {
  __shared__ int32_t hist[2][kBuckets];
  __shared__ int32_t scan[32];
  __shared__ unsigned long long work, listed;
  __shared__ int32_t nsplit;
  asm volatile("griddepcontrol.launch_dependents;");
  for (int i = threadIdx.x; i < 2 * kBuckets; i += kPlanThreads) (&hist[0][0])[i] = 0;
  if (threadIdx.x < 2) plan->next[threadIdx.x] = 0;
  if (threadIdx.x == 0) work = listed = 0, nsplit = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = span * kTile;
  const int64_t most = T / kTile + (S < T ? S : T);  // entries the lists hold
  auto bucket = [](int cost) { return kBuckets - min(cost, kBuckets); };  // most work first
  // Query tiles that all key tiles of a sample meet.
  auto tiles_met = [&](int64_t L, int64_t uih) {
    const int64_t all = (L + kTile - 1) / kTile, seen = (uih + kTile - 1) / kTile;
    return (causal ? seen * all - seen * (seen - 1) / 2 : seen * all) + (all - seen);
  };
  if (by_key) {
    unsigned long long mine = 0;
    for (int64_t s = threadIdx.x; s < S; s += kPlanThreads) {
      const int64_t b = offsets[s], e = offsets[s + 1];
      if (b < 0 || e < b || e > T) continue;
      int64_t c = cand ? cand[s] : 0;
      c = c < 0 ? 0 : (c > e - b ? e - b : c);
      mine += (unsigned long long)(tiles_met(e - b, e - b - c));
    }
    if (mine) atomicAdd(&work, mine);
    for (int64_t i = threadIdx.x; i < most_split(sms) * 8; i += kPlanThreads) flags[i] = 0;
    __syncthreads();
  }
  const int64_t share = (S + kPlanWarps - 1) / kPlanWarps;
  const int take = share < 32 ? int(share) : 32;  // samples a warp takes at a time
  // half of an SM's share, in query tiles of one unit's `group` heads
  const int64_t half = by_key ? int64_t(work) * kv_heads / (2 * sms) : 0;
  auto cut = [&](int nq) { return by_key && nq * group > 1 && nq > half; };
  // f of every entry, as long as this warp's share fits the lists (it does where the offsets are in
  // order); returns how many there are, in 64 bits: of samples that overlap there can be S * T / kTile.
  auto each = [&](bool report, auto f) {
    int64_t entries = 0;
    for (int64_t s0 = int64_t(warp) * take; s0 < S; s0 += int64_t(kPlanWarps) * take) {
      int32_t begin = 0, L = 0, c = 0;
      if (lane < take && s0 + lane < S) {
        const int64_t b = offsets[s0 + lane], e = offsets[s0 + lane + 1];
        if (b < 0 || e < b || e > T) {
          if (report) set_err(err, FS_ERR_BAD_OFFSETS);
        } else {
          begin = int32_t(b);
          L = int32_t(e - b);
          c = cand ? cand[s0 + lane] : 0;
          if (c < 0 || c > L) {
            if (report) set_err(err, FS_ERR_INVALID_ARG);
            c = c < 0 ? 0 : L;
          }
        }
      }
      const int32_t mine = (L + rows - 1) / rows;
      int32_t upto = mine;  // inclusive over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const int32_t all = __shfl_sync(0xffffffffu, upto, 31);
      entries += all;
      if (entries > most) continue;
      for (int32_t i0 = 0; i0 < all; i0 += 32) {
        const int32_t i = i0 + lane;
        int who = 0;  // lanes whose tiles end at or before i
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (__shfl_sync(0xffffffffu, upto, (who + o - 1) & 31) <= i) who += o;
        who &= 31;
        Tile x{__shfl_sync(0xffffffffu, begin, who), __shfl_sync(0xffffffffu, L, who), 0, 0, 0, -1};
        x.uih = x.L - __shfl_sync(0xffffffffu, c, who);
        x.t = i - (__shfl_sync(0xffffffffu, upto, who) - __shfl_sync(0xffffffffu, mine, who));
        if (i < all) {
          int own, first;
          Tile last = x;  // the entry's last tile has the most key tiles
          last.t = min(x.t * span + span - 1, (x.L - 1) / kTile);
          const int nk = key_tiles(last, causal, own) + own;
          f(x, nk, query_tiles(x, causal, first));
        }
        __syncwarp();
      }
    }
    return entries;
  };
  const int64_t mine = each(true, [&](const Tile&, int nk, int nq) {
    atomicAdd(&hist[0][bucket(nk)], 1);
    if (by_key) atomicAdd(&hist[1][bucket(cut(nq) ? (nq + 1) / 2 : nq)], cut(nq) ? 2 : 1);
  });
  if (lane == 0) atomicAdd(&listed, (unsigned long long)(mine));
  __syncthreads();
  for (int w = 0; w < (by_key ? 2 : 1); ++w) {
    int32_t n;
    const int32_t mine = hist[w][threadIdx.x];
    const int32_t at = block_exclusive_scan<int32_t>(mine, scan, &n);
    hist[w][threadIdx.x] = at;
    if (threadIdx.x == 0) plan->ntiles[w] = n;
  }
  __syncthreads();
  // Offsets that are not in order can describe more tiles than the lists hold:
  // then nothing is listed (the error word says so).
  if (listed > (unsigned long long)(most)) {
    if (threadIdx.x == 0) {
      set_err(err, FS_ERR_BAD_OFFSETS);
      plan->ntiles[0] = plan->ntiles[1] = 0;
    }
    return;
  }
  each(false, [&](Tile x, int nk, int nq) {
    by_query[atomicAdd(&hist[0][bucket(nk)], 1)] = x;
    if (by_key) {
      if (cut(nq)) {
        const int32_t at = atomicAdd(&hist[1][bucket((nq + 1) / 2)], 2);
        x.split = atomicAdd(&nsplit, 1);
        by_key[at] = x;
        x.part = 1;
        by_key[at + 1] = x;
      } else {
        by_key[atomicAdd(&hist[1][bucket(nq)], 1)] = x;
      }
    }
  });
}

// ------------------------------------------------------------- shared pieces

struct AttnArgs {
  Plan* plan;               // null: no lists, the loading warp of each block finds its one unit itself
  const Tile* tiles;
  const int64_t* offsets;   // (for that)
  const int32_t* cand;
  int32_t S;
  int32_t heads, kv_heads;
  int64_t T;
  bool causal;
  float scale;
  __nv_bfloat16* o;           // forward: out
  float* lse;
  float* delta;               // [heads, T]: written by the dq kernel, read by the dk / dv kernel
  float* partial;             // sums of the halves of key tiles
  int32_t* flags;             // and who of the two came first, for each warp of a unit
  __nv_bfloat16 *dq, *dk, *dv;
  int64_t dq_stride, dk_stride, dv_stride;
  int32_t* err;
  uint64_t wait_ns;
  int64_t skip_block;  // test hook: the first tile of this block's ring is never loaded (-1: none)
};

// Wait of a whole warp for a barrier's phase, with a limit.  The hand-overs
// between the warps of a block come every few hundred cycles, so it polls
// without asking to sleep and looks at the clock only now and then.  Every lane polls
// and a vote decides: beside running products that costs nothing, where one lane's poll, its
// branch and the broadcast of the answer took 16 to 160 cycles (measured).
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

// Tile of 128 rows of DH columns from position y of head h, as DH / 64 boxes (one thread).
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

// The loading warp's side of a ring of NS tile slots in shared memory, filled in
// order.  full[s]: the tile has arrived; free[s]: its last reader is done.  A
// tile with rows past its sample's end (a tail) arrives on a barrier of its own
// (tail[4]), is mended here, and only then reported full.  Whenever this warp has to wait for something
// it mends what has arrived in the meantime, so that neither holds up the other.
template <int DH, int NS>
struct Feeder {
  static constexpr int TB = DH / 64 * kBox;
  unsigned char* tiles;
  uint32_t full, free, tail;
  const AttnArgs& a;
  uint32_t slot = 0;              // tiles asked for
  uint32_t tails = 0, mended = 0; // at most four outstanding
  uint64_t notes = 0;             // of those, the oldest in the low bits: slot | first foreign row << 8, 16 bits each

  __device__ __forceinline__ Feeder(unsigned char* tiles, uint32_t full, uint32_t free, uint32_t tail, const AttnArgs& a)
      : tiles(tiles), full(full), free(free), tail(tail), a(a) {}

  __device__ __forceinline__ void mend() {  // the oldest tail, which has arrived
    const int s = int(notes & 255u), from = int((notes >> 8) & 255u);
    zero_rows<DH>(tiles + s * TB, from);
    if ((threadIdx.x & 31) == 0) tc::arrive(full + 8 * s);
    notes >>= 16;
    ++mended;
  }
  __device__ __forceinline__ bool mend_all() {
    while (mended != tails) {
      if (!wait(tail + 8 * (mended & 3u), mended >> 2, a)) return false;
      mend();
    }
    return true;
  }
  // Waits for a barrier, mending meanwhile.
  __device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t phase) {
    polls = 0;
    while (mended != tails) {
      if (__all_sync(0xffffffffu, tc::test(bar, phase & 1u))) return true;
      if (__all_sync(0xffffffffu, tc::test(tail + 8 * (mended & 3u), (mended >> 2) & 1u))) mend();
      else if (late()) return false;
    }
    return wait(bar, phase, a);
  }
  uint64_t since = 0;
  uint32_t polls = 0;
  __device__ __forceinline__ bool late() {  // the limit of wait_for's first loop
    if ((++polls & 1023u) != 0) return false;
    const uint64_t now = bulk::global_ns();
    if (polls == 1024u) since = now;
    if (!__any_sync(0xffffffffu, now - since > a.wait_ns)) return false;
    if ((threadIdx.x & 31) == 0) set_err(a.err, FS_ERR_TIMEOUT);
    return true;
  }
  // The next tile: position y of head h of `map`, the first `valid` rows (of at most 128) the sample's.
  // mend_tail: whether the other rows must be zero.
  __device__ __forceinline__ bool put(const CUtensorMap* map, int h, int y, int valid, bool mend_tail) {
    const int lane = threadIdx.x & 31;
    const int s = int(slot % NS);
    if (slot >= NS && !wait_for(free + 8 * s, slot / NS - 1)) return false;
    if (slot == 0 && a.skip_block == int64_t(blockIdx.x)) {
      ++slot;
      return true;
    }
    uint32_t bar = full + 8 * s;
    if (mend_tail && valid < kTile) {
      if (tails - mended == 4) {
        if (!wait(tail + 8 * (mended & 3u), mended >> 2, a)) return false;
        mend();
      }
      bar = tail + 8 * (tails & 3u);
      notes |= uint64_t(uint32_t(s) | uint32_t(valid) << 8) << (16 * (tails - mended));
      ++tails;
    }
    if (lane == 0) {
      bulk::arrive_expect_tx(bar, TB);
      load_tile<DH>(bulk::smem_addr(tiles) + s * TB, map, h, y, bar);
    }
    ++slot;
    return true;
  }
  // After a wait that gave up: every copy still in flight lands first.
  __device__ __forceinline__ void drain() {
    uint32_t tail_slots = 0;
    for (uint32_t m = mended; m != tails; ++m, notes >>= 16) {
      bulk::warp_wait(tail + 8 * (m & 3u), (m >> 2) & 1u, a.wait_ns);
      tail_slots |= 1u << (notes & 31u);
    }
    for (uint32_t s = slot > NS ? slot - NS : 0; s < slot; ++s)
      if (!((tail_slots >> (s % NS)) & 1u)) bulk::warp_wait(full + 8 * (s % NS), (s / NS) & 1u, a.wait_ns);
  }
};

// Tile `index` (of groups of `span`) of a batch of at most 32 samples, found by one warp
// from the offsets; false where there are not so many.  Does the checks of the planning kernel.
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int span, int index, Tile& x) {
  const int lane = threadIdx.x & 31;
  int32_t begin = 0, L = 0, c = 0;
  if (lane < a.S) {
    const int64_t b = a.offsets[lane], e = a.offsets[lane + 1];
    if (b < 0 || e < b || e > a.T) {
      set_err(a.err, FS_ERR_BAD_OFFSETS);
    } else {
      begin = int32_t(b), L = int32_t(e - b);
      c = a.cand ? a.cand[lane] : 0;
      if (c < 0 || c > L) {
        set_err(a.err, FS_ERR_INVALID_ARG);
        c = c < 0 ? 0 : L;
      }
    }
  }
  const int32_t mine = (L + span * kTile - 1) / (span * kTile);
  int32_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  const int who = __popc(__ballot_sync(0xffffffffu, upto <= index));
  if (who == 32) return false;
  x.begin = __shfl_sync(0xffffffffu, begin, who);
  x.L = __shfl_sync(0xffffffffu, L, who);
  x.uih = x.L - __shfl_sync(0xffffffffu, c, who);
  x.t = index - (__shfl_sync(0xffffffffu, upto, who) - __shfl_sync(0xffffffffu, mine, who));
  x.part = 0, x.split = -1;
  return true;
}

// Units of a block, `parts` for each tile: its own index first, then whatever
// comes next in the list (without lists every block has one unit).  The loading warp takes them and
// leaves them for the others under the barrier that announces the unit's first
// tiles (given[4]: no reader is two units behind).
struct Taker {
  const AttnArgs& a;
  int which, parts, span;  // list; units per tile; tiles per entry
  int64_t units;
  int round = 0;
  Tile tile;
  int part = 0;
  __device__ __forceinline__ Taker(const AttnArgs& a, int which, int parts, int span)
      : a(a), which(which), parts(parts), span(span), units(a.plan ? int64_t(a.plan->ntiles[which]) * parts : 0) {}
  __device__ __forceinline__ bool next() {
    if (!a.plan) {
      part = int(blockIdx.x % unsigned(parts));
      return round++ == 0 && find_tile(a, span, int(blockIdx.x / unsigned(parts)), tile);
    }
    int64_t u = blockIdx.x;
    if (round++ > 0) {
      int32_t v = 0;
      if ((threadIdx.x & 31) == 0) v = atomicAdd(&a.plan->next[which], 1);
      u = int64_t(gridDim.x) + __shfl_sync(0xffffffffu, v, 0);
    }
    if (u >= units) return false;
    tile = a.tiles[u / parts];
    part = int(u % parts);
    return true;
  }
};

// The products are issued by one warp in batches: what one batch waits for and
// the descriptors of its operands are found before, so that between two products
// of a batch there is nothing but the products (a few dozen instructions of one warp
// beside busy ones take longer than the queue of products lasts).

// D[128 x 128] = A B^T over DH columns, both tiles K-major: descriptors of tc::desc_k.
template <int DH>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t id = tc::idesc(kTile, kTile, false);
  tc::mma_ss<true>(d, tc::at(a, 0), tc::at(b, 0), id, false);
#pragma unroll
  for (int k = 1; k < DH / 16; ++k) {
    const uint32_t off = (k / 4) * kBox + (k % 4) * 32;
    tc::mma_ss<false>(d, tc::at(a, off), tc::at(b, off), id, true);
  }
}

// D[128 x DH] (+)= A B, A [128 x 128] bf16 in tensor memory, its first 64 columns at a0, the
// others at a1, B a tile of 128 rows: a descriptor of tc::desc_mn.
template <int DH>
__device__ __forceinline__ void mma_cols(uint32_t d, uint32_t a0, uint32_t a1, uint32_t b, bool acc) {
  constexpr uint32_t id = tc::idesc(kTile, DH, true);
  tc::mma_ts<true>(d, a0, tc::at(b, 0), id, acc);
#pragma unroll
  for (int k = 1; k < kTile / 16; ++k)
    tc::mma_ts<false>(d, (k < 4 ? a0 + 8 * k : a1 + 8 * (k - 4)), tc::at(b, k * 2048), id, true);
}

// The same from shared-memory addresses.
template <int DH>
__device__ __forceinline__ void mma_rows_at(uint32_t d, uint32_t a, uint32_t b) {
  mma_rows<DH>(d, tc::desc_k(a), tc::desc_k(tc::uni(b)));
}
template <int DH>
__device__ __forceinline__ void mma_cols_at(uint32_t d, uint32_t a0, uint32_t a1, uint32_t b, bool acc) {
  mma_cols<DH>(d, a0, a1, tc::desc_mn(tc::uni(b), kBox), acc);
}

// 32 fp32 columns of each lane's row, scaled, as bf16: `to` is column 0 of the
// warp's first row, rows are `stride` elements apart, the first `live` of the 32
// exist.  Four neighbouring lanes exchange 16-byte pieces (a 4 x 4 transpose by shuffles), so that a
// store writes 64 bytes of 8 rows instead of 16 bytes of 32 (an epilogue of 128 rows of
// 256 bytes took 4000 to 6000 cycles that way).
__device__ __forceinline__ void store32(__nv_bfloat16* to, int64_t stride, int live, const float* x, float f) {
  const int lane = threadIdx.x & 31, s = lane & 3, q = lane >> 2;
  uint32_t v[4][4];
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int w = 0; w < 4; ++w) v[c][w] = tc::pack2(x[8 * c + 2 * w] * f, x[8 * c + 2 * w + 1] * f);
#pragma unroll
  for (int c = 0; c < 4; c += 2)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, (s & 1) ? v[c][w] : v[c + 1][w], 1);
      if (s & 1) v[c][w] = got;
      else v[c + 1][w] = got;
    }
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, (s & 2) ? v[c][w] : v[c + 2][w], 2);
      if (s & 2) v[c][w] = got;
      else v[c + 2][w] = got;
    }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (4 * q + j < live)
      *reinterpret_cast<uint4*>(to + int64_t(4 * q + j) * stride + 8 * s) = make_uint4(v[j][0], v[j][1], v[j][2], v[j][3]);
}

// What two fp32 values leave when they are rounded to the bf16 pair `w`, itself as a bf16 pair: together within
// 2^-17 of the values.
__device__ __forceinline__ uint32_t rest2(uint32_t w, float lo, float hi) {
  return tc::pack2(lo - __uint_as_float(w << 16), hi - __uint_as_float(w & 0xFFFF0000u));
}

template <int DH>
constexpr int tile_bytes() { return DH / 64 * kBox; }

// Place in a ring of NS slots: item i is in slot i % NS, its phase i / NS.
template <int NS>
struct Place {
  int s;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Place(int first) : s(first) {}
  __device__ __forceinline__ void skip(int k) {  // k <= NS items further on
    s += k;
    if (s >= NS) s -= NS, ++phase;
  }
  __device__ __forceinline__ void back(int k) {
    s -= k;
    if (s < 0) s += NS, --phase;
  }
};

__device__ __forceinline__ void wait_for_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;"); }

// The block's tensor memory, and everyone's barriers and addresses in place; called by all
// threads, `taker` one warp.  Only after wait_for_launch(): the launch before may still have to take tensor memory on
// this SM, and a block that held all of it while waiting for that launch's end would never see it.  For the same
// reason a kernel lets the next launch begin only after this.
__device__ __forceinline__ void take_tmem(uint32_t* at, bool taker) {
  if (taker) {
    __syncwarp();
    tc::alloc(at, 512);
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
}

// ------------------------------------------------------------- forward

// A unit is two query tiles that read the same keys and values, so each loaded
// tile serves two products: the same positions of two query heads that share a
// key/value head, or, where the number of sharing heads is odd, neighbouring
// tiles of one head.  A warpgroup per query tile, one row a thread, does the
// softmax; one thread issues the products of the two tiles in turn, so that one tile's products run
// under the other's softmax.  Tensor memory: x of each tile in 128 columns, p (bf16) over it, o
// beside them.
//
// A softmax thread holds a row of 128 scores: the third warpgroup (products and
// loads) gives registers to the other two.  384 threads are launched with
// kFwdRegs each; 2 * 128 * 208 + 128 * 88 is that total.
constexpr int kFwdThreads = 384, kFwdRegs = 168;
template <int DH> constexpr int fwd_slots() { return DH == 64 ? 10 : 5; }
template <int DH> constexpr int fwd_smem() { return tile_bytes<DH>() * (2 + fwd_slots<DH>()); }

struct FwdUnit {
  Tile x;
  int head0, head1, row0, row1;  // query head and tile index of each query tile
  int nk0, nk1, own0, own1;      // key tiles of the history, and whether its own tile follows
  int kv_head, common, n;        // n < 0: no more units
  int by_head, both;

  FwdUnit() = default;
  __device__ __forceinline__ FwdUnit(const Tile& tile, int part, const AttnArgs& a) : x(tile) {
    const int group = a.heads / a.kv_heads;
    by_head = group % 2 == 0;
    head0 = by_head ? 2 * part : part, head1 = by_head ? 2 * part + 1 : part;
    row0 = by_head ? x.t : 2 * x.t, row1 = by_head ? x.t : 2 * x.t + 1;
    kv_head = head0 / group;
    both = row1 * kTile < x.L;
    Tile y = x;
    y.t = row0;
    nk0 = key_tiles(y, a.causal, own0);
    y.t = row1;
    nk1 = key_tiles(y, a.causal, own1);
    if (!both) nk1 = own1 = 0;
    common = max(nk0, nk1);
    n = common + own0 + (by_head ? 0 : own1);
  }
  // The unit's j-th key tile, and whether query tile i meets it.
  __device__ __forceinline__ int key_tile(int j) const {
    return j < common ? j : ((j == common && own0) || by_head ? row0 : row1);
  }
  __device__ __forceinline__ bool meets(int i, int j) const {
    if (by_head) return true;
    return i ? j < nk1 || (own1 && j == common + own0) : j < nk0 || (own0 && j == common);
  }
  // A copy whose fields the compiler knows to be the same in every lane: branches on them are the warp's.
  __device__ __forceinline__ FwdUnit uniform() const {
    FwdUnit u = *this;
    auto same = [](int& v) { v = int(tc::uni(uint32_t(v))); };
    same(u.x.begin), same(u.x.L), same(u.x.uih);
    same(u.head0), same(u.head1), same(u.row0), same(u.row1), same(u.nk0), same(u.nk1), same(u.own0), same(u.own1);
    same(u.kv_head), same(u.common), same(u.n), same(u.by_head), same(u.both);
    return u;
  }
};

template <int DH>
__global__ void __launch_bounds__(kFwdThreads, 1) attn_fwd_kernel(const __grid_constant__ CUtensorMap mq,
                                                                  const __grid_constant__ CUtensorMap mk,
                                                                  const __grid_constant__ CUtensorMap mv, AttnArgs a,
                                                                  int parts) {
  constexpr int TB = tile_bytes<DH>(), NS = fwd_slots<DH>();
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[13 + 2 * NS];
  __shared__ uint32_t tmem_at;
  __shared__ FwdUnit given[4];  // units handed over by the loading warp (no reader is two units behind)
  const uint32_t q_at = bulk::smem_addr(smem), kv_at = q_at + 2 * TB;
  const uint32_t bar = bulk::smem_addr(bars);
  const uint32_t q_full = bar, q_free = bar + 8, s_full = bar + 16, p_ready = bar + 32, o_full = bar + 48, tail = bar + 64,
                 drain = bar + 96, full = bar + 104, free = full + 8 * NS;
  const int warp = int(tc::uni(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (warp == 8) {
    if (lane == 0) {
      for (int i = 0; i < 13 + 2 * NS; ++i)
        bulk::mbar_init(bar + 8 * i, i == 1 ? 9 : (i == 4 || i == 5 ? 4 : 1));
      bulk::fence_init();
    }
  } else if (warp == 9 && lane == 0) {
    tc::prefetch_map(&mq), tc::prefetch_map(&mk), tc::prefetch_map(&mv);
  }
  wait_for_launch();
  take_tmem(&tmem_at, warp == 8);
  const uint32_t s_at = tc::uni(tmem_at), o_at = s_at + 256;  // of query tile 0; tile 1's follow

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 9) {
      Feeder<DH, NS> feed(smem + 2 * TB, full, free, tail, a);
      Taker take(a, 0, parts, a.heads / a.kv_heads % 2 == 0 ? 1 : 2);
      bool ok = true;
      int k = 0;
      bool more = take.next();
      for (;; ++k) {
        FwdUnit f;
        f.n = -1;
        if (more) f = FwdUnit(take.tile, take.part, a).uniform();
        if (lane == 0) given[k & 3] = f;
        if (f.n < 0) break;
        // the first key and value tile need only a slot, the query tiles the end of the last unit's scores
        auto put = [&](int j) {
          const int at = f.key_tile(j) * kTile;
          return feed.put(&mk, f.kv_head, f.x.begin + at, f.x.L - at, false) &&
                 feed.put(&mv, f.kv_head, f.x.begin + at, f.x.L - at, true);
        };
        if (!(ok = put(0))) break;
        if (k > 0 && !(ok = feed.wait_for(q_free, k - 1))) break;
        if (lane == 0) {
          bulk::arrive_expect_tx(q_full, f.both ? 2 * TB : TB);
          load_tile<DH>(q_at, &mq, f.head0, f.x.begin + f.row0 * kTile, q_full);
          if (f.both) load_tile<DH>(q_at + TB, &mq, f.head1, f.x.begin + f.row1 * kTile, q_full);
        }
        more = take.next();
        for (int j = 1; ok && j < f.n; ++j) ok = put(j);
        if (!ok || !(ok = feed.mend_all())) break;
      }
      if (ok && (ok = feed.mend_all() && (k == 0 || wait(q_free, k - 1, a))) && lane == 0) tc::arrive(q_full);
      if (!ok) {
        bulk::warp_wait(q_full, uint32_t(k) & 1u, a.wait_ns);
        feed.drain();
      }
    } else if (warp == 8) {
      // products: at step j, o += p v of key tile j - 1 and x of key tile j, of query tile 0, then of 1
      // (one issuing thread: two would fall into step, and both tiles' softmax would wait together)
      Place<NS> ks(0), vs(1);
      uint32_t done[2] = {0, 0};  // p's consumed
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!(ok = wait(q_full, k, a))) break;
        const FwdUnit f = given[k & 3].uniform();
        if (f.n < 0) break;
        bool acc[2] = {false, false};
        if (!(ok = wait(full + 8 * ks.s, ks.phase, a))) break;
        for (int j = 0; j <= f.n; ++j) {
          const Place<NS> v = vs, key = ks;
          if (j > 0) vs.skip(2);
          ks.skip(2);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // while the first tile's products run: this step's value tile is there for both; the next
            // step's tiles are looked for before the second tile's
            if (i == 1 && j + 1 < f.n && !(ok = wait(full + 8 * vs.s, vs.phase, a) && wait(full + 8 * ks.s, ks.phase, a)))
              break;
            if (i == 0 && j == f.n && !(ok = wait(full + 8 * v.s, v.phase, a))) break;  // (the last may be mended)
            if (i == 1 && !f.both) continue;
            if (j > 0 && f.meets(i, j - 1)) {
              if (!(ok = wait(p_ready + 8 * i, done[i], a))) break;
              ++done[i];
              tc::fence_after();
              mma_cols_at<DH>(o_at + DH * i, s_at + 128 * i, s_at + 128 * i + 32, kv_at + v.s * TB, acc[i]);
              acc[i] = true;
            }
            if (j < f.n && f.meets(i, j)) {
              // x overwrites p: the products execute in the order they are issued
              mma_rows_at<DH>(s_at + 128 * i, q_at + i * TB, kv_at + key.s * TB);
              tc::commit(s_full + 8 * i);
            }
          }
          if (!ok) break;
          if (j > 0) tc::commit(free + 8 * v.s);
          if (j < f.n) tc::commit(free + 8 * key.s);
          if (j == f.n - 1) tc::commit(q_free);
          if (j == f.n) {  // (a barrier for each: a warpgroup without work would fall phases behind one of both)
            tc::commit(o_full);
            if (f.both) tc::commit(o_full + 8);
          }
        }
        ks.back(2);  // (the last step has no key tile)
      }
      if (!ok) {
        tc::commit(drain);
        wait(drain, 0, a);
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int i = warp >> 2;  // query tile of this warpgroup
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t x_at = s_at + 128 * i + lanes, acc_at = o_at + DH * i + lanes;
    const float c = a.scale * kLog2e;
    uint32_t seen = 0, units = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!(ok = wait(q_full, k, a))) break;
      const FwdUnit f = given[k & 3].uniform();
      if (f.n < 0) break;
      __syncwarp();
      if (lane == 0) tc::arrive(q_free);  // (a warpgroup without work in this unit keeps step with the others)
      if (i == 1 && !f.both) continue;
      const int tile = i ? f.row1 : f.row0;
      const int row = tile * kTile + int(threadIdx.x & 127);  // position inside the sample
      float m = -INFINITY, l = 0.f;
      bool first = true;
      for (int j = 0; j < f.n; ++j) {
        if (!f.meets(i, j)) continue;
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
      if (!ok || !(ok = wait(o_full + 8 * i, units, a))) break;
      ++units;
      tc::fence_after();
      const int64_t pos = int64_t(f.x.begin) + row;
      const int head = i ? f.head1 : f.head0;
      const float inv = 1.f / l;
#pragma unroll
      for (int b = 0; b < DH / 32; ++b) {
        float o[32];
        tc::ld32(acc_at + 32 * b, o);
        tc::wait_ld();
        tc::tie32(o);
        store32(a.o + ((pos - lane) * a.heads + head) * DH + 32 * b, int64_t(a.heads) * DH, f.x.L - row + lane, o, inv);
      }
      if (row < f.x.L) a.lse[int64_t(head) * a.T + pos] = (m * c + log2f(l)) * (1.f / kLog2e);
      tc::fence_before();
    }
  }
  __syncthreads();
  if (warp == 8) {
    tc::fence_after();
    tc::dealloc(s_at, 512);
  }
}

// ------------------------------------------------------------- backward

constexpr int kBwdThreads = 320;  // eight warps for the elementwise part, one for products, one for loads
template <int DH> constexpr int bwd_slots() { return DH == 64 ? 10 : 5; }
template <int DH> constexpr int bwd_smem() { return tile_bytes<DH>() * (2 + bwd_slots<DH>()); }

__device__ __forceinline__ Tile uniform_tile(Tile x) {
  auto same = [](int& v) { v = int(tc::uni(uint32_t(v))); };
  same(x.begin), same(x.L), same(x.uih), same(x.t), same(x.part), same(x.split);
  return x;
}

// dq of one query tile and head a unit.  A thread holds one query row and 64 of
// the 128 keys.  Per key tile: x = q k^T and do v^T into 128 columns each; p = exp(x - lse)
// stays in registers and frees x; ds = p * (do v^T - delta), in bf16, goes over do v^T and
// multiplies k.  do v^T has two places that take turns, so the next tile's x and do v^T are computed while
// ds is formed (with one place they waited for the product of ds: 323 us a backward pass instead of 314).
// delta = dout.out: the unit's rows of out come through the ring in front of its
// keys.  Where there is one key tile delta = sum p * (do v^T) is at hand instead, free of the rounding
// of out, which matters most there: few keys leave out about as large as v (8 samples of up to
// 511 positions, p and ds rounded once: dq and dk 2.6e-3 from 64 bits with dout.out, 2.4e-3 with the sum;
// bf16 results alone are 1.7e-3).
struct DqUnit {
  Tile x;
  int head, kv_head, nk, n;  // n < 0: no more units
  DqUnit() = default;
  __device__ __forceinline__ DqUnit(const Tile& tile, int h, const AttnArgs& a) : x(tile), head(h) {
    kv_head = head / (a.heads / a.kv_heads);
    int own;
    nk = key_tiles(x, a.causal, own);
    n = nk + own;
  }
  __device__ __forceinline__ int key_tile(int j) const { return j < nk ? j : x.t; }
  __device__ __forceinline__ DqUnit uniform() const {
    DqUnit u = *this;
    auto same = [](int& v) { v = int(tc::uni(uint32_t(v))); };
    u.x = uniform_tile(x);
    same(u.head), same(u.kv_head), same(u.nk), same(u.n);
    return u;
  }
};

template <int DH, bool FINE>
__global__ void __launch_bounds__(kBwdThreads, 1) attn_dq_kernel(const __grid_constant__ CUtensorMap mq,
                                                                 const __grid_constant__ CUtensorMap mk,
                                                                 const __grid_constant__ CUtensorMap mv,
                                                                 const __grid_constant__ CUtensorMap mo,
                                                                 const __grid_constant__ CUtensorMap mdo, AttnArgs a) {
  constexpr int TB = tile_bytes<DH>(), NS = bwd_slots<DH>();
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[15 + 2 * NS];
  __shared__ uint32_t tmem_at;
  __shared__ DqUnit given[4];
  __shared__ float half_delta[2][kTile];
  const uint32_t q_at = bulk::smem_addr(smem), do_at = q_at + TB, kv_at = do_at + TB;
  const uint32_t bar = bulk::smem_addr(bars);
  const uint32_t q_full = bar, q_free = bar + 8, s_full = bar + 16, dp_full = bar + 24, s_read = bar + 40,
                 ds_ready = bar + 48, delta_in = bar + 64, dq_full = bar + 72, tail = bar + 80, drain = bar + 112,
                 full = bar + 120, free = full + 8 * NS;  // (dp_full, ds_ready: one for each place)
  const int warp = int(tc::uni(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (warp == 8) {
    if (lane == 0) {
      for (int i = 0; i < 15 + 2 * NS; ++i) bulk::mbar_init(bar + 8 * i, i == 1 ? 9 : (i >= 5 && i <= 8 ? 8 : 1));
      bulk::fence_init();
    }
  } else if (warp == 9 && lane == 0) {
    tc::prefetch_map(&mq), tc::prefetch_map(&mk), tc::prefetch_map(&mv), tc::prefetch_map(&mo), tc::prefetch_map(&mdo);
  }
  wait_for_launch();
  take_tmem(&tmem_at, warp == 8);
  let_next_launch();
  const uint32_t s_at = tc::uni(tmem_at), dq_at = s_at + 256;
  auto dp_at = [&](uint32_t tile) { return s_at + 128 + 256 * (tile & 1); };

  if (warp == 9) {
    Feeder<DH, NS> feed(smem + 2 * TB, full, free, tail, a);
    Taker take(a, 0, a.heads, 1);
    bool ok = true;
    int k = 0;
    bool more = take.next();
    for (;; ++k) {
      DqUnit f;
      f.n = -1;
      if (more) f = DqUnit(take.tile, take.part, a).uniform();
      if (lane == 0) given[k & 3] = f;
      if (f.n < 0) break;
      auto put = [&](int j) {
        const int at = f.key_tile(j) * kTile;
        return feed.put(&mk, f.kv_head, f.x.begin + at, f.x.L - at, true) &&
               feed.put(&mv, f.kv_head, f.x.begin + at, f.x.L - at, false);
      };
      const int at = f.x.begin + f.x.t * kTile;
      if (!(ok = (f.n == 1 || feed.put(&mo, f.head, at, kTile, false)) && put(0))) break;
      if (k > 0 && !(ok = feed.wait_for(q_free, k - 1))) break;
      if (lane == 0) {
        bulk::arrive_expect_tx(q_full, 2 * TB);
        load_tile<DH>(q_at, &mq, f.head, at, q_full);
        load_tile<DH>(do_at, &mdo, f.head, at, q_full);
      }
      more = take.next();
      for (int j = 1; ok && j < f.n; ++j) ok = put(j);
      if (!ok) break;
    }
    if (ok && (ok = feed.mend_all() && (k == 0 || wait(q_free, k - 1, a))) && lane == 0) tc::arrive(q_full);
    if (!ok) {
      bulk::warp_wait(q_full, uint32_t(k) & 1u, a.wait_ns);
      feed.drain();
    }
  } else if (warp == 8) {
    Place<NS> ks(0), vs(1), kq(0);  // next key and value tile to read, and the key tile of the next dq product
    const uint32_t q_desc = tc::desc_k(q_at), do_desc = tc::desc_k(do_at);
    uint32_t c = 0, sums = 0;       // key tiles so far: do v^T issued, and dq products
    bool ok = true;
    auto scores = [&]() {  // x of the next key tile, into columns that the last tile's readers have left
      const uint32_t k_desc = tc::uni(tc::desc_k(kv_at + ks.s * TB));
      if (!wait(full + 8 * ks.s, ks.phase, a) || (c > 0 && !wait(s_read, c - 1, a))) return false;
      tc::fence_after();
      mma_rows<DH>(s_at, q_desc, k_desc);
      tc::commit(s_full);
      ks.skip(2);
      return true;
    };
    auto products = [&]() {  // its do v^T, over the ds of the last tile but one: the products execute in the order they are issued
      const uint32_t v_desc = tc::uni(tc::desc_k(kv_at + vs.s * TB));
      const uint32_t v_free = tc::uni(free + 8 * vs.s), dp = tc::uni(dp_at(c)), dp_bar = tc::uni(dp_full + 8 * (c & 1));
      if (!wait(full + 8 * vs.s, vs.phase, a)) return false;
      tc::fence_after();
      mma_rows<DH>(dp, do_desc, v_desc);
      tc::commit(dp_bar);
      tc::commit(v_free);
      vs.skip(2);
      ++c;
      return true;
    };
    auto sum = [&](bool acc, bool last) {
      const uint32_t kq_desc = tc::uni(tc::desc_mn(kv_at + kq.s * TB, kBox)), k_free = tc::uni(free + 8 * kq.s);
      const uint32_t dp = tc::uni(dp_at(sums));
      if (!wait(ds_ready + 8 * (sums & 1), sums >> 1, a)) return false;
      tc::fence_after();
      mma_cols<DH>(dq_at, dp, dp + 64, kq_desc, acc);
      if (FINE) mma_cols<DH>(dq_at, dp + 32, dp + 96, kq_desc, true);
      tc::commit(k_free);
      if (last) tc::commit(dq_full);
      kq.skip(2);
      ++sums;
      return true;
    };
    for (int k = 0; ok; ++k) {
      if (!(ok = wait(q_full, k, a))) break;
      const int n = int(tc::uni(uint32_t(given[k & 3].n)));
      if (n < 0) break;
      if (n > 1) ks.skip(1), vs.skip(1), kq.skip(1);  // (the tile of out)
      if (!(ok = scores() && products())) break;
      for (int j = 0; j < n; ++j) {
        const bool more = j + 1 < n;
        // a value tile that is there goes first, one still under way does not hold up dq
        bool here = false;
        if (!more) tc::commit(q_free);
        else if (!(ok = scores())) break;
        else if ((here = __all_sync(0xffffffffu, tc::test(full + 8 * vs.s, vs.phase & 1u))) && !(ok = products())) break;
        if (!(ok = sum(j != 0, !more) && (!more || here || products()))) break;
      }
    }
    if (!ok) {
      tc::commit(drain);
      wait(drain, 0, a);
    }
  } else {
    const int r = threadIdx.x & 127, half = threadIdx.x >> 7;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t cols = 64 * half;
    const float c = a.scale * kLog2e;
    uint32_t seen = 0, item = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!(ok = wait(q_full, k, a))) break;
      const DqUnit f = given[k & 3].uniform();
      if (f.n < 0) break;
      const Tile& x = f.x;
      const int row = x.t * kTile + r;
      const bool live = row < x.L;
      const int64_t pos = int64_t(x.begin) + row;
      const float lse2 = live ? a.lse[int64_t(f.head) * a.T + pos] * kLog2e : 0.f;
      // half of the row's sum each; then everyone's is in
      auto join_delta = [&](float d, float& delta) {
        half_delta[half][r] = d;
        __syncwarp();
        if (lane == 0) tc::arrive(delta_in);
        if (!wait(delta_in, k, a)) return false;
        delta = half_delta[0][r] + half_delta[1][r];
        if (live && half == 0) a.delta[int64_t(f.head) * a.T + pos] = delta;
        return true;
      };
      float delta = 0.f;
      if (f.n > 1) {
        // from the loaded tiles (16-byte pieces of a row lie swizzled: piece c of row r at c ^ (r & 7))
        const int o_slot = int(item % NS);
        if (!(ok = wait(full + 8 * o_slot, item / NS, a))) break;
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < DH / 16; ++i) {
          const int piece = half * (DH / 16) + i;
          const int at = (piece / 8) * kBox + r * 128 + (((piece % 8) ^ (r & 7)) * 16);
          const uint4 v = *reinterpret_cast<const uint4*>(smem + (2 + o_slot) * TB + at);
          const uint4 w = *reinterpret_cast<const uint4*>(smem + TB + at);
          const uint32_t vv[4] = {v.x, v.y, v.z, v.w}, ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            d = fmaf(__uint_as_float(vv[q] << 16), __uint_as_float(ww[q] << 16), d);
            d = fmaf(__uint_as_float(vv[q] & 0xFFFF0000u), __uint_as_float(ww[q] & 0xFFFF0000u), d);
          }
        }
        if (!(ok = join_delta(d, delta))) break;
        if (threadIdx.x == 0) tc::arrive(free + 8 * o_slot);  // everyone has read the tiles of out and dout
        __syncwarp();
      }
      if (lane == 0) tc::arrive(q_free);  // (every warp has its say: none falls phases behind q_full)
      __syncwarp();
      item += (f.n > 1 ? 1u : 0u) + 2 * uint32_t(f.n);
      for (int j = 0; j < f.n; ++j, ++seen) {
        if (!(ok = wait(s_full, seen, a))) break;
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
        const int t0 = f.key_tile(j) * kTile, k0 = t0 + int(cols);
        const bool masked = t0 + kTile > x.uih || (a.causal && t0 + kTile > x.t * kTile);
        const int lim = (a.causal ? min(x.uih, row + 1) : x.uih) - k0, self = row - k0;
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          tc::fma2(p + i, c, c, -lse2, -lse2);
          p[i] = tc::ex2(p[i]);
          p[i + 1] = tc::ex2(p[i + 1]);
        }
        if (!(ok = wait(dp_full + 8 * (seen & 1), seen >> 1, a))) break;
        tc::fence_after();
        const uint32_t dp = dp_at(seen) + lanes + cols;
        if (f.n == 1) {
          float d = 0.f;
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float g[32];
            tc::ld32(dp + 32 * b, g);
            tc::wait_ld();
            tc::tie32(g);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!masked || 32 * b + i < lim || 32 * b + i == self) d = fmaf(p[32 * b + i], g[i], d);
          }
          if (!(ok = join_delta(d, delta))) break;
        }
        uint32_t w[32], rest[32];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float g[32];
          tc::ld32(dp + 32 * b, g);
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
          for (int i = 0; i < 32; i += 2) {
            w[16 * b + i / 2] = tc::pack2(g[i], g[i + 1]);
            if (FINE) rest[16 * b + i / 2] = rest2(w[16 * b + i / 2], g[i], g[i + 1]);
          }
        }
        tc::st32(dp, w);
        if (FINE) tc::st32(dp + 32, rest);
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::arrive(ds_ready + 8 * (seen & 1));
      }
      if (!ok || !(ok = wait(dq_full, k, a))) break;
      tc::fence_after();
#pragma unroll
      for (int b = 0; b < DH / 64; ++b) {
        const int col = half * (DH / 2) + 32 * b;
        float g[32];
        tc::ld32(dq_at + lanes + col, g);
        tc::wait_ld();
        tc::tie32(g);
        store32(a.dq + (pos - lane) * a.dq_stride + f.head * DH + col, a.dq_stride, x.L - row + lane, g, a.scale);
      }
      tc::fence_before();
    }
  }
  __syncthreads();
  if (warp == 8) {
    tc::fence_after();
    tc::dealloc(s_at, 512);
  }
}

// dk and dv of one key tile and key/value head a unit, over the query heads that
// share it and the query tiles that see it, or over half of those.  A thread holds one key and 64 of
// the 128 queries (everything transposed: x^T = k q^T, v do^T).  p^T (bf16)
// goes over x^T and multiplies do, then the next x^T is computed while
// ds^T = p^T * (v do^T - delta) is formed; ds^T goes over v do^T and multiplies q.
// Of two halves each leaves its sums in fp32, and the one that comes second
// adds the other's: two terms, so the order does not show.
struct DkvUnit {
  Tile x;
  int kv_head, first, nq, begin, n;  // query tiles [begin, begin + n) of the list (head by head, nq each); n < 0: no more
  DkvUnit() = default;
  __device__ __forceinline__ DkvUnit(const Tile& tile, int h, const AttnArgs& a) : x(tile), kv_head(h) {
    nq = query_tiles(x, a.causal, first);
    const int all = nq * (a.heads / a.kv_heads), cut = (all + 1) / 2;
    begin = x.split >= 0 && x.part ? cut : 0;
    n = x.split >= 0 ? (x.part ? all - cut : cut) : all;
  }
  __device__ __forceinline__ DkvUnit uniform() const {
    DkvUnit u = *this;
    auto same = [](int& v) { v = int(tc::uni(uint32_t(v))); };
    u.x = uniform_tile(x);
    same(u.kv_head), same(u.first), same(u.nq), same(u.begin), same(u.n);
    return u;
  }
};

// Walks a unit's query tiles: tile index and query head.
struct QueryWalk {
  int tile, head, first, last;
  __device__ __forceinline__ QueryWalk(const DkvUnit& f, const AttnArgs& a)
      : tile(f.first + f.begin % f.nq), head(f.kv_head * (a.heads / a.kv_heads) + f.begin / f.nq), first(f.first),
        last(f.first + f.nq) {}
  __device__ __forceinline__ void next() {
    if (++tile == last) tile = first, ++head;
  }
};

template <int DH, bool FINE>
__global__ void __launch_bounds__(kBwdThreads, 1) attn_dkv_kernel(const __grid_constant__ CUtensorMap mq,
                                                                  const __grid_constant__ CUtensorMap mk,
                                                                  const __grid_constant__ CUtensorMap mv,
                                                                  const __grid_constant__ CUtensorMap mdo, AttnArgs a) {
  constexpr int TB = tile_bytes<DH>(), NS = bwd_slots<DH>();
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[13 + 2 * NS];
  __shared__ uint32_t tmem_at;
  __shared__ DkvUnit given[4];
  __shared__ __align__(16) float row_lse[2][kTile], row_delta[2][kTile];
  const uint32_t k_at = bulk::smem_addr(smem), v_at = k_at + TB, qd_at = v_at + TB;
  const uint32_t bar = bulk::smem_addr(bars);
  const uint32_t kv_full = bar, kv_free = bar + 8, s_full = bar + 16, dp_full = bar + 24, p_ready = bar + 32,
                 ds_ready = bar + 40, rows_in = bar + 48, sums_full = bar + 56, tail = bar + 64, drain = bar + 96,
                 full = bar + 104, free = full + 8 * NS;
  const int warp = int(tc::uni(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (warp == 8) {
    if (lane == 0) {
      for (int i = 0; i < 13 + 2 * NS; ++i) bulk::mbar_init(bar + 8 * i, i == 1 ? 9 : (i >= 4 && i <= 6 ? 8 : 1));
      bulk::fence_init();
    }
  } else if (warp == 9 && lane == 0) {
    tc::prefetch_map(&mq), tc::prefetch_map(&mk), tc::prefetch_map(&mv), tc::prefetch_map(&mdo);
  }
  wait_for_launch();
  take_tmem(&tmem_at, warp == 8);
  const uint32_t s_at = tc::uni(tmem_at), dp_at = s_at + 128, dv_at = s_at + 256, dk_at = s_at + 256 + DH;

  if (warp == 9) {
    Feeder<DH, NS> feed(smem + 2 * TB, full, free, tail, a);
    Taker take(a, 1, a.kv_heads, 1);
    bool ok = true;
    int k = 0;
    bool more = take.next();
    for (;; ++k) {
      DkvUnit f;
      f.n = -1;
      if (more) f = DkvUnit(take.tile, take.part, a).uniform();
      if (lane == 0) given[k & 3] = f;
      if (f.n < 0) break;
      QueryWalk w(f, a);
      auto put = [&]() {
        const int at = w.tile * kTile;
        const bool fine = feed.put(&mq, w.head, f.x.begin + at, f.x.L - at, true) &&
                          feed.put(&mdo, w.head, f.x.begin + at, f.x.L - at, true);
        w.next();
        return fine;
      };
      if (!(ok = put())) break;
      if (k > 0 && !(ok = feed.wait_for(kv_free, k - 1))) break;
      if (lane == 0) {
        bulk::arrive_expect_tx(kv_full, 2 * TB);
        load_tile<DH>(k_at, &mk, f.kv_head, f.x.begin + f.x.t * kTile, kv_full);
        load_tile<DH>(v_at, &mv, f.kv_head, f.x.begin + f.x.t * kTile, kv_full);
      }
      more = take.next();
      for (int j = 1; ok && j < f.n; ++j) ok = put();
      if (!ok) break;
    }
    if (ok && (ok = feed.mend_all() && (k == 0 || wait(kv_free, k - 1, a))) && lane == 0) tc::arrive(kv_full);
    if (!ok) {
      bulk::warp_wait(kv_full, uint32_t(k) & 1u, a.wait_ns);
      feed.drain();
    }
  } else if (warp == 8) {
    Place<NS> qs(0), ds(1);  // tiles of the next x and v do^T
    Place<NS> qk(0), dv(1);  // tiles of the next dk and dv products
    const uint32_t k_desc = tc::desc_k(k_at), v_desc = tc::desc_k(v_at);
    uint32_t c = 0;          // query tiles so far
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!(ok = wait(kv_full, k, a))) break;
      const int n = int(tc::uni(uint32_t(given[k & 3].n)));
      if (n < 0) break;
      // step -1 has the first tile's x^T and v do^T alone; step j dv and dk of tile j and the next tile's; x^T
      // overwrites p^T, v do^T overwrites ds^T: the products execute in the order they are issued
      for (int j = -1; j < n; ++j) {
        const bool sum = j >= 0, more = j + 1 < n;
        {
          const uint32_t do_desc = tc::uni(tc::desc_mn(qd_at + dv.s * TB, kBox)), q_desc = tc::uni(tc::desc_k(qd_at + qs.s * TB));
          const uint32_t do_free = tc::uni(free + 8 * dv.s);
          if (more && !(ok = wait(full + 8 * qs.s, qs.phase, a))) break;
          if (sum && !(ok = wait(p_ready, c, a))) break;
          tc::fence_after();
          if (sum) {
            mma_cols<DH>(dv_at, s_at, s_at + 64, do_desc, j != 0);
            if (FINE) mma_cols<DH>(dv_at, s_at + 32, s_at + 96, do_desc, true);
            tc::commit(do_free);
          }
          if (more) {
            mma_rows<DH>(s_at, k_desc, q_desc);
            tc::commit(s_full);
          }
        }
        const uint32_t q_desc = tc::uni(tc::desc_mn(qd_at + qk.s * TB, kBox)), do_desc = tc::uni(tc::desc_k(qd_at + ds.s * TB));
        const uint32_t q_free = tc::uni(free + 8 * qk.s);
        if (more && !(ok = wait(full + 8 * ds.s, ds.phase, a))) break;
        if (sum && !(ok = wait(ds_ready, c, a))) break;
        tc::fence_after();
        if (sum) {
          mma_cols<DH>(dk_at, dp_at, dp_at + 64, q_desc, j != 0);
          if (FINE) mma_cols<DH>(dk_at, dp_at + 32, dp_at + 96, q_desc, true);
          tc::commit(q_free);
        }
        if (more) {
          mma_rows<DH>(dp_at, v_desc, do_desc);
          tc::commit(dp_full);
          if (j + 2 == n) tc::commit(kv_free);
        } else {
          tc::commit(sums_full);
        }
        if (sum) {
          dv.skip(2), qk.skip(2);
          ++c;
        }
        if (more) qs.skip(2), ds.skip(2);
      }
    }
    if (!ok) {
      tc::commit(drain);
      wait(drain, 0, a);
    }
  } else {
    const int r = threadIdx.x & 127, half = threadIdx.x >> 7;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t cols = 64 * half;
    const float c = a.scale * kLog2e;
    uint32_t seen = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!(ok = wait(kv_full, k, a))) break;
      const DkvUnit f = given[k & 3].uniform();
      if (f.n < 0) break;
      __syncwarp();
      if (lane == 0) tc::arrive(kv_free);  // (every warp has its say: none falls phases behind kv_full)
      const Tile& x = f.x;
      const int key = x.t * kTile + r;
      // lse (in powers of two) or delta of query r of a tile; queries past the sample's end weigh nothing
      QueryWalk w(f, a);
      auto row_value = [&]() {
        const int i = w.tile * kTile + r;
        const int64_t at = int64_t(w.head) * a.T + x.begin + i;
        if (half == 0) return i < x.L ? a.lse[at] * kLog2e : INFINITY;
        return i < x.L ? a.delta[at] : 0.f;
      };
      float next = row_value();
      for (int j = 0; j < f.n; ++j, ++seen) {
        // this tile's values are in for everyone (and everyone is done with the last tile but one's)
        (half == 0 ? row_lse : row_delta)[seen & 1][r] = next;
        __syncwarp();
        if (lane == 0) tc::arrive(rows_in);
        const int i0 = w.tile * kTile;
        w.next();
        if (j + 1 < f.n) next = row_value();
        if (!(ok = wait(rows_in, seen, a) && wait(s_full, seen, a))) break;
        tc::fence_after();
        float p[64];
        tc::ld32(s_at + lanes + cols, p);
        tc::ld32(s_at + lanes + cols + 32, p + 32);
        tc::wait_ld();
        tc::tie32(p);
        tc::tie32(p + 32);
        const float4* ls = reinterpret_cast<const float4*>(&row_lse[seen & 1][cols]);
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          const float4 z = ls[i / 4];
          tc::fma2(p + i, c, c, -z.x, -z.y);
          tc::fma2(p + i + 2, c, c, -z.z, -z.w);
#pragma unroll
          for (int q = 0; q < 4; ++q) p[i + q] = tc::ex2(p[i + q]);
        }
        if (x.t * kTile + kTile > x.uih || (a.causal && i0 < x.t * kTile + kTile)) {
          // query i0 + cols + i sees this key from `from` on, or only where it is the key's own position
          const int self = key - i0 - int(cols);
          const int from = key >= x.uih ? 128 : (a.causal ? self : -1);
#pragma unroll
          for (int i = 0; i < 64; ++i) p[i] = (i >= from || i == self) ? p[i] : 0.f;
        }
        uint32_t pk[32], rest[32];
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          pk[i / 2] = tc::pack2(p[i], p[i + 1]);
          if (FINE) rest[i / 2] = rest2(pk[i / 2], p[i], p[i + 1]);
        }
        tc::st32(s_at + lanes + cols, pk);
        if (FINE) tc::st32(s_at + lanes + cols + 32, rest);
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::arrive(p_ready);
        if (!(ok = wait(dp_full, seen, a))) break;
        tc::fence_after();
        const float4* dl = reinterpret_cast<const float4*>(&row_delta[seen & 1][cols]);
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
            pk[16 * b + i / 2] = tc::pack2(g[i], g[i + 1]);
            pk[16 * b + i / 2 + 1] = tc::pack2(g[i + 2], g[i + 3]);
            if (FINE) {
              rest[16 * b + i / 2] = rest2(pk[16 * b + i / 2], g[i], g[i + 1]);
              rest[16 * b + i / 2 + 1] = rest2(pk[16 * b + i / 2 + 1], g[i + 2], g[i + 3]);
            }
          }
        }
        tc::st32(dp_at + lanes + cols, pk);
        if (FINE) tc::st32(dp_at + lanes + cols + 32, rest);
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::arrive(ds_ready);
      }
      if (!ok || !(ok = wait(sums_full, k, a))) break;
      tc::fence_after();
      const int64_t pos = int64_t(x.begin) + key - lane;  // of the warp's first key
      const int live = x.L - key + lane;
      const int64_t stride = half == 0 ? a.dv_stride : a.dk_stride;
      __nv_bfloat16* to = (half == 0 ? a.dv : a.dk) + pos * stride + f.kv_head * DH;
      const uint32_t from = (half == 0 ? dv_at : dk_at) + lanes;
      const float scale = half == 0 ? 1.f : a.scale;
      const float4* other = nullptr;
      if (x.split >= 0) {
        const int64_t unit = int64_t(x.split) * a.kv_heads + f.kv_head;
        float4* both = reinterpret_cast<float4*>(a.partial) + (unit * 8 + warp) * (2 * DH * 8);
        int32_t* flag = a.flags + unit * 8 + warp;
        // is the other half's share there?  If not, leave this one's, and ask again
        int32_t came = 0;
        if (lane == 0) came = *reinterpret_cast<volatile int32_t*>(flag);
        came = __shfl_sync(0xffffffffu, came, 0);
        if (came == 0) {
          float4* mine = both + x.part * (DH * 8);
#pragma unroll
          for (int b = 0; b < DH / 32; ++b) {
            float g[32];
            tc::ld32(from + 32 * b, g);
            tc::wait_ld();
            tc::tie32(g);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              __stcg(mine + (b * 8 + i) * 32 + lane, make_float4(g[4 * i], g[4 * i + 1], g[4 * i + 2], g[4 * i + 3]));
          }
          __threadfence();
          __syncwarp();
          if (lane == 0) came = atomicAdd(flag, 1);
          came = __shfl_sync(0xffffffffu, came, 0);
          if (came == 0) {
            tc::fence_before();
            continue;  // the other half adds them up
          }
        }
        __threadfence();
        other = both + (1 - x.part) * (DH * 8);
      }
#pragma unroll
      for (int b = 0; b < DH / 32; ++b) {
        float g[32];
        tc::ld32(from + 32 * b, g);
        tc::wait_ld();
        tc::tie32(g);
        if (other) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 z = __ldcg(other + (b * 8 + i) * 32 + lane);
            g[4 * i] += z.x, g[4 * i + 1] += z.y, g[4 * i + 2] += z.z, g[4 * i + 3] += z.w;
          }
        }
        store32(to + 32 * b, stride, live, g, scale);
      }
      tc::fence_before();
    }
  }
  __syncthreads();
  if (warp == 8) {
    tc::fence_after();
    tc::dealloc(s_at, 512);
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
  Plan* plan = nullptr;
  Tile *by_query = nullptr, *by_key = nullptr;
  float *delta = nullptr, *partial = nullptr;
  int32_t* flags = nullptr;
};

// Both passes take the same workspace; the forward pass uses its first two parts.
template <class Ws>
void take_attn(int64_t T, int64_t S, int32_t Hq, int32_t Hkv, int32_t Dh, Ws& ws, AttnWs& W) {
  const int64_t tiles = most_tiles(T, S), cut = most_split(sm_count());
  const int64_t halves = tiles * Hkv < cut ? tiles * Hkv : cut;  // units cut in half
  W.plan = ws.template take<Plan>(1);
  W.by_query = ws.template take<Tile>(size_t(tiles));
  W.by_key = ws.template take<Tile>(size_t(2 * tiles < tiles + cut ? 2 * tiles : tiles + cut));
  W.delta = ws.template take<float>(size_t(Hq) * size_t(T));
  W.flags = ws.template take<int32_t>(size_t(cut) * 8);
  W.partial = ws.template take<float>(size_t(halves) * 2 * 2 * kTile * size_t(Dh));
}

// Small batches do without the planning kernel: where every unit has an SM of its own there is no
// order to find, and with at most 32 samples a warp finds a unit's tile faster than a launch takes
// (8 samples of up to 511 positions, 4 heads: about 3 us less a pass, 12 to 14 us forward and 21 to 22 backward).
bool each_its_own(int64_t S, int64_t units) { return S <= 32 && units <= sm_count(); }

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

// Launches a kernel that may start while the one before it in the stream still runs (it waits
// for that one's end itself, before it reads anything).
template <class... Params, class... Args>
void launch_after(void (*kern)(Params...), int64_t grid, int threads, int smem, cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

std::atomic<uint64_t> g_fwd_ready[2];

}  // namespace
}  // namespace fs

using namespace fs;

extern "C" size_t fs_jagged_attn_workspace_size(int64_t T, int64_t S, int32_t heads, int32_t kv_heads,
                                                int32_t head_dim) {
  if (T < 0 || S < 0 || heads < 1 || kv_heads < 1 || (head_dim != 64 && head_dim != 128)) return 0;
  WsCounter c;
  AttnWs W;
  take_attn(T, S, heads, kv_heads, head_dim, c, W);
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
  take_attn(T, S, heads, kv_heads, head_dim, cur, W);
  CUtensorMap mq, mk, mv;
  if (!encode(&mq, q, T, int64_t(heads) * head_dim, q_stride) || !encode(&mk, k, T, int64_t(kv_heads) * head_dim, k_stride) ||
      !encode(&mv, v, T, int64_t(kv_heads) * head_dim, v_stride))
    return FS_ERR_CUDA;
  AttnArgs a{};
  a.plan = W.plan, a.tiles = W.by_query;
  a.heads = heads, a.kv_heads = kv_heads, a.T = T, a.causal = causal != 0, a.scale = scale;
  a.offsets = offsets, a.cand = cand_len, a.S = int32_t(S);
  a.o = static_cast<__nv_bfloat16*>(out), a.lse = lse, a.err = err;
  a.wait_ns = uint64_t(spin_limit()) * 256u, a.skip_block = debug_skip_tile();
  const bool by_head = heads / kv_heads % 2 == 0;  // two heads of one tile share a block, else two tiles of one head
  const int parts = by_head ? heads / 2 : heads;
  const int64_t units = most_tiles(T, S) * parts;
  const bool listed = !each_its_own(S, units);
  if (listed)
    attn_plan_kernel<<<1, kPlanThreads, 0, st>>>(offsets, S, T, cand_len, a.causal, by_head ? 1 : 2, kv_heads,
                                                 heads / kv_heads, sm_count(), W.plan, W.by_query, nullptr, nullptr, err);
  else
    a.plan = nullptr;
  const int64_t grid = units < sm_count() ? units : sm_count();
  if (head_dim == 64) {
    if (!prepare_kernel(attn_fwd_kernel<64>, fwd_smem<64>(), kFwdRegs, g_fwd_ready[0])) return FS_ERR_CUDA;
    launch_after(attn_fwd_kernel<64>, grid, kFwdThreads, fwd_smem<64>(), st, mq, mk, mv, a, parts);
  } else {
    if (!prepare_kernel(attn_fwd_kernel<128>, fwd_smem<128>(), kFwdRegs, g_fwd_ready[1])) return FS_ERR_CUDA;
    launch_after(attn_fwd_kernel<128>, grid, kFwdThreads, fwd_smem<128>(), st, mq, mk, mv, a, parts);
  }
  count_launch(listed ? 2 : 1);
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
  take_attn(T, S, heads, kv_heads, head_dim, cur, W);
  CUtensorMap mq, mk, mv, mo, mdo;
  if (!encode(&mq, q, T, ow, q_stride) || !encode(&mk, k, T, kw, k_stride) || !encode(&mv, v, T, kw, v_stride) ||
      !encode(&mo, out, T, ow, ow) || !encode(&mdo, dout, T, ow, ow))
    return FS_ERR_CUDA;
  AttnArgs a{};
  a.plan = W.plan;
  a.heads = heads, a.kv_heads = kv_heads, a.T = T, a.causal = causal != 0, a.scale = scale;
  a.offsets = offsets, a.cand = cand_len, a.S = int32_t(S);
  a.lse = const_cast<float*>(lse), a.delta = W.delta, a.partial = W.partial, a.flags = W.flags, a.err = err;
  a.dq = static_cast<__nv_bfloat16*>(dq), a.dk = static_cast<__nv_bfloat16*>(dk), a.dv = static_cast<__nv_bfloat16*>(dv);
  a.dq_stride = dq_stride, a.dk_stride = dk_stride, a.dv_stride = dv_stride;
  a.wait_ns = uint64_t(spin_limit()) * 256u, a.skip_block = debug_skip_tile();
  const bool listed = !each_its_own(S, most_tiles(T, S) * heads);
  if (listed)
    attn_plan_kernel<<<1, kPlanThreads, 0, st>>>(offsets, S, T, cand_len, a.causal, 1, kv_heads, heads / kv_heads,
                                                 sm_count(), W.plan, W.by_query, W.by_key, W.flags, err);
  else
    a.plan = nullptr;
  const int64_t tiles = most_tiles(T, S), sms = sm_count();
  const int64_t gq = tiles * heads < sms ? tiles * heads : sms, gk = 2 * tiles * kv_heads < sms ? 2 * tiles * kv_heads : sms;
  AttnArgs b = a;
  a.tiles = W.by_query, b.tiles = W.by_key;
  auto launch = [&](auto dh, auto fine) {
    constexpr int DH = decltype(dh)::value;
    constexpr bool FINE = decltype(fine)::value;
    static std::atomic<uint64_t> ready[2];
    if (!prepare_kernel(attn_dq_kernel<DH, FINE>, bwd_smem<DH>(), 0, ready[0]) ||
        !prepare_kernel(attn_dkv_kernel<DH, FINE>, bwd_smem<DH>(), 0, ready[1]))
      return false;
    launch_after(attn_dq_kernel<DH, FINE>, gq, kBwdThreads, bwd_smem<DH>(), st, mq, mk, mv, mo, mdo, a);
    launch_after(attn_dkv_kernel<DH, FINE>, gk, kBwdThreads, bwd_smem<DH>(), st, mq, mk, mv, mdo, b);
    return true;
  };
  using std::integral_constant;
  const integral_constant<int, 64> d64;
  const integral_constant<int, 128> d128;
  const bool ok = !listed ? (head_dim == 64 ? launch(d64, std::true_type{}) : launch(d128, std::true_type{}))
                          : (head_dim == 64 ? launch(d64, std::false_type{}) : launch(d128, std::false_type{}));
  if (!ok) return FS_ERR_CUDA;
  count_launch(listed ? 3 : 2);
  return launch_status();
}
