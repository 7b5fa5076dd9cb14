// Root-mean-square norm of rows with the residual's addition in front of it,
// its output optionally in 8 bits with a scale per row, and its backward pass.
//   h = x + res (stored in the rows' type; res optional)
//   r = 1 / sqrt(mean_d h_d^2 + eps),  y_d = h_d * r * gamma_d
//   8 bits: s = max_d |y_d| / 448,  q_d = e4m3(y_d / s)
// backward, with n_d = h_d * r and w_d = gamma_d * dy_d:
//   dh_d = dsum_d + r * (w_d - n_d * mean_e(w_e * n_e)),  dgamma_d = sum_rows dy_d * n_d
// h is normed as it is stored, so the backward pass, which reads the stored h,
// differentiates what the forward pass computed.  Sums are fp32.
//
// Both passes are bound by HBM: every input is read once and every output
// written once, a row staying in the registers of the G threads that own it.
// 400,000 rows of 512 bf16: forward with residual and 8-bit output 223 us, 6.4 TB/s;
// backward 272 us, 6.0 TB/s.  A few hundred rows take 3 and 4.5 us.
#include <cooperative_groups.h>

#include <type_traits>

#include "convert.cuh"
#include "fs_common.cuh"

namespace fs {
namespace {

constexpr int kNormThreads = 256;
constexpr int kMaxNormDim = 8192;

template <class Op>
__device__ __forceinline__ float group_all(float v, int lanes, Op op) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Sum or maximum of one value per thread over the G threads that own a row:
// lanes of a warp (G <= 32), or the whole block (G = kNormThreads).  `red`
// holds one value per warp and alternates between calls (`turn`), so one
// barrier per call is enough.
template <int G, class Op>
__device__ __forceinline__ float row_all(float v, Op op, float (*red)[kNormThreads / 32], int& turn) {
  if constexpr (G <= 32) {
    return group_all(v, G, op);
  } else {
    v = group_all(v, 32, op);
    if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = v;
    __syncthreads();
    float s = red[turn][0];
#pragma unroll
    for (int w = 1; w < kNormThreads / 32; ++w) s = op(s, red[turn][w]);
    turn = turn == 2 ? 0 : turn + 1;
    return s;
  }
}

struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// a NaN on either side stays
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return (a > b || a != a) ? a : b; }
};

template <int VEC>
__device__ __forceinline__ void load_gamma(const float* gamma, int c, float (&w)[VEC]) {
  if constexpr (VEC == 8) {
    float a[4], b[4];
    load_vec<F32, 4, false>(gamma, c, a);
    load_vec<F32, 4, false>(gamma, c + 4, b);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = a[k], w[k + 4] = b[k];
  } else {
    load_vec<F32, VEC, false>(gamma, c, w);
  }
}

// G threads per row, each with NC chunks of VEC elements (chunk j of thread g
// starts at (j * G + g) * VEC).  The next row's chunks are loaded, and held as
// loaded, before the current row is worked on.
template <class E, class EY, int VEC, int G, int NC, bool RES>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const void* x, const void* res, int64_t T,
                                                            int32_t dim, const float* __restrict__ gamma, float eps,
                                                            void* sum_out /* may be x or res */, void* __restrict__ y,
                                                            float* __restrict__ y_scale, float* __restrict__ rstd) {
  __shared__ float red[3][kNormThreads / 32];
  int turn = 0;
  constexpr int RPB = kNormThreads / G;
  const int g = threadIdx.x % G;
  const int64_t step = int64_t(gridDim.x) * RPB;
  Raw<E, VEC> nx[NC], nr[NC];
  auto load_row = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = (j * G + g) * VEC;
      if (row < T && c < dim) {
        fetch<true>(nx[j], x, row * dim + c);
        if (RES) fetch<true>(nr[j], res, row * dim + c);
      }
    }
  };
  load_row(int64_t(blockIdx.x) * RPB + threadIdx.x / G);
  // every thread of a warp or block runs the same iterations (its row may lie past the end)
  for (int64_t base = int64_t(blockIdx.x) * RPB; base < T; base += step) {
    const int64_t row = base + threadIdx.x / G;
    const bool live = row < T;
    float h[NC][VEC];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = (j * G + g) * VEC;
      const bool in = live && c < dim;
      if (in) {
        unpack(nx[j], h[j]);
        if constexpr (RES) {
          float r[VEC];
          unpack(nr[j], r);
#pragma unroll
          for (int k = 0; k < VEC; ++k) h[j][k] += r[k];
          if constexpr (E::kBytes == 2) {  // the norm is of the sum as it is stored
#pragma unroll
            for (int k = 0; k < VEC; ++k) h[j][k] = __bfloat162float(__float2bfloat16_rn(h[j][k]));
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) h[j][k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) ss = fmaf(h[j][k], h[j][k], ss);
    }
    load_row(row + step);
    if constexpr (RES) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int c = (j * G + g) * VEC;
        if (live && c < dim) store_vec<E, VEC, false>(sum_out, row * dim + c, h[j]);
      }
    }
    ss = row_all<G>(ss, Add{}, red, turn);
    const float rs = 1.f / sqrtf(ss / float(dim) + eps);
    if (live && g == 0 && rstd) rstd[row] = rs;
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = (j * G + g) * VEC;
      if (live && c < dim) {
        float w[VEC];
        load_gamma<VEC>(gamma, c, w);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          h[j][k] = h[j][k] * rs * w[k];
          if constexpr (EY::kBytes == 1) top = Max{}(fabsf(h[j][k]), top);
        }
        if constexpr (EY::kBytes != 1) store_vec<EY, VEC, true>(y, row * dim + c, h[j]);
      }
    }
    if constexpr (EY::kBytes == 1) {
      top = row_all<G>(top, Max{}, red, turn);
      const float s = top / 448.f;
      if (live && g == 0) y_scale[row] = s;
      // q is e4m3 of the fp32 quotient y / s, rounded once: one reciprocal a row and per element a product and one
      // correction by its residual (Markstein, IBM J. Res. Dev. 34, 1990: y - q s is exact in an fma, and the
      // corrected quotient correctly rounded).  The product alone sends one in sixteen quotients that lie in the middle
      // between two e4m3 values the wrong way.  Small rows are lifted by 2^100 first, exactly, so that no residual
      // and no reciprocal leaves the normal range.  No scale (a row of zeros, or NaN): y as it is; an
      // infinite one: 0, and NaN where y is infinite.
      float d = s;
      if (s < 0x1p-90f && s > 0.f) {
        d *= 0x1p100f;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int k = 0; k < VEC; ++k) h[j][k] *= 0x1p100f;
      }
      const float f = s > 0.f ? 1.f / d : 1.f;
      if (!(s > 0.f)) d = 1.f;
      if (isinf(s)) d = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int c = (j * G + g) * VEC;
        if (live && c < dim) {
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            const float q = h[j][k] * f;
            h[j][k] = fmaf(-fmaf(q, d, -h[j][k]), f, q);  // (signs so that -0 stays -0)
          }
          store_vec<EY, VEC, true>(y, row * dim + c, h[j]);
        }
      }
    }
  }
}

// Backward: as the forward pass; a thread keeps its columns' share of dgamma
// in registers over its rows, a block adds its threads' shares in thread
// order, and gamma_sum_kernel adds the blocks' shares in block order: the
// result does not depend on the order in which blocks run.
// CLUSTER: the whole grid is one thread-block cluster, and the blocks' shares are added through distributed shared
// memory in block order: one launch (`part` is dgamma then).
template <class E, int VEC, int G, int NC, bool SUM, bool CLUSTER>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_kernel(const void* dy, const void* dsum, const void* hin,
                                                                int64_t T, int32_t dim, const float* __restrict__ gamma,
                                                                const float* __restrict__ rstd,
                                                                void* dh /* may be dy or dsum */,
                                                                float* __restrict__ part) {
  __shared__ float red[3][kNormThreads / 32];
  extern __shared__ float cols[];  // [RPB][dim] shares of dgamma (not needed where one row has the block, outside clusters)
  int turn = 0;
  constexpr int RPB = kNormThreads / G;
  const int g = threadIdx.x % G;
  const int64_t step = int64_t(gridDim.x) * RPB;
  float dg[NC][VEC];
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int k = 0; k < VEC; ++k) dg[j][k] = 0.f;
  Raw<E, VEC> nh[NC], ny[NC], nd[NC];
  float nrs = 0.f;
  auto load_row = [&](int64_t row) {
    if (row < T) nrs = __ldcs(rstd + row);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = (j * G + g) * VEC;
      if (row < T && c < dim) {
        fetch<true>(nh[j], hin, row * dim + c);
        fetch<true>(ny[j], dy, row * dim + c);
        if (SUM) fetch<true>(nd[j], dsum, row * dim + c);
      }
    }
  };
  load_row(int64_t(blockIdx.x) * RPB + threadIdx.x / G);
  for (int64_t base = int64_t(blockIdx.x) * RPB; base < T; base += step) {
    const int64_t row = base + threadIdx.x / G;
    const bool live = row < T;
    const float rs = nrs;
    float n[NC][VEC], w[NC][VEC];
    Raw<E, VEC> d[NC];
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = (j * G + g) * VEC;
      d[j] = nd[j];
      if (live && c < dim) {
        float gm[VEC];
        unpack(nh[j], n[j]);
        unpack(ny[j], w[j]);
        load_gamma<VEC>(gamma, c, gm);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          n[j][k] *= rs;
          dg[j][k] = fmaf(w[j][k], n[j][k], dg[j][k]);
          w[j][k] *= gm[k];
          dot = fmaf(w[j][k], n[j][k], dot);
        }
      }
    }
    load_row(row + step);
    dot = row_all<G>(dot, Add{}, red, turn) / float(dim);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = (j * G + g) * VEC;
      if (live && c < dim) {
        float v[VEC];
        if constexpr (SUM) {
          unpack(d[j], v);
#pragma unroll
          for (int k = 0; k < VEC; ++k) v[k] += rs * (w[j][k] - n[j][k] * dot);
        } else {
#pragma unroll
          for (int k = 0; k < VEC; ++k) v[k] = rs * (w[j][k] - n[j][k] * dot);
        }
        store_vec<E, VEC, true>(dh, row * dim + c, v);
      }
    }
  }
  if constexpr (RPB == 1 && !CLUSTER) {
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const int c = (j * G + g) * VEC + k;
        if (c < dim) part[int64_t(blockIdx.x) * dim + c] = dg[j][k];
      }
  } else {
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const int c = (j * G + g) * VEC + k;
        if (c < dim) cols[(threadIdx.x / G) * dim + c] = dg[j][k];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < dim; c += kNormThreads) {
      float s = cols[c];
      for (int r = 1; r < RPB; ++r) s += cols[r * dim + c];
      if constexpr (CLUSTER) cols[c] = s;
      else part[int64_t(blockIdx.x) * dim + c] = s;
    }
    if constexpr (CLUSTER) {
      namespace cg = cooperative_groups;
      cg::cluster_group all = cg::this_cluster();
      all.sync();
      for (int c = int(blockIdx.x) * kNormThreads + threadIdx.x; c < dim; c += int(gridDim.x) * kNormThreads) {
        float s = 0.f;
        for (unsigned b = 0; b < gridDim.x; ++b) s += *all.map_shared_rank(cols + c, b);
        part[c] = s;
      }
      all.sync();  // no block leaves while another reads its shares
    }
  }
}

// dgamma[c] = sum over the blocks' shares, 8 rows of threads in block order
// (fp32 within a row of threads, then across them).
__global__ void __launch_bounds__(256) gamma_sum_kernel(const float* __restrict__ part, int32_t blocks, int32_t dim,
                                                        float* __restrict__ dgamma) {
  __shared__ float s[8][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
  float a = 0.f;
  if (c < dim)
    for (int b = r; b < blocks; b += 8) a += part[int64_t(b) * dim + c];
  s[r][threadIdx.x & 31] = a;
  __syncthreads();
  if (r == 0 && c < dim) {
#pragma unroll
    for (int q = 1; q < 8; ++q) a += s[q][threadIdx.x & 31];
    dgamma[c] = a;
  }
}

// Threads per row and chunks per thread for a row of `dim` elements, VEC each:
// a warp's lanes up to 64 chunks a row, the whole block beyond (kMaxNormDim
// elements are 8 chunks of 4 or 32 of 1).
template <int VEC, class F>
bool pick_shape(int32_t dim, F f) {
  const int chunks = (dim + VEC - 1) / VEC;
  if (chunks <= 8) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  else if (chunks <= 16) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  else if (chunks <= 32) f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
  else if (chunks <= 64) f(std::integral_constant<int, 32>{}, std::integral_constant<int, 2>{});
  else if (chunks <= kNormThreads) f(std::integral_constant<int, kNormThreads>{}, std::integral_constant<int, 1>{});
  else if (chunks <= 2 * kNormThreads) f(std::integral_constant<int, kNormThreads>{}, std::integral_constant<int, 2>{});
  else if (chunks <= 8 * kNormThreads) f(std::integral_constant<int, kNormThreads>{}, std::integral_constant<int, 8>{});
  else if constexpr (VEC == 1) f(std::integral_constant<int, kNormThreads>{}, std::integral_constant<int, 32>{});
  else return false;
  return true;
}

// Blocks of the forward pass: many more than fit at once, so that they end together (400K rows of 512 bf16 to
// 8 bits: 227 us with 32 an SM, 242 with 8, of which three fit at a time).
int norm_grid(int64_t T, int rows_per_block) {
  const int64_t want = (T + rows_per_block - 1) / rows_per_block, most = int64_t(sm_count()) * 32;
  return int(want < most ? want : most);
}

// Blocks of the backward pass: as many as run at once, since each leaves a share of
// dgamma that is read once more (400K rows of 512 bf16: 275 us with the two an SM that fit, 286 with eight).
constexpr int kMostResident = 8;

template <class K>
int resident_blocks(K kern, size_t smem) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kNormThreads, smem) != cudaSuccess || n < 1) n = 1;
  return n < kMostResident ? n : kMostResident;
}

// A batch that would take at most kOneCluster blocks runs as one cluster of at most 8:
// the second launch costs more than the blocks it saves (515 rows of 64 f32: about 4 us less, 9.3 us a pass).
constexpr int kOneCluster = 64, kClusterBlocks = 8;

template <class... Params, class... Args>
bool cluster_launch(void (*kern)(Params...), int blocks, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(kNormThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(blocks);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, Params(args)...) == cudaSuccess;
}

}  // namespace
}  // namespace fs

using namespace fs;

extern "C" fs_status fs_rmsnorm(const void* x, const void* res, int64_t T, int32_t dim, fs_dtype dtype,
                                const float* gamma, float eps, void* sum_out, void* y, fs_dtype y_dtype,
                                float* y_scale, float* rstd, fs_stream_t stream) {
  FS_NVTX_RANGE();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T < 0 || T > INT32_MAX || dim < 1 || dim > kMaxNormDim || !(eps >= 0.f)) return FS_ERR_INVALID_ARG;
  if ((dtype != FS_F32 && dtype != FS_BF16) || (y_dtype != dtype && y_dtype != FS_E4M3)) return FS_ERR_INVALID_ARG;
  if (y_dtype != FS_E4M3 && y_scale) return FS_ERR_INVALID_ARG;
  if (T == 0) return FS_OK;  // (an empty tensor's pointer may be NULL)
  if ((res == nullptr) != (sum_out == nullptr) || (y_dtype == FS_E4M3) != (y_scale != nullptr)) return FS_ERR_INVALID_ARG;
  if (!x || !gamma || !y) return FS_ERR_INVALID_ARG;
  const size_t eb = dtype == FS_F32 ? 4 : 2, yb = y_dtype == FS_E4M3 ? 1 : eb;
  if (!aligned(x, eb) || !aligned(res, eb) || !aligned(sum_out, eb) || !aligned(y, yb) || !aligned(gamma, 4) ||
      !aligned(y_scale, 4) || !aligned(rstd, 4))
    return FS_ERR_ALIGNMENT;
  const size_t vec = dtype == FS_F32 ? 4 : 8;
  const bool wide = dim % vec == 0 && aligned(x, 16) && aligned(res, 16) && aligned(sum_out, 16) &&
                    aligned(y, vec * yb) && aligned(gamma, 16);
  auto go = [&](auto e, auto ey, auto v) {
    constexpr int VEC = decltype(v)::value;
    return pick_shape<VEC>(dim, [&](auto gg, auto nc) {
      constexpr int G = decltype(gg)::value, NC = decltype(nc)::value;
      const int grid = norm_grid(T, kNormThreads / G);
      if (res)
        norm_kernel<decltype(e), decltype(ey), VEC, G, NC, true><<<grid, kNormThreads, 0, st>>>(
            x, res, T, dim, gamma, eps, sum_out, y, y_scale, rstd);
      else
        norm_kernel<decltype(e), decltype(ey), VEC, G, NC, false><<<grid, kNormThreads, 0, st>>>(
            x, res, T, dim, gamma, eps, sum_out, y, y_scale, rstd);
    });
  };
  using std::integral_constant;
  bool ok;
  if (dtype == FS_F32) {
    if (y_dtype == FS_E4M3)
      ok = wide ? go(F32{}, E4m3{}, integral_constant<int, 4>{}) : go(F32{}, E4m3{}, integral_constant<int, 1>{});
    else
      ok = wide ? go(F32{}, F32{}, integral_constant<int, 4>{}) : go(F32{}, F32{}, integral_constant<int, 1>{});
  } else {
    if (y_dtype == FS_E4M3)
      ok = wide ? go(Bf16{}, E4m3{}, integral_constant<int, 8>{}) : go(Bf16{}, E4m3{}, integral_constant<int, 1>{});
    else
      ok = wide ? go(Bf16{}, Bf16{}, integral_constant<int, 8>{}) : go(Bf16{}, Bf16{}, integral_constant<int, 1>{});
  }
  if (!ok) return FS_ERR_INVALID_ARG;
  count_launch(1);
  return launch_status();
}

extern "C" size_t fs_rmsnorm_backward_workspace_size(int64_t T, int32_t dim) {
  if (T < 0 || dim < 1 || dim > kMaxNormDim) return 0;
  return align_up(size_t(sm_count()) * kMostResident * size_t(dim) * sizeof(float));
}

extern "C" fs_status fs_rmsnorm_backward(const void* dy, const void* dsum, const void* h, int64_t T, int32_t dim,
                                         fs_dtype dtype, const float* gamma, const float* rstd, void* dh,
                                         float* dgamma, void* ws, size_t ws_bytes, fs_stream_t stream) {
  FS_NVTX_RANGE();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T < 0 || T > INT32_MAX || dim < 1 || dim > kMaxNormDim) return FS_ERR_INVALID_ARG;
  if (dtype != FS_F32 && dtype != FS_BF16) return FS_ERR_INVALID_ARG;
  if (!dgamma) return FS_ERR_INVALID_ARG;
  if (!aligned(dgamma, 4)) return FS_ERR_ALIGNMENT;
  if (T == 0) return cudaMemsetAsync(dgamma, 0, size_t(dim) * sizeof(float), st) == cudaSuccess ? FS_OK : FS_ERR_CUDA;
  if (!dy || !h || !gamma || !rstd || !dh) return FS_ERR_INVALID_ARG;
  const size_t eb = dtype == FS_F32 ? 4 : 2, vec = dtype == FS_F32 ? 4 : 8;
  if (!aligned(dy, eb) || !aligned(dsum, eb) || !aligned(h, eb) || !aligned(dh, eb) || !aligned(gamma, 4) ||
      !aligned(rstd, 4))
    return FS_ERR_ALIGNMENT;
  if (!ws || ws_bytes < fs_rmsnorm_backward_workspace_size(T, dim)) return FS_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return FS_ERR_ALIGNMENT;
  const bool wide = dim % vec == 0 && aligned(dy, 16) && aligned(dsum, 16) && aligned(h, 16) && aligned(dh, 16) &&
                    aligned(gamma, 16);
  float* part = static_cast<float*>(ws);
  int blocks = 0;
  bool launched = true;
  auto go = [&](auto e, auto v) {
    constexpr int VEC = decltype(v)::value;
    return pick_shape<VEC>(dim, [&](auto gg, auto nc) {
      constexpr int G = decltype(gg)::value, NC = decltype(nc)::value;
      constexpr int RPB = kNormThreads / G;
      const int64_t want = (T + RPB - 1) / RPB;
      const size_t sm = size_t(RPB) * dim * sizeof(float);  // at most 32 rows of 64 columns, 8 of 512, one of 8192
      auto launch = [&](auto sum) {
        constexpr bool SUM = decltype(sum)::value;
        if (want <= kOneCluster) {
          launched = cluster_launch(norm_bwd_kernel<decltype(e), VEC, G, NC, SUM, true>,
                                    want < kClusterBlocks ? int(want) : kClusterBlocks, sm, st, dy, dsum, h, T, dim, gamma,
                                    rstd, dh, dgamma);
        } else {
          auto kern = norm_bwd_kernel<decltype(e), VEC, G, NC, SUM, false>;
          const size_t used = RPB > 1 ? sm : 0;
          static const int resident = resident_blocks(kern, size_t(RPB > 1 ? RPB * G * NC * VEC : 0) * sizeof(float));
          const int64_t most = int64_t(sm_count()) * resident;
          blocks = int(want < most ? want : most);
          kern<<<blocks, kNormThreads, used, st>>>(dy, dsum, h, T, dim, gamma, rstd, dh, part);
        }
      };
      if (dsum) launch(std::integral_constant<bool, true>{});
      else launch(std::integral_constant<bool, false>{});
    });
  };
  using std::integral_constant;
  bool ok;
  if (dtype == FS_F32) ok = wide ? go(F32{}, integral_constant<int, 4>{}) : go(F32{}, integral_constant<int, 1>{});
  else ok = wide ? go(Bf16{}, integral_constant<int, 8>{}) : go(Bf16{}, integral_constant<int, 1>{});
  if (!ok) return FS_ERR_INVALID_ARG;
  if (!launched) return FS_ERR_CUDA;
  if (blocks > 0) gamma_sum_kernel<<<(dim + 31) / 32, 256, 0, st>>>(part, blocks, dim, dgamma);
  count_launch(blocks > 0 ? 2 : 1);
  return launch_status();
}
