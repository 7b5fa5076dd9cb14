// Scaled embedding lookup: out[p, :] = scale * table[ids[p], :], computed in
// fp32 and rounded once to the output's type.  The sequence model that reads
// the gathered rows (FreeScale, arXiv 2604.24073, §2.1: an ID list becomes a
// sequence of embeddings) often wants them in another type and multiplied by
// a constant (sqrt(dim) for tied input and output embeddings); done here it
// costs no second pass over the [T, dim] output.
#include "convert.cuh"
#include "fs_common.cuh"

namespace fs {
namespace {

constexpr int kLookupThreads = 256;

// 32 / LPR rows per warp instruction (LPR lanes a row, VEC elements a lane),
// U rows in flight per lane, held as loaded; the next iteration's IDs are
// loaded before this iteration's rows.  Rows of more than LPR * VEC elements
// take several steps.
// Bound by HBM: 8 B of ID, one table row (distinct rows once, the others from
// L2) and one output row per position.  2M Zipf IDs over 10M rows of 128 bf16:
// 119 us, 5.7 TB/s of those bytes.  257 IDs: 3 us, two dependent reads.
template <class EI, class EO, int VEC, int LPR>
__global__ void __launch_bounds__(kLookupThreads, 3) lookup_kernel(const void* __restrict__ table, int64_t R, int32_t dim,
                                                                   const int64_t* __restrict__ ids, int64_t T,
                                                                   float scale, void* __restrict__ out, int32_t* err) {
  constexpr int RPI = 32 / LPR;
  constexpr int U = RPI * 8 <= 32 ? 8 : 32 / RPI;
  constexpr int RPW = RPI * U;
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, c0 = (lane % LPR) * VEC;
  const int64_t nwarps = (int64_t(gridDim.x) * blockDim.x) >> 5;
  const int64_t stride = nwarps * RPW;
  int64_t p0 = ((int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5) * RPW;
  auto load_id = [&](int64_t p) { return (lane < RPW && p + lane < T) ? __ldcs(ids + p + lane) : int64_t(-1); };
  int64_t next = load_id(p0);
  for (; p0 < T; p0 += stride) {
    int64_t id = next;
    next = load_id(p0 + stride);
    if (uint64_t(id) >= uint64_t(R)) {
      if (lane < RPW && p0 + lane < T) set_err(err, FS_ERR_ID_RANGE);
      id = -1;  // a row of zeros
    }
    for (int c = c0; c - c0 < dim; c += LPR * VEC) {  // (the same steps for every lane: the shuffles need them all)
      Raw<EI, VEC> r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = __shfl_sync(0xffffffffu, id, u * RPI + sub);
        memset(&r[u], 0, sizeof(r[u]));
        if (row >= 0 && c < dim) fetch<false>(r[u], table, row * dim + c);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t p = p0 + u * RPI + sub;
        if (p < T && c < dim) {
          float x[VEC];
          unpack(r[u], x);
#pragma unroll
          for (int k = 0; k < VEC; ++k) x[k] *= scale;
          store_vec<EO, VEC, true>(out, p * dim + c, x);
        }
      }
    }
  }
}

template <class EI, class EO, int VEC>
void launch_lookup(const void* table, int64_t R, int32_t dim, const int64_t* ids, int64_t T, float scale, void* out,
                   int32_t* err, cudaStream_t st) {
  const int chunks = (dim + VEC - 1) / VEC;
  auto go = [&](auto kern, int lpr) {
    const int rpi = 32 / lpr;
    const int64_t rows = int64_t(rpi * 8 <= 32 ? rpi * 8 : 32) * (kLookupThreads / 32);
    const int64_t want = (T + rows - 1) / rows, most = int64_t(sm_count()) * (2048 / kLookupThreads);
    kern<<<unsigned(want < most ? want : most), kLookupThreads, 0, st>>>(table, R, dim, ids, T, scale, out, err);
  };
  if (chunks <= 4) go(lookup_kernel<EI, EO, VEC, 4>, 4);
  else if (chunks <= 8) go(lookup_kernel<EI, EO, VEC, 8>, 8);
  else if (chunks <= 16) go(lookup_kernel<EI, EO, VEC, 16>, 16);
  else go(lookup_kernel<EI, EO, VEC, 32>, 32);
}

}  // namespace
}  // namespace fs

using namespace fs;

extern "C" fs_status fs_emb_lookup_scaled(const void* table, int64_t num_rows, int32_t dim, fs_dtype table_dtype,
                                          const int64_t* ids, int64_t T, float scale, void* out, fs_dtype out_dtype,
                                          int32_t* err, fs_stream_t stream) {
  FS_NVTX_RANGE();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T < 0 || T > INT32_MAX || num_rows < 1 || dim < 1 || !err) return FS_ERR_INVALID_ARG;
  if ((table_dtype != FS_F32 && table_dtype != FS_BF16) || (out_dtype != FS_F32 && out_dtype != FS_BF16))
    return FS_ERR_INVALID_ARG;
  if (T == 0) return FS_OK;
  if (!table || !ids || !out) return FS_ERR_INVALID_ARG;
  const size_t ib = table_dtype == FS_F32 ? 4 : 2, ob = out_dtype == FS_F32 ? 4 : 2;
  if (!aligned(table, ib) || !aligned(out, ob) || !aligned(ids, 8)) return FS_ERR_ALIGNMENT;
  // 16 bytes a lane on the wider side (8 elements bf16 to bf16, else 4); rows
  // or addresses that do not allow it move element by element
  const int vec = (ib == 2 && ob == 2) ? 8 : 4;
  const bool wide = dim % vec == 0 && aligned(table, vec * ib) && aligned(out, vec * ob);
#define FS_LOOKUP(EI, EO, V) \
  (wide ? launch_lookup<EI, EO, V>(table, num_rows, dim, ids, T, scale, out, err, st) \
        : launch_lookup<EI, EO, 1>(table, num_rows, dim, ids, T, scale, out, err, st))
  if (ib == 4 && ob == 4) FS_LOOKUP(F32, F32, 4);
  else if (ib == 4) FS_LOOKUP(F32, Bf16, 4);
  else if (ob == 4) FS_LOOKUP(Bf16, F32, 4);
  else FS_LOOKUP(Bf16, Bf16, 8);
#undef FS_LOOKUP
  count_launch(1);
  return launch_status();
}
