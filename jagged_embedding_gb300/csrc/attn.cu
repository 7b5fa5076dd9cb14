// Attention inside each sample of a jagged batch, and its backward pass.
// Row i of a sample of L positions, the last `cand` of them candidates, sees
// key j iff (j <= i or not causal) and (j < L - cand or j == i).
//   s = scale * q.k,  lse = log sum_j exp(s_j),  o = sum_j exp(s_j - lse) v_j
// backward, recomputing p = exp(s - lse):
//   delta = do.o,  ds = p * (do.v - delta)
//   dq = scale * sum_j ds k_j,  dk = scale * sum_i ds q_i,  dv = sum_i p do_i
#include "convert.cuh"
#include "fs_common.cuh"

namespace fs {
namespace {

struct AttnArgs {
  const __nv_bfloat16 *q, *k, *v, *out, *dout;
  int64_t q_stride, k_stride, v_stride;
  __nv_bfloat16 *o, *dq, *dk, *dv;
  int64_t dq_stride, dk_stride, dv_stride;
  const int64_t* offsets;
  int64_t S, T;
  int32_t Hq, Hkv;
  const int32_t* cand;
  int32_t causal;
  float scale;
  float* lse;
  int32_t* err;
};

struct Sample {
  int64_t begin;
  int32_t L, uih;
};

// Sample of position t (binary search; L = 0 where t belongs to none).
__device__ Sample sample_of(const AttnArgs& a, int64_t t) {
  int64_t lo = 0, hi = a.S;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (a.offsets[mid + 1] <= t) lo = mid + 1; else hi = mid;
  }
  if (lo >= a.S || a.offsets[lo] > t || a.offsets[lo] < 0 || a.offsets[lo + 1] > a.T) return {0, 0, 0};
  const int64_t b = a.offsets[lo];
  const int32_t L = int32_t(a.offsets[lo + 1] - b);
  int32_t c = a.cand ? a.cand[lo] : 0;
  c = c < 0 ? 0 : (c > L ? L : c);
  return {b, L, L - c};
}

// Offsets and candidate counts are checked once for the whole call.
__global__ void attn_check_kernel(AttnArgs a) {
  const int64_t s = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (s >= a.S) return;
  const int64_t b = a.offsets[s], e = a.offsets[s + 1];
  if (b < 0 || e < b || e > a.T) {
    set_err(a.err, FS_ERR_BAD_OFFSETS);
    return;
  }
  const int32_t c = a.cand ? a.cand[s] : 0;
  if (c < 0 || c > e - b) set_err(a.err, FS_ERR_INVALID_ARG);
}

template <int E>
__device__ __forceinline__ void row(const __nv_bfloat16* p, int lane, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = __bfloat162float(p[lane + 32 * i]);
}

template <int E>
__device__ __forceinline__ float dot(const float (&x)[E], const float (&y)[E]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) s = fmaf(x[i], y[i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__device__ __forceinline__ bool sees(const AttnArgs& a, const Sample& s, int i, int j) {
  return (j <= i || !a.causal) && (j < s.uih || j == i);
}

// One warp per position and query head; E = head_dim / 32 elements a lane.
template <int E>
__global__ void attn_fwd_kernel(AttnArgs a) {
  const int64_t w = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t t = w / a.Hq;
  const int h = int(w % a.Hq), hk = h * a.Hkv / a.Hq;
  if (t >= a.T) return;
  const Sample s = sample_of(a, t);
  if (s.L == 0) return;
  const int i = int(t - s.begin);
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
  row<E>(a.q + t * a.q_stride + h * 32 * E, lane, q);
  for (int j = 0; j < s.L; ++j) {
    if (!sees(a, s, i, j)) continue;
    float k[E], v[E];
    row<E>(a.k + (s.begin + j) * a.k_stride + hk * 32 * E, lane, k);
    row<E>(a.v + (s.begin + j) * a.v_stride + hk * 32 * E, lane, v);
    const float x = dot<E>(q, k) * a.scale, mn = fmaxf(m, x);
    const float f = expf(m - mn), p = expf(x - mn);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * v[e];
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) a.o[(t * a.Hq + h) * 32 * E + lane + 32 * e] = __float2bfloat16_rn(o[e] / l);
  if (lane == 0) a.lse[int64_t(h) * a.T + t] = m + logf(l);
}

template <int E>
__global__ void attn_dq_kernel(AttnArgs a) {
  const int64_t w = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t t = w / a.Hq;
  const int h = int(w % a.Hq), hk = h * a.Hkv / a.Hq;
  if (t >= a.T) return;
  const Sample s = sample_of(a, t);
  if (s.L == 0) return;
  const int i = int(t - s.begin);
  float q[E], o[E], g[E], d[E] = {};
  row<E>(a.q + t * a.q_stride + h * 32 * E, lane, q);
  row<E>(a.out + (t * a.Hq + h) * 32 * E, lane, o);
  row<E>(a.dout + (t * a.Hq + h) * 32 * E, lane, g);
  const float delta = dot<E>(o, g), lse = a.lse[int64_t(h) * a.T + t];
  for (int j = 0; j < s.L; ++j) {
    if (!sees(a, s, i, j)) continue;
    float k[E], v[E];
    row<E>(a.k + (s.begin + j) * a.k_stride + hk * 32 * E, lane, k);
    row<E>(a.v + (s.begin + j) * a.v_stride + hk * 32 * E, lane, v);
    const float p = expf(dot<E>(q, k) * a.scale - lse);
    const float ds = p * (dot<E>(g, v) - delta) * a.scale;
#pragma unroll
    for (int e = 0; e < E; ++e) d[e] = fmaf(ds, k[e], d[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) a.dq[t * a.dq_stride + h * 32 * E + lane + 32 * e] = __float2bfloat16_rn(d[e]);
}

// One warp per position and key/value head, over the query heads that share it.
template <int E>
__global__ void attn_dkv_kernel(AttnArgs a) {
  const int64_t w = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t t = w / a.Hkv;
  const int hk = int(w % a.Hkv), G = a.Hq / a.Hkv;
  if (t >= a.T) return;
  const Sample s = sample_of(a, t);
  if (s.L == 0) return;
  const int j = int(t - s.begin);
  float k[E], v[E], dk[E] = {}, dv[E] = {};
  row<E>(a.k + t * a.k_stride + hk * 32 * E, lane, k);
  row<E>(a.v + t * a.v_stride + hk * 32 * E, lane, v);
  for (int h = hk * G; h < (hk + 1) * G; ++h)
    for (int i = 0; i < s.L; ++i) {
      if (!sees(a, s, i, j)) continue;
      const int64_t r = s.begin + i;
      float q[E], o[E], g[E];
      row<E>(a.q + r * a.q_stride + h * 32 * E, lane, q);
      row<E>(a.out + (r * a.Hq + h) * 32 * E, lane, o);
      row<E>(a.dout + (r * a.Hq + h) * 32 * E, lane, g);
      const float p = expf(dot<E>(q, k) * a.scale - a.lse[int64_t(h) * a.T + r]);
      const float ds = p * (dot<E>(g, v) - dot<E>(g, o)) * a.scale;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        dk[e] = fmaf(ds, q[e], dk[e]);
        dv[e] = fmaf(p, g[e], dv[e]);
      }
    }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    a.dk[t * a.dk_stride + hk * 32 * E + lane + 32 * e] = __float2bfloat16_rn(dk[e]);
    a.dv[t * a.dv_stride + hk * 32 * E + lane + 32 * e] = __float2bfloat16_rn(dv[e]);
  }
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

unsigned warps_grid(int64_t warps) { return unsigned((warps + 3) / 4); }

}  // namespace
}  // namespace fs

using namespace fs;

extern "C" size_t fs_jagged_attn_workspace_size(int64_t T, int64_t S, int32_t heads, int32_t kv_heads,
                                                int32_t head_dim) {
  if (T < 0 || S < 0 || heads < 1 || kv_heads < 1 || (head_dim != 64 && head_dim != 128)) return 0;
  return 256;
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
  AttnArgs a{};
  using B = __nv_bfloat16;
  a.q = static_cast<const B*>(q), a.k = static_cast<const B*>(k), a.v = static_cast<const B*>(v);
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.o = static_cast<B*>(out);
  a.offsets = offsets, a.S = S, a.T = T, a.Hq = heads, a.Hkv = kv_heads, a.cand = cand_len, a.causal = causal;
  a.scale = scale, a.lse = lse, a.err = err;
  attn_check_kernel<<<unsigned((S + 127) / 128), 128, 0, st>>>(a);
  if (head_dim == 64) attn_fwd_kernel<2><<<warps_grid(T * heads), 128, 0, st>>>(a);
  else attn_fwd_kernel<4><<<warps_grid(T * heads), 128, 0, st>>>(a);
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
  const int64_t ow = int64_t(heads) * head_dim;
  if ((s = check_rows(q, q_stride, heads, head_dim)) != FS_OK || (s = check_rows(k, k_stride, kv_heads, head_dim)) != FS_OK ||
      (s = check_rows(v, v_stride, kv_heads, head_dim)) != FS_OK || (s = check_rows(out, ow, heads, head_dim)) != FS_OK ||
      (s = check_rows(dout, ow, heads, head_dim)) != FS_OK || (s = check_rows(dq, dq_stride, heads, head_dim)) != FS_OK ||
      (s = check_rows(dk, dk_stride, kv_heads, head_dim)) != FS_OK ||
      (s = check_rows(dv, dv_stride, kv_heads, head_dim)) != FS_OK)
    return s;
  if (!ws || ws_bytes < fs_jagged_attn_workspace_size(T, S, heads, kv_heads, head_dim)) return FS_ERR_WORKSPACE;
  AttnArgs a{};
  using B = __nv_bfloat16;
  a.q = static_cast<const B*>(q), a.k = static_cast<const B*>(k), a.v = static_cast<const B*>(v);
  a.out = static_cast<const B*>(out), a.dout = static_cast<const B*>(dout);
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.dq = static_cast<B*>(dq), a.dk = static_cast<B*>(dk), a.dv = static_cast<B*>(dv);
  a.dq_stride = dq_stride, a.dk_stride = dk_stride, a.dv_stride = dv_stride;
  a.offsets = offsets, a.S = S, a.T = T, a.Hq = heads, a.Hkv = kv_heads, a.cand = cand_len, a.causal = causal;
  a.scale = scale, a.lse = const_cast<float*>(lse), a.err = err;
  attn_check_kernel<<<unsigned((S + 127) / 128), 128, 0, st>>>(a);
  if (head_dim == 64) {
    attn_dq_kernel<2><<<warps_grid(T * heads), 128, 0, st>>>(a);
    attn_dkv_kernel<2><<<warps_grid(T * kv_heads), 128, 0, st>>>(a);
  } else {
    attn_dq_kernel<4><<<warps_grid(T * heads), 128, 0, st>>>(a);
    attn_dkv_kernel<4><<<warps_grid(T * kv_heads), 128, 0, st>>>(a);
  }
  count_launch(3);
  return launch_status();
}
