// Loads and stores of VEC consecutive elements as fp32, for rows of f32 or
// bf16 (and e4m3 on the way out).  One vector access of VEC * element bytes
// (at most 16); the caller checks that the address allows it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>
#include <string.h>

namespace fs {

struct F32 {
  static constexpr int kBytes = 4;
};
struct Bf16 {
  static constexpr int kBytes = 2;
};
struct E4m3 {
  static constexpr int kBytes = 1;
};

template <int BYTES> struct Pack;
template <> struct Pack<1> { using T = unsigned char; };
template <> struct Pack<2> { using T = unsigned short; };
template <> struct Pack<4> { using T = unsigned int; };
template <> struct Pack<8> { using T = uint2; };
template <> struct Pack<16> { using T = uint4; };

// VEC elements as they lie in memory: loaded by `fetch`, widened by `unpack`.
// Kept in this form while several loads are in flight, bf16 takes half the registers.
template <class E, int VEC>
struct Raw {
  static constexpr int kBytes = E::kBytes * VEC;
  static_assert(kBytes <= 16, "one access");
  typename Pack<kBytes>::T v;
};

template <bool STREAM, class E, int VEC>
__device__ __forceinline__ void fetch(Raw<E, VEC>& r, const void* base, int64_t i) {
  using V = typename Pack<Raw<E, VEC>::kBytes>::T;
  const V* p = reinterpret_cast<const V*>(static_cast<const char*>(base) + i * E::kBytes);
  r.v = STREAM ? __ldcs(p) : __ldg(p);
}

template <class E, int VEC>
__device__ __forceinline__ void unpack(const Raw<E, VEC>& r, float (&x)[VEC]) {
  uint32_t w[(Raw<E, VEC>::kBytes + 3) / 4] = {0};
  memcpy(w, &r.v, Raw<E, VEC>::kBytes);
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    if constexpr (E::kBytes == 2) x[k] = __uint_as_float((k & 1) ? (w[k / 2] & 0xFFFF0000u) : (w[k / 2] << 16));
    else x[k] = __uint_as_float(w[k]);
  }
}

// x = elements [i, i + VEC) of `base`; STREAM: the data is read once.
template <class E, int VEC, bool STREAM>
__device__ __forceinline__ void load_vec(const void* base, int64_t i, float (&x)[VEC]) {
  Raw<E, VEC> r;
  fetch<STREAM>(r, base, i);
  unpack(r, x);
}

// Elements [i, i + VEC) of `base` = x, rounded to nearest even (e4m3: the
// values are already scaled into range; NaN stays NaN).
template <class E, int VEC, bool STREAM>
__device__ __forceinline__ void store_vec(void* base, int64_t i, const float (&x)[VEC]) {
  constexpr int B = E::kBytes * VEC;
  static_assert(B <= 16, "one access");
  using V = typename Pack<B>::T;
  uint32_t w[(B + 3) / 4] = {0};
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    if constexpr (E::kBytes == 4) {
      w[k] = __float_as_uint(x[k]);
    } else if constexpr (VEC % 2 == 0) {
      if (k & 1) continue;
      if constexpr (E::kBytes == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[k], x[k + 1]);
        memcpy(&w[k / 2], &h, 4);
      } else {
        w[k / 4] |= uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(x[k], x[k + 1]), __NV_SATFINITE, __NV_E4M3))
                    << ((k & 3) * 8);
      }
    } else if constexpr (E::kBytes == 2) {
      w[k / 2] |= uint32_t(__bfloat16_as_ushort(__float2bfloat16_rn(x[k]))) << ((k & 1) * 16);
    } else {
      w[k / 4] |= uint32_t(__nv_cvt_float_to_fp8(x[k], __NV_SATFINITE, __NV_E4M3)) << ((k & 3) * 8);
    }
  }
  V v;
  memcpy(&v, w, B);
  V* p = reinterpret_cast<V*>(static_cast<char*>(base) + i * E::kBytes);
  if (STREAM) __stcs(p, v);
  else *p = v;
}

}  // namespace fs
