// Device helpers of the convolution and the norm: VEC elements at a time, and sums of
// partial rows.
#pragma once
#include "gdn_device.h"

namespace gdn {

// 1 / (1 + exp(-z)) for tensors of type E.  bf16: from the hardware's exp2 and reciprocal (an
// ulp each; the argument's rounding adds |z| 2^-24, far below the result's own): expf and a
// division would make a SiLU the most of a memory-bound kernel's instructions.  fp32: expf
// and a division, since |z| 2^-24 of it is |z| half steps of the result.
template <typename E>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(E) == 2)
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
  else
    return 1.f / (1.f + expf(-z));
}

// VEC elements as they are in memory: loaded long before they are converted.
template <typename E, int VEC>
struct Raw {
  E e[VEC];
  __device__ __forceinline__ void load(const E* p) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = p[i];
  }
  __device__ __forceinline__ float operator[](int i) const { return to_f32(e[i]); }
};
template <int VEC>
struct Raw<bf16, VEC> {
  static constexpr int NW = VEC > 1 ? VEC / 2 : 1;
  uint32_t w[NW];
  __device__ __forceinline__ void load(const bf16* p) {
    if constexpr (VEC == 8) {
      const u32x4 r = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = r[i];
    } else if constexpr (VEC == 4) {
      const uint2 r = *reinterpret_cast<const uint2*>(p);
      w[0] = r.x;
      w[1] = r.y;
    } else if constexpr (VEC == 2) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      static_assert(VEC == 1, "8, 4, 2 or 1 elements");
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};
template <>
struct Raw<float, 2> {
  float2 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ float operator[](int i) const { return i ? v.y : v.x; }
};
template <>
struct Raw<float, 4> {
  f32x4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const f32x4*>(p); }
  __device__ __forceinline__ float operator[](int i) const { return v[i]; }
};

template <typename E, int VEC>
__device__ __forceinline__ void load_vec(const E* p, float (&v)[VEC]) {
  Raw<E, VEC> r;
  r.load(p);
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = r[i];
}
template <typename E, int VEC>
__device__ __forceinline__ void store_vec(E* p, const float (&v)[VEC]) {
  if constexpr (VEC % 2 == 0) {
    typedef E vec __attribute__((ext_vector_type(VEC)));
    vec e;
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = from_f32<E>(v[i]);
    *reinterpret_cast<vec*>(p) = e;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = from_f32<E>(v[i]);
  }
}
// VEC consecutive parameters (bf16 or fp32); VEC elements start on 16 bytes where VEC is
// a multiple of 8 (bf16) or 4 (fp32).
template <int VEC>
__device__ __forceinline__ void load_params(const void* p, int64_t i, int is_bf16, float (&v)[VEC]) {
  if (is_bf16) {
    if constexpr (VEC % 8 == 0) {
#pragma unroll
      for (int k = 0; k < VEC; k += 8) {
        float x[8];
        load_vec<bf16, 8>(reinterpret_cast<const bf16*>(p) + i + k, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k + e] = x[e];
      }
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[k] = (float)reinterpret_cast<const bf16*>(p)[i + k];
    }
  } else if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int k = 0; k < VEC; k += 4) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p) + i + k);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[k + e] = x[e];
    }
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = reinterpret_cast<const float*>(p)[i + k];
  }
}

// out[c] = sum over rows of in[r * cols + c], c in [0, cols), in a fixed order; element
// c goes to out(c).  1024 threads: 32 columns x 32 row groups.
template <typename F>
__device__ __forceinline__ void column_sums(const float* in, int64_t rows, int64_t cols, F out) {
  __shared__ float red[32][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + cx;
  float s = 0.f;
  if (c < cols) {
    float p[4] = {0.f, 0.f, 0.f, 0.f};
    int64_t r = ry;
    for (; r + 96 < rows; r += 128)
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] += in[(r + 32 * k) * cols + c];
    for (; r < rows; r += 32) p[0] += in[r * cols + c];
    s = (p[0] + p[1]) + (p[2] + p[3]);
  }
  red[ry][cx] = s;
  __syncthreads();
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    if (ry < d) red[ry][cx] += red[ry + d][cx];
    __syncthreads();
  }
  if (ry == 0 && c < cols) out(c, red[0][cx]);
}

}  // namespace gdn
