// Rows of bf16 or fp32 in vectors of 8, at any element alignment, and sums
// over a workgroup: shared by the kernels that keep a row in registers.
#pragma once

#include <type_traits>

#include "ffn.h"

namespace tgemm {

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 8 elements from column c of a row of n (zeros past the end).  The end of a row
// is read as its last 8 elements, one load as elsewhere, and moved down: loaded
// one by one, each would wait for the one before.
__device__ __forceinline__ u16x8_any load8(const uint16_t* p, int64_t c, int64_t n) {
  u16x8_any v = {{0, 0, 0, 0}};
  if (c + 8 <= n) {
    v = *reinterpret_cast<const u16x8_any*>(p + c);
  } else if (c < n && n >= 8) {
    v = *reinterpret_cast<const u16x8_any*>(p + n - 8);
    const int s = 16 * (int)(c + 8 - n);  // bits, 16 to 112
    const uint64_t lo = v.w[0] | ((uint64_t)v.w[1] << 32), hi = v.w[2] | ((uint64_t)v.w[3] << 32);
    const uint64_t l = s < 64 ? (lo >> s) | (hi << (64 - s)) : hi >> (s - 64);
    const uint64_t h = s < 64 ? hi >> s : 0;
    v = u16x8_any{{(uint32_t)l, (uint32_t)(l >> 32), (uint32_t)h, (uint32_t)(h >> 32)}};
  } else if (c < n) {  // (a row of less than 8)
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < n) v.w[i >> 1] |= (uint32_t)p[c + i] << (16 * (i & 1));
  }
  return v;
}

__device__ __forceinline__ void store8(uint16_t* p, int64_t c, int64_t n, const u16x8_any& v) {
  if (c + 8 <= n) {
    *reinterpret_cast<u16x8_any*>(p + c) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) p[c + i] = (uint16_t)(v.w[i >> 1] >> ((i & 1) * 16));
  }
}

struct f32x8_any {
  x4_any<float> a, b;
};

__device__ __forceinline__ f32x8_any load8(const float* p, int64_t c, int64_t n) {
  f32x8_any v = {};
  if (c + 8 <= n) {
    v.a = *reinterpret_cast<const x4_any<float>*>(p + c);
    v.b = *reinterpret_cast<const x4_any<float>*>(p + c + 4);
  } else if (c < n && n >= 8) {
    v.a = *reinterpret_cast<const x4_any<float>*>(p + n - 8);
    v.b = *reinterpret_cast<const x4_any<float>*>(p + n - 4);
    const int s = (int)(c + 8 - n);  // elements, 1 to 7
    float f[8] = {v.a.v[0], v.a.v[1], v.a.v[2], v.a.v[3], v.b.v[0], v.b.v[1], v.b.v[2], v.b.v[3]};
#pragma unroll
    for (int m = 1; m < 8; m *= 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = (s & m) ? (i + m < 8 ? f[i + m] : 0.f) : f[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v.a.v[i] = f[i], v.b.v[i] = f[4 + i];
  } else if (c < n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c + i < n) v.a.v[i] = p[c + i];
      if (c + 4 + i < n) v.b.v[i] = p[c + 4 + i];
    }
  }
  return v;
}

// The value i (a constant after unrolling) of such a vector.
__device__ __forceinline__ float value(const u16x8_any& v, int i) {
  return (i & 1) ? hi_f(v.w[i >> 1]) : lo_f(v.w[i >> 1]);
}
__device__ __forceinline__ float value(const f32x8_any& v, int i) {
  return i < 4 ? v.a.v[i & 3] : v.b.v[i & 3];
}

// 8 fp32 values to a row of either type.
__device__ __forceinline__ void put8(uint16_t* p, int64_t c, int64_t n, const float (&f)[8]) {
  u16x8_any v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v.w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  store8(p, c, n, v);
}
__device__ __forceinline__ void put8(float* p, int64_t c, int64_t n, const float (&f)[8]) {
  if (c + 8 <= n) {
    *reinterpret_cast<x4_any<float>*>(p + c) = x4_any<float>{{f[0], f[1], f[2], f[3]}};
    *reinterpret_cast<x4_any<float>*>(p + c + 4) = x4_any<float>{{f[4], f[5], f[6], f[7]}};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) p[c + i] = f[i];
  }
}

// The type a row of T is held in.
template <class T>
struct Vec8;
template <>
struct Vec8<uint16_t> {
  typedef u16x8_any type;
};
template <>
struct Vec8<float> {
  typedef f32x8_any type;
};

// The sum over a wave, in every lane, without the LDS that shuffles go
// through: within rows of 16 lanes, then across them to the last lane.
__device__ __forceinline__ float wave_sum(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
  auto moved = [](float x, auto ctrl, auto rows) __attribute__((always_inline)) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value,
                                                      decltype(rows)::value, 0xf, false));
  };
  using std::integral_constant;
  v += moved(v, integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});  // row_shr 1
  v += moved(v, integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});  // 2
  v += moved(v, integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});  // 4
  v += moved(v, integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});  // 8
  v += moved(v, integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});  // row_bcast 15
  v += moved(v, integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});  // row_bcast 31
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
#else
  return v;
#endif
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sums of N values each over the workgroup, in wave order (the same in every
// thread).  `buf`: LDS for the waves' sums, not to be in use by another wave:
// callers in a loop alternate between two.
template <int N, class T>
__device__ __forceinline__ void group_sum(T (&v)[N], T (*buf)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  const int waves = (int)blockDim.x >> 6;
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[threadIdx.x >> 6][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = buf[0][i];
  for (int w = 1; w < waves; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += buf[w][i];
}

}  // namespace tgemm
