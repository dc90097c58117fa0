// The row products' side passes: the sum of K chunks with its epilogue, the
// copy of an operand into the layout the products read, and the gated
// product's gradient.  All are bound by HBM bandwidth: each element is read
// and written once, 8 or 4 per thread.
#include "bf16_cvt.h"
#include "ffn.h"

#include <type_traits>

namespace tgemm {
namespace {

constexpr int kThr = 256;

template <class T>
struct __attribute__((packed, aligned(4))) x4_any {
  T v[4];
};

// n (1 to 4) values as bf16 / fp32 at any element alignment.
__device__ __forceinline__ void put4(uint16_t* o, const float* v, int n) {
  if (n == 4) {
    u16x4_any w;
    w.w[0] = pack_bf16x2(v[0], v[1]);
    w.w[1] = pack_bf16x2(v[2], v[3]);
    *reinterpret_cast<u16x4_any*>(o) = w;
  } else {
    for (int i = 0; i < n; ++i) o[i] = to_bf16(v[i]);
  }
}
__device__ __forceinline__ void put4(float* o, const float* v, int n) {
  if (n == 4) {
    *reinterpret_cast<x4_any<float>*>(o) = x4_any<float>{{v[0], v[1], v[2], v[3]}};
  } else {
    for (int i = 0; i < n; ++i) o[i] = v[i];
  }
}
template <class T>
__device__ __forceinline__ void add4(T* a, const T* p, int n) {
  if (n == 4) {
    const x4_any<T> t = *reinterpret_cast<const x4_any<T>*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] += t.v[i];
  } else {
    for (int i = 0; i < n; ++i) a[i] += p[i];
  }
}

// out = epilogue(sum over chunks, in ascending order), four consecutive
// outputs per thread.  Partials [split][M][N] (gated: N = 2F, outputs
// [M][F]).
template <class T, int EPI>
__global__ void __launch_bounds__(kThr) finish_kernel(RowsParams p) {
  constexpr bool I8 = std::is_same<T, int>::value;
  constexpr bool GATE = EPI == kRowsGated;
  const int nout = GATE ? p.F : p.N;
  const int per_row = (nout + 4 * kThr - 1) / (4 * kThr);
  const int row = (int)(blockIdx.x / per_row);
  const int c = ((int)(blockIdx.x % per_row) * kThr + (int)threadIdx.x) * 4;
  if (c >= nout) return;
  const int n = min(4, nout - c);
  const T* part = static_cast<const T*>(p.part) + (int64_t)row * p.N + c;
  const int64_t slice = (int64_t)p.M * p.N;
  T a[4] = {0, 0, 0, 0}, a2[4] = {0, 0, 0, 0};
  for (int q = 0; q < p.split; ++q) {
    add4(a, part + q * slice, n);
    if constexpr (GATE) add4(a2, part + q * slice + p.F, n);
  }
  float v[4], u[4], h[4];
  const float sa = I8 ? p.scale_a[row] : 1.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = (float)a[i];
    u[i] = (float)a2[i];
    if constexpr (I8) {
      const int ci = min(c + i, nout - 1);
      v[i] = v[i] * sa * p.scale_b[ci];
      if constexpr (GATE) u[i] = u[i] * sa * p.scale_b[p.F + ci];
    }
    h[i] = GATE ? act_value(v[i], p.act) * u[i] : v[i];
  }
  const int64_t o = (int64_t)row * p.ldc + c;
  if constexpr (EPI == kRowsStoreF32)
    put4(static_cast<float*>(p.C) + o, h, n);
  else
    put4(static_cast<uint16_t*>(p.C) + o, h, n);
  if constexpr (GATE && !I8) {
    if (p.gu != nullptr) {
      uint16_t* const w = p.gu + (int64_t)row * p.ldgu + c;
      put4(w, v, n);
      put4(w + p.F, u, n);
    }
  }
}

// Copy a K-contiguous operand: 16 output bytes per thread, from any
// alignment.  ES: bytes per element.
template <int ES>
__global__ void __launch_bounds__(kThr) pack_rows_kernel(PackRows p, int chunks) {
  const int64_t t = (int64_t)blockIdx.x * kThr + threadIdx.x;
  const int r = (int)(t / chunks), k = (int)(t - (int64_t)r * chunks) * (16 / ES);
  if (r >= p.Rz) return;
  b16_any v = {{0, 0, 0, 0}};
  if (r < p.R && k < p.K) {
    const char* src = static_cast<const char*>(p.X) + ((int64_t)r * p.ld + k) * ES;
    if (k + 16 / ES <= p.K) {
      v = *reinterpret_cast<const b16_any*>(src);
    } else {
      for (int i = 0; i < (p.K - k) * ES; ++i)
        v.w[i >> 2] |= (uint32_t)(uint8_t)src[i] << ((i & 3) * 8);
    }
  }
  *reinterpret_cast<b16_any*>(static_cast<char*>(p.out) + ((int64_t)r * p.ldo + k) * ES) = v;
}

// Copy an operand stored [K][R] into rows of K: 64 x 64 elements per
// workgroup, read 16 bytes along R, turned around in LDS (rows of 64 + 16 /
// ES elements, a multiple of 16 bytes) and written 16 bytes along K.
template <int ES>
__global__ void __launch_bounds__(kThr) pack_cols_kernel(PackRows p, int kblocks) {
  using E = std::conditional_t<ES == 1, uint8_t, uint16_t>;
  constexpr int V = 16 / ES, LD = 64 + V, NV = 64 * 64 / V;  // elements per vector, vectors
  __shared__ __attribute__((aligned(16))) E t[64 * LD];
  const int k0 = (int)(blockIdx.x % kblocks) * 64, r0 = (int)(blockIdx.x / kblocks) * 64;
  for (int i = threadIdx.x; i < NV; i += kThr) {
    const int kl = i / (64 / V), rl = (i % (64 / V)) * V;
    const int k = k0 + kl, r = r0 + rl;
    b16_any v = {{0, 0, 0, 0}};
    if (k < p.K && r < p.R) {
      const char* src = static_cast<const char*>(p.X) + ((int64_t)k * p.ld + r) * ES;
      if (r + V <= p.R) {
        v = *reinterpret_cast<const b16_any*>(src);
      } else {
        for (int e = 0; e < (p.R - r) * ES; ++e)
          v.w[e >> 2] |= (uint32_t)(uint8_t)src[e] << ((e & 3) * 8);
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
      t[(rl + e) * LD + kl] = (E)(v.w[e * ES >> 2] >> ((e * ES & 3) * 8));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < NV; i += kThr) {
    const int rl = i / (64 / V), kl = (i % (64 / V)) * V;
    const int r = r0 + rl, k = k0 + kl;
    // (ldo holds whole vectors)
    if (r < p.Rz && k < p.ldo)
      *reinterpret_cast<uint4*>(static_cast<char*>(p.out) + ((int64_t)r * p.ldo + k) * ES) =
          *reinterpret_cast<const uint4*>(t + rl * LD + kl);
  }
}

__device__ __forceinline__ void grad_pair(uint32_t dh, uint32_t g, uint32_t u, int act,
                                          uint32_t& dg, uint32_t& du) {
  float a[2], d[2], x[2], y[2];
  act_value_grad(__uint_as_float(g << 16), act, a[0], d[0]);
  act_value_grad(__uint_as_float(g & 0xffff0000u), act, a[1], d[1]);
  const float h[2] = {__uint_as_float(dh << 16), __uint_as_float(dh & 0xffff0000u)};
  const float v[2] = {__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[i] = h[i] * v[i] * d[i];
    y[i] = h[i] * a[i];
  }
  dg = pack_bf16x2(x[0], x[1]);
  du = pack_bf16x2(y[0], y[1]);
}

// 8 outputs per thread; the arithmetic is fp32, dg and du are rounded once
// to bf16, the type the gradient products read.  The padding (columns 2F ..
// cols - 1, rows past M) is written by the threads whose chunk lies past F
// and by the workgroups of rows past M.
__global__ void __launch_bounds__(kThr) gated_grad_kernel(
    const uint16_t* __restrict__ dh, int64_t lddh, const uint16_t* __restrict__ gu, int64_t ldgu,
    int M, int64_t F, int act, uint16_t* __restrict__ dgu, int64_t lddgu, int64_t cols,
    int64_t per_row) {
  const int64_t row = blockIdx.x / per_row;
  const int64_t c = ((int64_t)(blockIdx.x % per_row) * kThr + threadIdx.x) * 8;
  uint16_t* const out = dgu + row * lddgu;
  if (row >= M) {
    for (int64_t i = c; i < c + 8 && i < F; ++i) out[i] = out[F + i] = 0;
    for (int64_t i = 2 * F + c; i < 2 * F + c + 8 && i < cols; ++i) out[i] = 0;
    return;
  }
  for (int64_t i = 2 * F + c; i < 2 * F + c + 8 && i < cols; ++i) out[i] = 0;
  if (c >= F) return;
  const uint16_t* ph = dh + row * lddh + c;
  const uint16_t* pg = gu + row * ldgu + c;
  uint16_t* po = out + c;
  if (c + 8 <= F) {
    const u16x8_any h = *reinterpret_cast<const u16x8_any*>(ph);
    const u16x8_any g = *reinterpret_cast<const u16x8_any*>(pg);
    const u16x8_any u = *reinterpret_cast<const u16x8_any*>(pg + F);
    u16x8_any x, y;
#pragma unroll
    for (int i = 0; i < 4; ++i) grad_pair(h.w[i], g.w[i], u.w[i], act, x.w[i], y.w[i]);
    *reinterpret_cast<u16x8_any*>(po) = x;
    *reinterpret_cast<u16x8_any*>(po + F) = y;
  } else {
    for (int64_t i = 0; c + i < F; ++i) {
      uint32_t x, y;
      grad_pair(ph[i], pg[i], pg[F + i], act, x, y);
      po[i] = (uint16_t)x;
      po[F + i] = (uint16_t)y;
    }
  }
}

template <class T, int EPI>
hipError_t finish_one(const RowsParams& p, hipStream_t s) {
  const int64_t blocks = (int64_t)p.M * ceil_div(EPI == kRowsGated ? p.F : p.N, 4 * kThr);
  if (blocks > kMaxWorkgroups) return hipErrorInvalidValue;
  hipLaunchKernelGGL((finish_kernel<T, EPI>), dim3((unsigned)blocks), dim3(kThr), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rows_finish(int type, int epi, const RowsParams& p, hipStream_t s) {
  if (type == kRowsI8) {
    if (epi == kRowsStoreBf16) return finish_one<int, kRowsStoreBf16>(p, s);
    if (epi == kRowsStoreF32) return finish_one<int, kRowsStoreF32>(p, s);
    if (epi == kRowsGated) return finish_one<int, kRowsGated>(p, s);
  } else if (epi == kRowsGated) {
    return finish_one<float, kRowsGated>(p, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_pack_rows(const PackRows& p, int elem, hipStream_t s) {
  if (p.k_contiguous) {
    const int chunks = (int)(p.ldo * elem / 16);
    const int64_t blocks = ((int64_t)p.Rz * chunks + kThr - 1) / kThr;
    if (blocks > kMaxWorkgroups) return hipErrorInvalidValue;
    if (elem == 1)
      hipLaunchKernelGGL(pack_rows_kernel<1>, dim3((unsigned)blocks), dim3(kThr), 0, s, p, chunks);
    else
      hipLaunchKernelGGL(pack_rows_kernel<2>, dim3((unsigned)blocks), dim3(kThr), 0, s, p, chunks);
  } else {
    const int kblocks = ceil_div(p.ldo, 64);
    const int64_t blocks = (int64_t)kblocks * ceil_div(p.Rz, 64);
    if (blocks > kMaxWorkgroups) return hipErrorInvalidValue;
    if (elem == 1)
      hipLaunchKernelGGL(pack_cols_kernel<1>, dim3((unsigned)blocks), dim3(kThr), 0, s, p, kblocks);
    else
      hipLaunchKernelGGL(pack_cols_kernel<2>, dim3((unsigned)blocks), dim3(kThr), 0, s, p, kblocks);
  }
  return hipGetLastError();
}

hipError_t launch_gated_grad(const uint16_t* dh, int64_t lddh, const uint16_t* gu, int64_t ldgu,
                             int M, int64_t F, int act, uint16_t* dgu, int64_t lddgu, int rows,
                             int64_t cols, hipStream_t s) {
  // (the padding of a row, cols - 2F < 64 elements, needs at most 8 threads)
  const int64_t chunks = (F + 7) / 8 > 8 ? (F + 7) / 8 : 8;
  const int64_t per_row = (chunks + kThr - 1) / kThr;
  if (rows * per_row > kMaxWorkgroups) return hipErrorInvalidValue;
  hipLaunchKernelGGL(gated_grad_kernel, dim3((unsigned)(rows * per_row)), dim3(kThr), 0, s, dh,
                     lddh, gu, ldgu, M, F, act, dgu, lddgu, cols, per_row);
  return hipGetLastError();
}

}  // namespace tgemm
