// The row products' side passes: the sum of K chunks with its epilogue, the
// copy of an int8 operand into the layout the products read, and the gated
// product's gradient.  All are bound by HBM bandwidth: each element is read
// and written once, 8 or 4 per thread.
#include "bf16_cvt.h"
#include "ffn.h"

namespace tgemm {
namespace {

constexpr int kThr = 256;

// out = epilogue(sum over chunks, in ascending order), one thread per
// output.  Partials [split][M][N] (gated: N = 2F, outputs [M][F]).
template <class T, int EPI>
__global__ void __launch_bounds__(kThr) finish_kernel(RowsParams p) {
  constexpr bool I8 = std::is_same<T, int>::value;
  constexpr bool GATE = EPI == kRowsGated;
  const int nout = GATE ? p.F : p.N;
  const int64_t per_row = (nout + kThr - 1) / kThr;
  const int row = (int)(blockIdx.x / per_row);
  const int c = (int)(blockIdx.x % per_row) * kThr + (int)threadIdx.x;
  if (c >= nout) return;
  const T* part = static_cast<const T*>(p.part) + (int64_t)row * p.N + c;
  const int64_t slice = (int64_t)p.M * p.N;
  T a = part[0], a2 = GATE ? part[p.F] : T(0);
  for (int q = 1; q < p.split; ++q) {
    a += part[q * slice];
    if constexpr (GATE) a2 += part[q * slice + p.F];
  }
  float v = (float)a, u = (float)a2;
  if constexpr (I8) {
    const float sa = p.scale_a[row];
    v = v * sa * p.scale_b[c];
    if constexpr (GATE) u = u * sa * p.scale_b[p.F + c];
  }
  const int64_t o = (int64_t)row * p.ldc + c;
  if constexpr (EPI == kRowsStoreF32) {
    static_cast<float*>(p.C)[o] = v;
  } else if constexpr (EPI == kRowsStoreBf16) {
    static_cast<uint16_t*>(p.C)[o] = to_bf16(v);
  } else {
    static_cast<uint16_t*>(p.C)[o] = to_bf16(act_value(v, p.act) * u);
    if constexpr (!I8) {
      if (p.gu != nullptr) {
        p.gu[(int64_t)row * p.ldgu + c] = to_bf16(v);
        p.gu[(int64_t)row * p.ldgu + p.F + c] = to_bf16(u);
      }
    }
  }
}

// 64 x 64 bytes per workgroup.  K-contiguous operands are copied, others
// transposed through LDS (65-byte rows: the column reads hit all banks).
template <bool KC>
__global__ void __launch_bounds__(kThr) pack_i8_kernel(const int8_t* __restrict__ X, int64_t ld,
                                                       int R, int K, int8_t* __restrict__ out,
                                                       int Kp, int kblocks) {
  __shared__ int8_t t[64][65];
  const int k0 = (int)(blockIdx.x % kblocks) * 64, r0 = (int)(blockIdx.x / kblocks) * 64;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int y = ty + 4 * i;
    if constexpr (KC) {
      const int r = r0 + y, k = k0 + tx;
      if (r < R && k < Kp) out[(int64_t)r * Kp + k] = k < K ? X[(int64_t)r * ld + k] : int8_t(0);
    } else {
      const int k = k0 + y, r = r0 + tx;
      t[y][tx] = k < K && r < R ? X[(int64_t)k * ld + r] : int8_t(0);
    }
  }
  if constexpr (!KC) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = r0 + ty + 4 * i, k = k0 + tx;
      if (r < R && k < Kp) out[(int64_t)r * Kp + k] = t[tx][ty + 4 * i];
    }
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
// to bf16, the type the gradient products read.
__global__ void __launch_bounds__(kThr) gated_grad_kernel(
    const uint16_t* __restrict__ dh, int64_t lddh, const uint16_t* __restrict__ gu, int64_t ldgu,
    int64_t F, int act, uint16_t* __restrict__ dgu, int64_t lddgu, int64_t per_row) {
  const int64_t row = blockIdx.x / per_row;
  const int64_t c = ((int64_t)(blockIdx.x % per_row) * kThr + threadIdx.x) * 8;
  if (c >= F) return;
  const uint16_t* ph = dh + row * lddh + c;
  const uint16_t* pg = gu + row * ldgu + c;
  uint16_t* po = dgu + row * lddgu + c;
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
  const int64_t blocks = (int64_t)p.M * ceil_div(EPI == kRowsGated ? p.F : p.N, kThr);
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

hipError_t launch_pack_i8(const int8_t* X, int64_t ld, bool k_contiguous, int R, int K,
                          int8_t* out, int Kp, hipStream_t s) {
  const int kblocks = ceil_div(Kp, 64);
  const int64_t blocks = (int64_t)kblocks * ceil_div(R, 64);
  if (blocks > kMaxWorkgroups) return hipErrorInvalidValue;
  if (k_contiguous)
    hipLaunchKernelGGL(pack_i8_kernel<true>, dim3((unsigned)blocks), dim3(kThr), 0, s, X, ld, R, K,
                       out, Kp, kblocks);
  else
    hipLaunchKernelGGL(pack_i8_kernel<false>, dim3((unsigned)blocks), dim3(kThr), 0, s, X, ld, R,
                       K, out, Kp, kblocks);
  return hipGetLastError();
}

hipError_t launch_gated_grad(const uint16_t* dh, int64_t lddh, const uint16_t* gu, int64_t ldgu,
                             int M, int64_t F, int act, uint16_t* dgu, int64_t lddgu,
                             hipStream_t s) {
  const int64_t per_row = (F + 8 * kThr - 1) / (8 * kThr);
  if (M * per_row > kMaxWorkgroups) return hipErrorInvalidValue;
  hipLaunchKernelGGL(gated_grad_kernel, dim3((unsigned)(M * per_row)), dim3(kThr), 0, s, dh, lddh,
                     gu, ldgu, F, act, dgu, lddgu, per_row);
  return hipGetLastError();
}

}  // namespace tgemm
