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
    h[i] = GATE ? act_times(v[i], u[i], p.act) : v[i];
  }
  const int64_t o = (int64_t)row * p.ldc + c;
  if constexpr (EPI == kRowsStoreF32)
    put4(static_cast<float*>(p.C) + o, h, n);
  else
    put4(static_cast<uint16_t*>(p.C) + o, h, n);
  if constexpr (GATE && !I8) {
    if (p.gu != nullptr) {
      float* const w = p.gu + (int64_t)row * p.ldgu + c;
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

// N consecutive values of a row of bf16 or fp32 (no alignment asked for).
template <int N, class T>
__device__ __forceinline__ void load_values(const T* p, float (&v)[N]) {
  if constexpr (std::is_same<T, float>::value) {
    if constexpr (N == 8) {
      const x4_any<float> a = *reinterpret_cast<const x4_any<float>*>(p);
      const x4_any<float> b = *reinterpret_cast<const x4_any<float>*>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = a.v[i], v[4 + i] = b.v[i];
    } else {
      v[0] = p[0];
    }
  } else {
    if constexpr (N == 8) {
      const u16x8_any a = *reinterpret_cast<const u16x8_any*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a.w[i] << 16);
        v[2 * i + 1] = __uint_as_float(a.w[i] & 0xffff0000u);
      }
    } else {
      v[0] = from_bf16(p[0]);
    }
  }
}

template <int N, class T>
__device__ __forceinline__ void grad_values(const uint16_t* ph, const T* pg, int64_t F, int act,
                                            float (&x)[N], float (&y)[N]) {
  float h[N], g[N], u[N];
  load_values<N>(ph, h);
  load_values<N>(pg, g);
  load_values<N>(pg + F, u);
#pragma unroll
  for (int i = 0; i < N; ++i) act_gradients(g[i], u[i], h[i], act, x[i], y[i]);
}

// 8 outputs per thread, T the type g and u were kept in; the arithmetic is
// fp32, dg and du are rounded once to bf16, the type the gradient products
// read.  The padding (columns 2F .. cols - 1, rows past M) is written by the
// threads whose chunk lies past F and by the workgroups of rows past M.
template <class T>
__global__ void __launch_bounds__(kThr) gated_grad_kernel(
    const uint16_t* __restrict__ dh, int64_t lddh, const T* __restrict__ gu, int64_t ldgu, int M,
    int64_t F, int act, uint16_t* __restrict__ dgu, int64_t lddgu, int64_t cols, int64_t per_row) {
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
  const T* pg = gu + row * ldgu + c;
  uint16_t* po = out + c;
  if (c + 8 <= F) {
    float x[8], y[8];
    grad_values<8>(ph, pg, F, act, x, y);
    u16x8_any ox, oy;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ox.w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
      oy.w[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
    }
    *reinterpret_cast<u16x8_any*>(po) = ox;
    *reinterpret_cast<u16x8_any*>(po + F) = oy;
  } else {
    for (int64_t i = 0; c + i < F; ++i) {
      float x[1], y[1];
      grad_values<1>(ph + i, pg + i, F, act, x, y);
      po[i] = to_bf16(x[0]);
      po[F + i] = to_bf16(y[0]);
    }
  }
}

int64_t finish_blocks(const RowsParams& p, bool gate) {
  return (int64_t)p.M * ceil_div(gate ? p.F : p.N, 4 * kThr);
}

template <class T, int EPI>
hipError_t finish_one(const RowsParams& p, hipStream_t s) {
  return enqueue(finish_kernel<T, EPI>, dim3((unsigned)finish_blocks(p, EPI == kRowsGated)),
                 dim3(kThr), s, p);
}

}  // namespace

bool rows_finish_fits(const RowsParams& p, bool gate) {
  return finish_blocks(p, gate) <= kMaxWorkgroups;
}

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

namespace {
// workgroups of a copy, of the gradient pass
int64_t pack_blocks(const PackRows& p, int elem) {
  if (p.k_contiguous) return ((int64_t)p.Rz * (p.ldo * elem / 16) + kThr - 1) / kThr;
  return (int64_t)ceil_div(p.ldo, 64) * ceil_div(p.Rz, 64);
}
// (the padding of a row, less than 64 elements, needs at most 8 threads)
int64_t grad_blocks_per_row(int64_t F) {
  const int64_t chunks = (F + 7) / 8 > 8 ? (F + 7) / 8 : 8;
  return (chunks + kThr - 1) / kThr;
}
}  // namespace

bool pack_rows_fits(const PackRows& p, int elem) {
  return pack_blocks(p, elem) <= kMaxWorkgroups;
}

bool gated_grad_fits(int64_t rows, int64_t F) {
  return rows * grad_blocks_per_row(F) <= kMaxWorkgroups;
}

hipError_t launch_pack_rows(const PackRows& p, int elem, hipStream_t s) {
  const dim3 grid((unsigned)pack_blocks(p, elem)), block(kThr);
  if (p.k_contiguous)
    return enqueue(elem == 1 ? pack_rows_kernel<1> : pack_rows_kernel<2>, grid, block, s, p,
                   (int)(p.ldo * elem / 16));
  return enqueue(elem == 1 ? pack_cols_kernel<1> : pack_cols_kernel<2>, grid, block, s, p,
                 ceil_div(p.ldo, 64));
}

hipError_t launch_gated_grad(const uint16_t* dh, int64_t lddh, const void* gu, int64_t ldgu,
                             bool gu_f32, int M, int64_t F, int act, uint16_t* dgu, int64_t lddgu,
                             int rows, int64_t cols, hipStream_t s) {
  const int64_t per_row = grad_blocks_per_row(F);
  const dim3 grid((unsigned)(rows * per_row)), block(kThr);
  if (gu_f32)
    return enqueue(gated_grad_kernel<float>, grid, block, s, dh, lddh,
                   static_cast<const float*>(gu), ldgu, M, F, act, dgu, lddgu, cols, per_row);
  return enqueue(gated_grad_kernel<uint16_t>, grid, block, s, dh, lddh,
                 static_cast<const uint16_t*>(gu), ldgu, M, F, act, dgu, lddgu, cols, per_row);
}

}  // namespace tgemm
