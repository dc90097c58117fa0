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
  if constexpr (EPI == kRowsLinear) {
    float bias[4], res[4];
    linear_bias4(p, c, n, bias);
    linear_res4<false>(p, row, c, n, res);
    linear_put4<false>(p, row, c, n, a, bias, res);
    return;
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

// The first n of a vector's 16 / ES elements at src, zeros behind them.  Every
// load is made, past n from the last element on: in a loop each would wait for
// the one before (13 us for a copy of a megabyte).
template <int ES>
__device__ __forceinline__ b16_any part_vector(const char* src, int n) {
  using E = std::conditional_t<ES == 1, uint8_t, uint16_t>;
  constexpr int V = 16 / ES, PER = 4 / ES;
  uint32_t e[V];
#pragma unroll
  for (int i = 0; i < V; ++i) e[i] = reinterpret_cast<const E*>(src)[i < n ? i : n - 1];
  b16_any v = {{0, 0, 0, 0}};
#pragma unroll
  for (int i = 0; i < V; ++i)
    v.w[i / PER] |= i < n ? e[i] << (i % PER * 8 * ES) : 0;
  return v;
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
    if (k + 16 / ES <= p.K)
      v = *reinterpret_cast<const b16_any*>(src);
    else
      v = part_vector<ES>(src, p.K - k);
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
      if (r + V <= p.R)
        v = *reinterpret_cast<const b16_any*>(src);
      else
        v = part_vector<ES>(src, p.R - r);
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

// The linear product's dz = dy act'(z), rounded once to bf16, the type the
// gradient products read, and the column sums of dz before that rounding.  A
// workgroup takes 256 columns (8 per thread) of a strip of rows, eight rows at a
// time; its sums over the strip meet in LDS, in row order, and workgroups of
// the gradient products' launch (gated_bwd.hip) add the strips in order: nothing
// depends on timing.  Rows M .. rows - 1 and columns N .. cols - 1 of dz are set
// to zero.
template <class T>  // the type of z
__global__ void __launch_bounds__(kThr) linear_grad_kernel(
    const uint16_t* __restrict__ dy, int64_t lddy, const T* __restrict__ z, int64_t ldz, int M,
    int64_t N, int act, uint16_t* __restrict__ dz, int64_t lddz, int rows, int64_t cols,
    float* __restrict__ part, int cblocks, int strip_rows) {
  __shared__ float sums[8][256 + 8];
  const int strip = (int)(blockIdx.x / cblocks);
  const int64_t c0 = (int64_t)(blockIdx.x % cblocks) * 256;
  const int cl = ((int)threadIdx.x & 31) * 8, rl = (int)threadIdx.x >> 5;
  const int64_t c = c0 + cl;
  const int n = (int)min((int64_t)8, N - c);  // values this thread computes
  float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int i = 0; i < strip_rows; i += 8) {
    const int row = strip * strip_rows + i + rl;
    if (row >= rows || c >= cols) continue;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (row < M) {
      const uint16_t* const pd = dy + row * lddy + c;
      if (n == 8) {
        float d[8], v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        load_values<8>(pd, d);
        if (act != kActNone) load_values<8>(z + row * ldz + c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = linear_act_grad(v[e], d[e], act);
      } else {
        for (int e = 0; e < n; ++e) {
          float d[1], v[1] = {0.f};
          load_values<1>(pd + e, d);
          if (act != kActNone) load_values<1>(z + row * ldz + c + e, v);
          x[e] = linear_act_grad(v[0], d[0], act);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] += x[e];
    // (cols is a multiple of 64, lddz of 8)
    uint4 o;
    o.x = pack_bf16x2(x[0], x[1]);
    o.y = pack_bf16x2(x[2], x[3]);
    o.z = pack_bf16x2(x[4], x[5]);
    o.w = pack_bf16x2(x[6], x[7]);
    *reinterpret_cast<uint4*>(dz + row * lddz + c) = o;
  }
  if (part == nullptr) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[rl][cl + e] = t[e];
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int r = 0; r < 8; ++r) s += sums[r][threadIdx.x];
  if (c0 + (int)threadIdx.x < N) part[strip * N + c0 + (int)threadIdx.x] = s;
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
  } else if (epi == kRowsLinear) {
    return finish_one<float, kRowsLinear>(p, s);
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

// Rows per strip: 64, or fewer until there are two workgroups per compute unit
// (333 x 1000: strips of 64 rows, 24 workgroups, 11.9 us).
int linear_grad_strip(int64_t rows, int64_t cols) {
  int strip = 64;
  while (strip > 8 && (int64_t)ceil_div(rows, strip) * ceil_div(cols, 256) < 512) strip /= 2;
  return strip;
}

bool linear_grad_fits(int64_t rows, int64_t cols) {
  return (int64_t)ceil_div(rows, linear_grad_strip(rows, cols)) * ceil_div(cols, 256) <=
         kMaxWorkgroups;
}

hipError_t launch_linear_grad(const uint16_t* dy, int64_t lddy, const void* z, int64_t ldz,
                              bool z_f32, int M, int64_t N, int act, uint16_t* dz, int64_t lddz,
                              int rows, int64_t cols, float* part, hipStream_t s) {
  const int strip = linear_grad_strip(rows, cols), cblocks = ceil_div(cols, 256);
  const dim3 grid((unsigned)((int64_t)ceil_div(rows, strip) * cblocks)), block(kThr);
  if (z_f32)
    return enqueue(linear_grad_kernel<float>, grid, block, s, dy, lddy,
                   static_cast<const float*>(z), ldz, M, N, act, dz, lddz, rows, cols, part,
                   cblocks, strip);
  return enqueue(linear_grad_kernel<uint16_t>, grid, block, s, dy, lddy,
                 static_cast<const uint16_t*>(z), ldz, M, N, act, dz, lddz, rows, cols, part,
                 cblocks, strip);
}

}  // namespace tgemm
