// Shared by the feed-forward operators' translation units: the 8-bit and
// gated products (rows_gemm.hip, rows_skinny.hip, rows_finish.hip), the row
// quantiser (row_quant.hip) and their host entries (ffn.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bf16_cvt.h"
#include "tgemm_internal.h"

namespace tgemm {

// Enqueue a kernel; the status is this launch's own.  (hipGetLastError would
// also report, and clear, an error that an earlier HIP call of the thread
// left behind.)  Grids are checked by the entries, before the first launch.
template <class... P, class... A>
hipError_t enqueue(void (*kernel)(P...), dim3 grid, dim3 block, hipStream_t s, const A&... args) {
  return [&](P... p) {
    void* v[] = {static_cast<void*>(&p)...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, v, 0, s);
  }(args...);
}

// Operand element types of the row products.
enum RowsType : int { kRowsI8 = 0, kRowsBf16 = 1 };

// What a row product does with its sums.
//   kRowsStoreBf16 / F32  C[m][n] = sum * scale_a[m] * scale_b[n]   (int8)
//   kRowsGated            C[m][f] = bf16(act(g) * u), g = column f of the
//                         product, u = column F + f (int8: after the
//                         scales; bf16: optionally g, u kept)
//   kRowsPart             the raw sums (int32 or fp32) of one K chunk, into
//                         slice `chunk` of the partial buffer [split][M][N]
//   kRowsGatedKeep        kRowsGated of bf16 operands with g, u kept (chosen by
//                         the tiled kernel's launcher when gu is set)
enum RowsEpi : int {
  kRowsStoreBf16 = 0,
  kRowsStoreF32 = 1,
  kRowsGated = 2,
  kRowsPart = 3,
  kRowsGatedKeep = 4
};

// A product of two row-major, K-contiguous operands: A [M][K], B [N][K]
// (gated: N = 2F, rows 0..F-1 the gate, F..2F-1 the up projection).  Row
// strides and K are in BYTES.  The direct-copy kernels need both bases and
// every stride and K to be multiples of 16 bytes (rows_aligned).
struct RowsParams {
  const char* A;
  const char* B;
  int64_t lda, ldb;  // bytes
  int M, N, K;       // rows of A, rows of B, bytes of K
  int F;             // gated: N / 2
  int act;           // gated: tgemm_activation
  const float* scale_a;  // int8: [M]
  const float* scale_b;  // int8: [N]
  void* C;
  int64_t ldc;       // elements
  float* gu;         // bf16 gated: optional [M][ldgu], g then u
  int64_t ldgu;
  void* part;        // kRowsPart: [split][M][N] int32 / fp32
  int tilesM, tilesN, groupM;  // the tile grid,
  int col0;          // from this output column on
  int split, kchunk; // K chunks and bytes per chunk (a multiple of 128)
};

inline bool rows_aligned(const void* p, int64_t ld_bytes, int64_t k_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)ld_bytes | (uintptr_t)k_bytes) & 15) == 0;
}

// Products of up to 64 rows read the weight once, and load it non-temporally
// (auxiliary bit 1 of a buffer load) where it cannot stay in the 256 MB
// last-level cache beside its neighbours until the next call, from
// kCacheShare bytes on.  Cold weights (us, without and with; int8 unless
// bf16): 8 x 32000 x 4096 28.4 / 26.1, gated 13824 x 5120 16 rows 30.7 / 27.7,
// 32 rows 34.2 / 32.9, one row bf16 52.4 / 47.9.  A smaller weight gains less
// cold (1 x 5120 x 13824 16.2 / 15.4) than it loses where it would have stayed
// in the cache (12.5 / 15.3); 96 and 128 rows gain 2 to 4% at most (gated 128
// rows 43.6 / 42.6) and lose up to 8% (96 x 8192 x 13824 34.2 / 37.1).
constexpr int kNonTemporal = 2;
constexpr int64_t kCacheShare = int64_t(96) << 20;
inline bool streams_past_cache(const RowsParams& p) {
  return (int64_t)p.N * p.K >= kCacheShare;
}

// Output tile shapes of the large-product kernel.
enum RowsTile : int { kRows256 = 0, kRows128x256 = 1, kRows128 = 2, kRows64 = 3 };
inline int rows_tile_m(int t) { return t == kRows256 ? 256 : t == kRows64 ? 64 : 128; }
inline int rows_tile_n(int t) { return t >= kRows128 ? 128 : 256; }

// Large products (rows_gemm.hip).  `gate`: B's rows are interleaved in the
// tile (kRowsGated, or kRowsPart of a gated product).
hipError_t launch_rows_gemm(int type, int tile, int epi, bool gate, const RowsParams& p,
                            hipStream_t s);

// Products of at most kSkinnyRows rows of A (rows_skinny.hip).
constexpr int kSkinnyRows = 64;
hipError_t launch_rows_skinny(int type, int epi, const RowsParams& p, hipStream_t s);

// Sum the partial products over the K chunks and apply `epi` (one of
// kRowsStoreBf16, kRowsStoreF32, kRowsGated) (rows_finish.hip).
bool rows_finish_fits(const RowsParams& p, bool gate);  // its grid is launchable
hipError_t launch_rows_finish(int type, int epi, const RowsParams& p, hipStream_t s);

// Copy an operand of any layout and alignment into K-contiguous rows with
// 16-byte boundaries, out [Rz][ldo], zero past K and past R: X [R][K]
// (k_contiguous) or [K][R], row stride ld (elements of 1 or 2 bytes); ldo
// times the element size a multiple of 16 (rows_finish.hip).
struct PackRows {
  const void* X;
  int64_t ld;
  bool k_contiguous;
  int R, K;
  void* out;
  int Rz;
  int64_t ldo;
};
bool pack_rows_fits(const PackRows& p, int elem);  // the copy's grid is launchable
hipError_t launch_pack_rows(const PackRows& p, int elem, hipStream_t s);

// dgu = [dh * u * act'(g) | dh * act(g)]; columns 2F .. cols - 1 and rows M
// .. rows - 1 of dgu are set to zero (rows_finish.hip).
bool gated_grad_fits(int64_t rows, int64_t F);
hipError_t launch_gated_grad(const uint16_t* dh, int64_t lddh, const void* gu, int64_t ldgu,
                             bool gu_f32, int M, int64_t F, int act, uint16_t* dgu, int64_t lddgu,
                             int rows, int64_t cols, hipStream_t s);

// dX = G . W (px: A = G [M][K], B = W) and dW = G^T . X (pw: A = G stored
// [K][M], B = X), both bf16, in one launch (gated_bwd.hip).  M, N, A, B, C,
// strides, K (a multiple of 64, G zero-padded to it) and kvb (the rows B
// holds) are set by the caller; the plan sets tiles and K chunks, and
// returns the tiles' size.  Outputs are bf16, or fp32 where asked; the fp32
// partials of a product with more than one chunk go to its ws, and a second
// launch adds them.
int gated_bwd_plan(GemmParams* px, GemmParams* pw);
bool gated_bwd_fits(const GemmParams& px, const GemmParams& pw);
hipError_t launch_gated_bwd(int tile, const GemmParams& px, const GemmParams& pw, bool f32x,
                            bool f32w, hipStream_t s);

// Rows to 8-bit codes with one scale each (row_quant.hip).  weight null:
// codes of x itself; else of the RMS norm of x (+ residual, whose bf16 sum
// goes to sum).
struct RowQuantParams {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* residual;
  int64_t ldr;
  const uint16_t* weight;
  float eps;
  uint16_t* sum;
  int64_t lds;
  int8_t* q;
  int64_t ldq;
  float* scale;
  int M;
  int64_t K;
};
bool row_quant_fits(const RowQuantParams& p);
hipError_t launch_row_quant(const RowQuantParams& p, hipStream_t s);

// ----------------------------------------------------------------------
// Activations.  Both are g * sigmoid(s(g)): silu with s = g; the tanh form
// of gelu, g/2 (1 + tanh z) with z = sqrt(2/pi)(g + 0.044715 g^3), with
// s = 2z, since (1 + tanh z)/2 = sigmoid(2z).  fp32 throughout, on the
// hardware exp2 and reciprocal (1 ulp each): the error of the exponent's
// argument, |s| 2^-24 relative in the result, stays far below the bf16
// rounding of every output down to where the sigmoid counts as 0.
//
// The sigmoid is kept in two factors, w and w r with w = e^(s/2) and
// r = 1 / (1 + w^2), which go on before and after the product with u or dh:
// 1 / (1 + e^-s) by itself overflows from s = -88.7 on, where act(g) is still
// a normal bf16 value and a large u or dh brings it up further.  So a sigmoid
// counts as 0 from 2^-252 (s = -174.7) down only.  s is capped where the
// sigmoid is 1 in fp32; there r, which is 1 - sigmoid, is not used.
// (Three operations more per output than one factor takes: gated int8 2047 x
// 13824 x 5120 307 / 310 us, training step 4096 x 13824 x 5120 3091 / 3096.  A
// second form for the tail alone, selected per value, took 316; tested for per
// group of values, 328 beside 318.)
// ----------------------------------------------------------------------
constexpr float kGeluC2 = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluK = 0.044715f;
constexpr float kActCap = 12.5f;  // of log2 w: 1 + 2^-25 is 1

struct ActFactors {
  float t, w, r;  // t: log2 w, not capped
};

__device__ __forceinline__ ActFactors act_factors(float g, int act) {
  const float s = act == 0 ? g : kGeluC2 * (g + kGeluK * g * g * g);
  const float t = 0.7213475204444817f * s;
  const float w = __builtin_amdgcn_exp2f(fminf(t, kActCap));
  return {t, w, __builtin_amdgcn_rcpf(fmaf(w, w, 1.f))};
}

// act(g) * v
__device__ __forceinline__ float act_times(float g, float v, int act) {
  const ActFactors a = act_factors(g, act);
  return g * (a.w * a.r) * v * a.w;
}

// x = h u act'(g), y = h act(g): the gradients of h act(g) u.  The
// derivative is p + g p (1 - p) s'(g) = p (1 + g r s'(g)), and 1 at the cap
// (s' may be infinite there, as it may where the sigmoid counts as 0).
__device__ __forceinline__ void act_gradients(float g, float u, float h, int act, float& x,
                                              float& y) {
  const ActFactors a = act_factors(g, act);
  const float ds = act == 0 ? 1.f : kGeluC2 * (1.f + 3.f * kGeluK * g * g);
  const float k = a.t >= kActCap || a.w == 0.f ? 1.f : fmaf(g * a.r, ds, 1.f);
  const float hw = h * (a.w * a.r);
  x = hw * u * k * a.w;
  y = hw * g * a.w;
}

// Orders a wave's LDS accesses before this point and after it, for lanes of
// one wave that exchange words of their own buffer without a workgroup
// barrier.  The hardware keeps a wave's LDS accesses in order, so this costs
// no instruction: it keeps the compiler from moving one lane's read past
// another lane's write.
__device__ __forceinline__ void wave_lds_order() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
#endif
}

// Vectors at any element alignment: the hardware takes
// unaligned vector accesses to global memory, so rows of odd length cost no
// variant of their own.
struct __attribute__((packed, aligned(2))) u16x8_any {
  uint32_t w[4];
};
struct __attribute__((packed, aligned(2))) u16x4_any {
  uint32_t w[2];
};
template <class T>
struct __attribute__((packed, aligned(4))) x4_any {
  T v[4];
};
struct __attribute__((packed, aligned(1))) b16_any {
  uint32_t w[4];
};
struct __attribute__((packed, aligned(1))) u8x8_any {
  uint32_t w[2];
};

// n (1 to 4) consecutive values as bf16, fp32 or int32, at any element
// alignment.
__device__ __forceinline__ void put4(uint16_t* o, const float* v, int n) {
  if (n >= 4) {
    *reinterpret_cast<u16x4_any*>(o) = u16x4_any{{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}};
  } else {
    for (int i = 0; i < n; ++i) o[i] = to_bf16(v[i]);
  }
}
template <class T>
__device__ __forceinline__ void put4(T* o, const T* v, int n) {
  if (n >= 4) {
    *reinterpret_cast<x4_any<T>*>(o) = x4_any<T>{{v[0], v[1], v[2], v[3]}};
  } else {
    for (int i = 0; i < n; ++i) o[i] = v[i];
  }
}

}  // namespace tgemm
