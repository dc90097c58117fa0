// Row products with few rows of A (decode: one token up to kSkinnyRows):
// every byte of the weight B is used for a handful of products, so the
// kernel streams B from HBM once, at full width, and nothing else matters.
//
// The weight's rows take the matrix instruction's row side (16x16x64 int8,
// 16x16x32 bf16) and the tokens its column side: a lane loads 16 bytes of
// row l%16 at chunk l/16 of a 64-byte step straight into the operand
// register, with no LDS in between, since no other wave needs them.  The
// tokens' operand has the same shape and comes from L2.  Tokens past M
// repeat the last one (their columns are not stored), weight rows past N
// the last row.
//
// A workgroup's W waves share one block of weight rows and split K; their
// sums meet in LDS, in wave order, so the result does not depend on timing.
// Where the blocks alone leave compute units without work, K is split over
// workgroups too and rows_finish adds the chunks.
#include "ffn.h"
#include "gemm_kernel.h"

namespace tgemm {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

struct SkI8 {
  typedef i32x4_t acc;
  typedef int elem;
  static __device__ __forceinline__ acc mma(const i32x4_t& a, const i32x4_t& b, const acc& c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
#else
    return c;
#endif
  }
};
struct SkBf16 {
  typedef f32x4_t acc;
  typedef float elem;
  static __device__ __forceinline__ acc mma(const i32x4_t& a, const i32x4_t& b, const acc& c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
#else
    return c;
#endif
  }
};

constexpr int kStep = 64;  // bytes of K per row and matrix instruction

// MB blocks of 16 tokens, NB blocks of 16 weight rows per wave (GATE: the
// first half gate rows, the second half the up rows of the same outputs),
// W waves.
template <class Op, int MB, int NB, int W, bool GATE, int EPI>
__global__ void __launch_bounds__(W * 64) skinny_kernel(RowsParams p) {
  constexpr bool I8 = std::is_same<Op, SkI8>::value;
  constexpr int NO = GATE ? NB / 2 : NB;  // blocks of 16 outputs
  constexpr int U = NB * MB >= 8 ? 2 : (NB + MB > 4 ? 4 : 8);  // steps in flight
  __shared__ typename Op::acc red[W][NB * MB][64];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int nout = GATE ? p.F : p.N;
  const int nblk = (nout + 16 * NO - 1) / (16 * NO);
  const int blk = blockIdx.x % nblk, ks = blockIdx.x / nblk;
  const int n0 = blk * 16 * NO;
  // this wave's bytes of K: whole steps, except the last wave of the last
  // chunk
  const int cb = ks * p.kchunk, ce = min(p.K, cb + p.kchunk);
  const int steps = (ce - cb + kStep - 1) / kStep;
  const int per = (steps + W - 1) / W;
  const int s0 = min(steps, wave * per), s1 = min(steps, s0 + per);
  const int kb = cb + s0 * kStep, ke = min(ce, cb + s1 * kStep);

  const char* bp[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int o = min(n0 + (GATE ? b % NO : b) * 16 + r, nout - 1);
    const int64_t row = GATE && b >= NO ? (int64_t)p.F + o : o;
    bp[b] = p.B + row * p.ldb + g * 16;
  }
  const char* ap[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) ap[m] = p.A + (int64_t)min(m * 16 + r, p.M - 1) * p.lda + g * 16;

  typename Op::acc acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[m][b] = typename Op::acc{0, 0, 0, 0};

  int k = kb;
  for (; k + U * kStep <= ke; k += U * kStep) {
    i32x4_t wv[U][NB], av[U][MB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
        wv[u][b] = *reinterpret_cast<const i32x4_t*>(bp[b] + k + u * kStep);
#pragma unroll
      for (int m = 0; m < MB; ++m)
        av[u][m] = *reinterpret_cast<const i32x4_t*>(ap[m] + k + u * kStep);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[m][b] = Op::mma(wv[u][b], av[u][m], acc[m][b]);
  }
  for (; k < ke; k += kStep) {
    i32x4_t wv[NB], av[MB];
    const bool in = k + g * 16 < ke;  // (K is a multiple of 16 bytes)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      wv[b] = i32x4_t{0, 0, 0, 0};
      if (in) wv[b] = *reinterpret_cast<const i32x4_t*>(bp[b] + k);
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      av[m] = i32x4_t{0, 0, 0, 0};
      if (in) av[m] = *reinterpret_cast<const i32x4_t*>(ap[m] + k);
    }
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[m][b] = Op::mma(wv[b], av[m], acc[m][b]);
  }

#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int b = 0; b < NB; ++b) red[wave][m * NB + b][lane] = acc[m][b];
  __syncthreads();

  // One thread per (token, 4 consecutive outputs): lane l of a block holds
  // token l%16 and outputs 4*(l/16) .. +3.
  for (int t = threadIdx.x; t < MB * NO * 64; t += W * 64) {
    const int l = t & 63, q = t >> 6;
    const int m = q / NO, b = q % NO;
    const int row = m * 16 + (l & 15);
    const int c0 = n0 + b * 16 + 4 * (l >> 4);
    if (row >= p.M) continue;
    typename Op::acc a = red[0][m * NB + b][l], a2 = a;
#pragma unroll
    for (int w = 1; w < W; ++w) a += red[w][m * NB + b][l];
    if constexpr (GATE) {
      a2 = red[0][m * NB + NO + b][l];
#pragma unroll
      for (int w = 1; w < W; ++w) a2 += red[w][m * NB + NO + b][l];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = c0 + e;
      if (c >= nout) continue;
      if constexpr (EPI == kRowsPart) {
        auto* o = static_cast<typename Op::elem*>(p.part) + ((int64_t)ks * p.M + row) * p.N;
        o[c] = a[e];
        if constexpr (GATE) o[p.F + c] = a2[e];
      } else if constexpr (GATE) {
        float gv = (float)a[e], uv = (float)a2[e];
        if constexpr (I8) {
          const float sa = p.scale_a[row];
          gv = gv * sa * p.scale_b[c];
          uv = uv * sa * p.scale_b[p.F + c];
        }
        static_cast<uint16_t*>(p.C)[(int64_t)row * p.ldc + c] = to_bf16(act_value(gv, p.act) * uv);
        if constexpr (!I8) {
          if (p.gu != nullptr) {
            p.gu[(int64_t)row * p.ldgu + c] = to_bf16(gv);
            p.gu[(int64_t)row * p.ldgu + p.F + c] = to_bf16(uv);
          }
        }
      } else {
        const float v = (float)a[e] * p.scale_a[row] * p.scale_b[c];
        if constexpr (EPI == kRowsStoreBf16)
          static_cast<uint16_t*>(p.C)[(int64_t)row * p.ldc + c] = to_bf16(v);
        else
          static_cast<float*>(p.C)[(int64_t)row * p.ldc + c] = v;
      }
    }
  }
}

template <class Op, int MB, int NB, int W, bool GATE, int EPI>
hipError_t launch_one(const RowsParams& p, hipStream_t s) {
  constexpr int NO = GATE ? NB / 2 : NB;
  const int nblk = ceil_div(GATE ? p.F : p.N, 16 * NO);
  hipLaunchKernelGGL((skinny_kernel<Op, MB, NB, W, GATE, EPI>), dim3(nblk * p.split), dim3(W * 64),
                     0, s, p);
  return hipGetLastError();
}

// Waves per workgroup: 8 for gated blocks (two weight rows streams per
// wave), 16 for plain ones, 8 once the tokens' sums fill the LDS.
template <class Op, bool GATE, int EPI>
hipError_t launch_mb(const RowsParams& p, hipStream_t s) {
  constexpr int NB = GATE ? 2 : 1;
  if (p.M <= 16) return launch_one<Op, 1, NB, 8, GATE, EPI>(p, s);
  if (p.M <= 32) return launch_one<Op, 2, NB, 8, GATE, EPI>(p, s);
  return launch_one<Op, 4, NB, 8, GATE, EPI>(p, s);
}

}  // namespace

int rows_skinny_split(const RowsParams& p, bool gate) {
  const int nblk = ceil_div(gate ? p.F : p.N, 16);
  const int fill = 256 / nblk, by_k = p.K / 4096;
  const int n = fill < by_k ? fill : by_k;
  return n < 1 ? 1 : n;
}

hipError_t launch_rows_skinny(int type, int epi, bool gate, const RowsParams& p, hipStream_t s) {
  if (p.M > kSkinnyRows) return hipErrorInvalidValue;
  if (type == kRowsI8) {
    if (gate && epi == kRowsGated) return launch_mb<SkI8, true, kRowsGated>(p, s);
    if (gate && epi == kRowsPart) return launch_mb<SkI8, true, kRowsPart>(p, s);
    if (!gate && epi == kRowsStoreBf16) return launch_mb<SkI8, false, kRowsStoreBf16>(p, s);
    if (!gate && epi == kRowsStoreF32) return launch_mb<SkI8, false, kRowsStoreF32>(p, s);
    if (!gate && epi == kRowsPart) return launch_mb<SkI8, false, kRowsPart>(p, s);
  } else if (gate) {
    if (epi == kRowsGated) return launch_mb<SkBf16, true, kRowsGated>(p, s);
    if (epi == kRowsPart) return launch_mb<SkBf16, true, kRowsPart>(p, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace tgemm
