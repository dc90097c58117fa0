// Row products with few rows of A (decode: one token up to kSkinnyRows):
// every byte of the weight B is used for a handful of products, so the
// kernel streams B from HBM once, at full width, and nothing else matters.
//
// The weight's rows take the matrix instruction's row side (16x16x64 int8,
// 16x16x32 bf16) and the tokens its column side.  Its operand layout has
// consecutive lanes on different rows, and loading it that way from memory
// takes one request per lane (measured: 4.6 TB/s at best, bound by the
// address units).  So a wave loads whole 128-byte runs of its rows into
// registers and turns them around through LDS words of its own: no barrier,
// and the registers keep the next step's loads in flight meanwhile.
//
// A workgroup's W waves share one block of weight rows and take its 128-byte
// steps of K in turn, so together they read consecutive memory; their sums
// meet in LDS, in wave order, so the result does not depend on timing.  K is
// never split over workgroups: the second pass costs more than the idle
// compute units of a small weight (2048 x 8192: 6 us in all).
//
// Measured (MI355X) for one token: cold weights of 71 to 283 MB 4.8 to 5.9
// TB/s, where a large copy reaches 4.7; a 71 MB weight that stayed in part in
// the last-level cache 5.7.
#include "ffn.h"
#include "gemm_kernel.h"

namespace tgemm {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

struct SkI8 {
  typedef i32x4_t acc;
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
  static __device__ __forceinline__ acc mma(const i32x4_t& a, const i32x4_t& b, const acc& c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
#else
    return c;
#endif
  }
};

constexpr int kStep = 128;  // bytes of K per row and step

// TB groups of 8 tokens, NB blocks of 16 weight rows per wave (GATE: the
// first half gate rows, the second half the up rows of the same outputs),
// W waves.  ONCE: non-temporal weight loads.
template <class Op, int TB, int NB, int W, bool GATE, int EPI, bool ONCE>
__global__ void __launch_bounds__(W * 64) skinny_kernel(RowsParams p) {
  constexpr bool I8 = std::is_same<Op, SkI8>::value;
  constexpr int NO = GATE ? NB / 2 : NB;  // blocks of 16 outputs
  constexpr int MB = (TB + 1) / 2;        // blocks of 16 tokens
  // a wave's staged rows, 16-byte units: weight rows, then tokens
  constexpr int ROWS = NB * 16 + TB * 8, STAGE = ROWS * 8;
  constexpr int RED = NB * MB * 64;
  __shared__ i32x4_t lds[W * (STAGE > RED ? STAGE : RED)];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int nout = GATE ? p.F : p.N;
  const int n0 = blockIdx.x * 16 * NO;
  const int steps = (p.K + kStep - 1) / kStep;

  typename Op::acc acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[m][b] = typename Op::acc{0, 0, 0, 0};

#if defined(__HIP_DEVICE_COMPILE__)
  // Loads: lane l takes row l/8, chunk l%8 of each group of 8 rows.  Weight
  // rows past the last repeat it, tokens past M the last one (neither is
  // stored).  The buffers' range is 2^31 - 1 bytes, which no row passes
  // (the host checks the strides); a chunk at or past the end of K takes an
  // offset past it and reads as zero.
  const int lc = lane & 7, lr = lane >> 3;
  uint32_t woff[2 * NO], aoff[TB];
#pragma unroll
  for (int b = 0; b < 2 * NO; ++b)
    woff[b] = (uint32_t)((min(n0 + b * 8 + lr, nout - 1) - n0) * (int)p.ldb);
#pragma unroll
  for (int t = 0; t < TB; ++t) aoff[t] = (uint32_t)(min(t * 8 + lr, p.M - 1) * (int)p.lda);
  __amdgpu_buffer_rsrc_t rw[GATE ? 2 : 1], ra;
  ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p.A), (short)0, 0x7fffffff,
                                         0x00020000);
  rw[0] = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p.B + (int64_t)n0 * p.ldb),
                                            (short)0, 0x7fffffff, 0x00020000);
  if constexpr (GATE)
    rw[1] = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(p.B + ((int64_t)p.F + n0) * p.ldb), (short)0, 0x7fffffff,
        0x00020000);
  i32x4_t wv[2 * NB], av[TB];
  auto load = [&](int s) __attribute__((always_inline)) {
    const int k = s * kStep + lc * 16;
    const uint32_t ko = k < p.K ? (uint32_t)k : 0x80000000u;
#pragma unroll
    for (int b = 0; b < 2 * NB; ++b)
      wv[b] = __builtin_bit_cast(
          i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rw[GATE ? b / (2 * NO) : 0],
                                                         (int)(woff[b % (2 * NO)] + ko), 0,
                                                         ONCE ? kNonTemporal : 0));
#pragma unroll
    for (int t = 0; t < TB; ++t)
      av[t] = __builtin_bit_cast(
          i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(ra, (int)(aoff[t] + ko), 0, 0));
  };
  // Staged row R holds its chunk c at c ^ swz(R), as in the tiled kernels:
  // neither the writes nor the operand reads conflict.
  i32x4_t* const st = lds + wave * STAGE;
  int wr[2];  // even / odd groups of 8 rows
#pragma unroll
  for (int q = 0; q < 2; ++q) wr[q] = lr * 8 + (lc ^ swz(8 * q + lr));
  const int r = lane & 15, g = lane >> 4;
  const int ar = TB == 1 ? (r & 7) : r;  // (8 tokens: columns 8-15 repeat them)
  int fo[2], ao[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    fo[s] = r * 8 + ((4 * s + g) ^ swz(r));
    ao[s] = NB * 128 + ar * 8 + ((4 * s + g) ^ swz(ar));
  }

  if (wave < steps) load(wave);
  for (int s = wave; s < steps; s += W) {
#pragma unroll
    for (int b = 0; b < 2 * NB; ++b) st[b * 64 + wr[b & 1]] = wv[b];
#pragma unroll
    for (int t = 0; t < TB; ++t) st[NB * 128 + t * 64 + wr[t & 1]] = av[t];
    wave_lds_order();
    if (s + W < steps) load(s + W);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      i32x4_t wf[NB], af[MB];
#pragma unroll
      for (int b = 0; b < NB; ++b) wf[b] = st[b * 128 + fo[q]];
#pragma unroll
      for (int m = 0; m < MB; ++m) af[m] = st[m * 128 + ao[q]];
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[m][b] = Op::mma(wf[b], af[m], acc[m][b]);
    }
    wave_lds_order();
  }
#else
  (void)steps, (void)n0;
#endif

  __syncthreads();  // the staged rows become the sums' buffer
  typename Op::acc* const red = reinterpret_cast<typename Op::acc*>(lds);
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int b = 0; b < NB; ++b) red[wave * RED + (m * NB + b) * 64 + lane] = acc[m][b];
  __syncthreads();

  // One thread per (token, 4 consecutive outputs): lane l of a block holds
  // token l%16 and outputs 4*(l/16) .. +3.
  for (int t = threadIdx.x; t < MB * NO * 64; t += W * 64) {
    const int l = t & 63, q = t >> 6;
    const int m = q / NO, b = q % NO;
    const int row = m * 16 + (l & 15);
    const int c0 = n0 + b * 16 + 4 * (l >> 4);
    if (row >= p.M) continue;
    typename Op::acc a = red[(m * NB + b) * 64 + l], a2 = a;
#pragma unroll
    for (int w = 1; w < W; ++w) a += red[w * RED + (m * NB + b) * 64 + l];
    if constexpr (GATE) {
      a2 = red[(m * NB + NO + b) * 64 + l];
#pragma unroll
      for (int w = 1; w < W; ++w) a2 += red[w * RED + (m * NB + NO + b) * 64 + l];
    }
    const int n = min(4, nout - c0);
    if (n <= 0) continue;
    float v[4], g[4], u[4];
    const float sa = I8 ? p.scale_a[row] : 1.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = min(c0 + e, nout - 1);
      v[e] = (float)a[e];
      if constexpr (I8) v[e] = v[e] * sa * p.scale_b[c];
      if constexpr (GATE) {
        g[e] = v[e];
        u[e] = (float)a2[e];
        if constexpr (I8) u[e] = u[e] * sa * p.scale_b[p.F + c];
        v[e] = act_times(g[e], u[e], p.act);
      }
    }
    const int64_t o = (int64_t)row * p.ldc + c0;
    if constexpr (EPI == kRowsStoreF32)
      put4(static_cast<float*>(p.C) + o, v, n);
    else
      put4(static_cast<uint16_t*>(p.C) + o, v, n);
    if constexpr (GATE && !I8) {
      if (p.gu != nullptr) {
        float* const w = p.gu + (int64_t)row * p.ldgu + c0;
        put4(w, g, n);
        put4(w + p.F, u, n);
      }
    }
  }
}

template <class Op, int TB, int NB, int W, bool GATE, int EPI>
hipError_t launch_one(const RowsParams& p, hipStream_t s) {
  constexpr int NO = GATE ? NB / 2 : NB;
  const int nblk = ceil_div(GATE ? p.F : p.N, 16 * NO);
  const dim3 grid(nblk), block(W * 64);
  if (streams_past_cache(p))
    return enqueue(skinny_kernel<Op, TB, NB, W, GATE, EPI, true>, grid, block, s, p);
  return enqueue(skinny_kernel<Op, TB, NB, W, GATE, EPI, false>, grid, block, s, p);
}

// up to 32 tokens
template <class Op, int NB, bool GATE, int EPI>
hipError_t launch_few(const RowsParams& p, hipStream_t s) {
  if (p.M <= 8) return launch_one<Op, 1, NB, 8, GATE, EPI>(p, s);
  if (p.M <= 16) return launch_one<Op, 2, NB, 8, GATE, EPI>(p, s);
  return launch_one<Op, 4, NB, 8, GATE, EPI>(p, s);
}

// Blocks of weight rows per wave and waves per workgroup, by the number of
// tokens and of workgroups.  Figures in us on MI355X, N x K (gated: F x K) with
// cold weights (copies of 1.2 GB in turn):
//                       two blocks (gated four),  half the  4 waves  twice the blocks,
//                                       8 waves    blocks                     4 waves
//    1 token   int8 5120 x 13824           14.8      15.0     21.5
//              int8 32000 x 4096           24.9      25.5     27.3
//              gated int8 13824 x 5120     25.1      26.7     26.0
//              gated bf16 13824 x 5120     48.3      49.8     48.3
//   16 tokens  gated bf16 13824 x 5120     51.8      54.2     52.0
//   32 tokens  int8 5120 x 13824           21.0      28.2     23.3
//              int8 32000 x 4096           28.7      33.3     27.4
//   64 tokens  int8 5120 x 13824           27.7      38.1     28.3        37.1
//              int8 32000 x 4096           39.7      46.8     36.8        29.3
//              gated int8 8192 x 5120      21.9      27.2     22.1
//              gated bf16 8192 x 5120      37.5      48.3     37.9
// Up to 128 workgroups leave half the compute units idle, and half the blocks
// win (1 / 16 / 32 tokens, whole then half: int8 4096 x 4096 6.4 / 7.1 / 8.2,
// 6.1 / 6.4 / 7.0; gated bf16 4096 x 4096 17.0 / 17.7 / 20.2, 15.7 / 15.8 / 16.6;
// 33 / 64 tokens, four waves whole then eight half: int8 4096 x 4096 10.1 /
// 10.5, 8.0 / 8.9; gated bf16 4096 x 2048 14.9 / 15.0, 11.0 / 12.1, 4096 x 8192
// 42.8 / 46.2, 30.9 / 33.7).  About one workgroup per compute unit gives it,
// halved, two that overlap.  That pays for most gated weights (1 / 8 / 16 / 32
// tokens, whole then half: bf16 6688 x 4096 25.3 / 24.7 / 24.8 / 25.9, 21.6 /
// 21.7 / 23.5 / 25.8; 7680 x 4096 27.3 / 27.3 / 27.5 / 28.6, 23.8 / 23.7 / 24.2
// / 27.3; 8192 x 2048 17.7 / 17.4 / 17.5 / 17.8, 15.9 / 15.9 / 15.8 / 16.4; int8
// 7680 x 4096 15.7 / 15.3 / 15.4 / 15.9, 14.5 / 14.5 / 14.6 / 15.7), is even for
// short K (int8 8192 x 2048 8.2 / 8.0 / 8.2 / 9.2, 8.3 / 8.2 / 8.3 / 9.3) and
// loses at the band's upper end for long K (bf16 8192 x 5120 29.4 / 29.3 / 30.3
// / 32.8, 29.0 / 30.2 / 31.4 / 35.9).  Below the band whole blocks win (bf16
// 5504 x 4096 20.6 / 21.5 / 23.4 at 1 / 16 / 32 tokens, half 21.4 / 23.2 / 24.9),
// as they do for plain products (int8 8192 x 4096 9.3 / 9.6 / 10.2, 9.1 / 9.9 /
// 11.3).
template <class Op, bool GATE, int EPI>
hipError_t launch_blocks(const RowsParams& p, hipStream_t s) {
  constexpr int NB = GATE ? 4 : 2;
  const int nout = GATE ? p.F : p.N;
  const int blocks = ceil_div(nout, 32);
  const bool half = blocks <= 128 || (GATE && blocks > 208 && blocks <= 256);
  if (p.M <= 32)
    return half ? launch_few<Op, NB / 2, GATE, EPI>(p, s) : launch_few<Op, NB, GATE, EPI>(p, s);
  if (blocks <= 128) return launch_one<Op, 8, NB / 2, 8, GATE, EPI>(p, s);
  if constexpr (!GATE) {
    if (ceil_div(nout, 64) >= 256) return launch_one<Op, 8, 4, 4, GATE, EPI>(p, s);
  }
  return launch_one<Op, 8, NB, 4, GATE, EPI>(p, s);
}

}  // namespace

hipError_t launch_rows_skinny(int type, int epi, const RowsParams& p, hipStream_t s) {
  if (p.M > kSkinnyRows) return hipErrorInvalidValue;
  if (type == kRowsBf16)
    return epi == kRowsGated ? launch_blocks<SkBf16, true, kRowsGated>(p, s) : hipErrorInvalidValue;
  if (epi == kRowsGated) return launch_blocks<SkI8, true, kRowsGated>(p, s);
  if (epi == kRowsStoreBf16) return launch_blocks<SkI8, false, kRowsStoreBf16>(p, s);
  if (epi == kRowsStoreF32) return launch_blocks<SkI8, false, kRowsStoreF32>(p, s);
  return hipErrorInvalidValue;
}

}  // namespace tgemm
