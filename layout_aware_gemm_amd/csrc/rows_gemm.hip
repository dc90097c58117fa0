// Large products of two K-contiguous operands on the matrix cores, int8
// (scaled, or gated) and bf16 (gated, or with bias, activation and residual):
// out = epilogue(A . B^T), A [M][K], B [N][K].
//
// The LDS image, copy schedule and tile shapes are those of the bf16 NT
// kernel: a k-step is 128 bytes of every row (128 int8 or 64 bf16), copied
// straight from global memory into swizzled LDS rows, two A and three B
// panels in flight, one barrier per k-step.  A 16-byte chunk per lane feeds
// one matrix instruction of either type (32x32x32 int8, 32x32x16 bf16), so
// one loop serves both: an int8 k-step does twice the products in the same
// cycles, and the sums of int8 are exact in int32.
//
// Edges need no other loop.  Each panel is read through a buffer whose
// range ends with the operand's last row, so rows past it read as zero, and
// in the last k-step the lanes whose chunk starts at or past K take an
// offset outside the range.
//
// Gated products (B holds F gate rows, then F up rows) interleave the two
// halves in groups of 32 tile rows: accumulator blocks 2j and 2j + 1 of a
// lane are gate and up of the same output columns, so act(g) * u is formed
// in registers and the [M][2F] product never reaches memory.
#include "ffn.h"
#include "gemm_kernel.h"

namespace tgemm {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

struct OpI8 {
  typedef i32x4_t frag;
  typedef i32x16_t acc;
  static __device__ __forceinline__ acc mma(const frag& a, const frag& b, const acc& c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
#else
    return c;
#endif
  }
};
struct OpBf16 {
  typedef bf16x8_t frag;
  typedef f32x16_t acc;
  static __device__ __forceinline__ acc mma(const frag& a, const frag& b, const acc& c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
#else
    return c;
#endif
  }
};

// Stages of the ring of the smaller tiles (an A and a B panel each).
template <int BM, int BN>
constexpr int ring_rows() {
  return BM == 64 ? 6 : BN == 128 ? 5 : 3;  // 144, 160, 144 KB
}
constexpr int kRowBytes = 128;  // bytes of K per k-step (one LDS row)

// This wave's share of one panel's copies: R tile rows, 1 KB (8 rows) per
// copy.  Tile row r is row r of the operand, or with GATE row
// (r >> 6) * 32 + (r & 31) of its gate (r & 32 == 0) or up half.
// AUX: the loads' cache policy.
template <int R, bool GATE, int AUX = 0>
struct RowsPanel {
  static constexpr int PER_WAVE = R / 32;
  static_assert(PER_WAVE == 4 || PER_WAVE == 8 || (PER_WAVE % 2 == 0 && !GATE),
                "panels of 128 or 256 rows; without gates 64 or 192 too");
  uint32_t e[2];   // lane's byte offset in even / odd 8-row blocks
  uint32_t et[2];  // the same in a last, partial k-step: outside the range past K
  uint32_t row8;   // 8 rows in bytes
#if defined(__HIP_DEVICE_COMPILE__)
  __amdgpu_buffer_rsrc_t rs[GATE ? 2 : 1];
#endif

  static __device__ __forceinline__ uint64_t uniform(const char* p) {
    const uint64_t b = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
    return ((uint64_t)hi << 32) | lo;
  }

  // X: the operand; rows: its row count (GATE: of each half, which start
  // at X and X + rows * ld); r0: first row of this tile (of each half);
  // [kb, kend): the bytes of K to read.
  __device__ __forceinline__ void init(const char* X, int64_t ld, int rows, int r0, int kb,
                                       int kend, int wave_u, int lane) {
    // first operand row of the wave's block 0
    const int w0 = GATE ? (PER_WAVE == 8 ? wave_u * 32 : (wave_u >> 1) * 32)
                        : wave_u * PER_WAVE * 8;
    const int last = ((kend - kb - 1) & (kRowBytes - 1)) >> 4;  // last chunk of the last k-step
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      // (the swizzle of tile row 8 * block + lane / 8 depends on the block
      // only through its parity)
      const int c = (lane & 7) ^ swz((lane >> 3) + 8 * q);
      e[q] = (uint32_t)((w0 + (lane >> 3)) * ld + c * 16);
      et[q] = c <= last ? e[q] : 0x80000000u;
    }
    row8 = (uint32_t)(ld * 8);
    const int valid = min(R / (GATE ? 2 : 1), rows - r0);
    const int bytes = (int)((valid - 1) * ld + (kend - kb));
#if defined(__HIP_DEVICE_COMPILE__)
    const char* o = X + (int64_t)r0 * ld + kb;
    // word 3 = 0x00020000: 32-bit data format, the raw-buffer setting
    if constexpr (!GATE) {
      rs[0] = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uniform(o)), (short)0,
                                                __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
    } else {
      // 256 rows: a wave's blocks 0-3 are gate rows, 4-7 up rows; 128 rows:
      // even waves hold gate rows, odd waves up rows
      const char* u = o + (int64_t)rows * ld;
      const char* o0 = PER_WAVE == 8 ? o : ((wave_u & 1) ? u : o);
      const char* o1 = PER_WAVE == 8 ? u : o0;
      rs[0] = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uniform(o0)), (short)0,
                                                __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
      rs[1] = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uniform(o1)), (short)0,
                                                __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
    }
#else
    (void)X, (void)bytes;
#endif
  }

  // Copy block j of the k-step at byte kofs; tail: it is a partial one.
  // The whole offset sits in the lane's register (the range check takes
  // the scalar offset off the range, which must not pass below zero).
  __device__ __forceinline__ void issue_one(uint16_t* panel, int wave_u, int j, uint32_t kofs,
                                            bool tail) const {
    const int blk = wave_u * PER_WAVE + j;
    const int jj = GATE && PER_WAVE == 8 ? (j & 3) : j;
    const uint32_t off = (tail ? et[j & 1] : e[j & 1]) + (jj * row8 + kofs);
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rs[GATE && PER_WAVE == 8 ? (j >> 2) : 0],
        (__attribute__((address_space(3))) void*)(panel + blk * 512), 16, (int)off, 0, 0, AUX);
#else
    (void)panel, (void)blk, (void)off;
#endif
  }

  __device__ __forceinline__ void issue(uint16_t* panel, int wave_u, uint32_t kofs,
                                        bool tail) const {
#pragma unroll
    for (int j = 0; j < PER_WAVE; ++j) issue_one(panel, wave_u, j, kofs, tail);
  }
};

// One substep (16 bytes of K per lane): MFMA q, then one fragment read of
// the next substep and, with CP, this wave's copies of one panel, both
// spread over the slots.
template <class Op, int FM, int FN, bool CP, class Panel>
__device__ __forceinline__ void rows_substep(typename Op::acc (&acc)[FM][FN],
                                             const typename Op::frag* fa,
                                             const typename Op::frag* fb,
                                             typename Op::frag* na, typename Op::frag* nb,
                                             const uint16_t* pa, const uint16_t* pb,
                                             const Panel& d, uint16_t* dst, int wave_u,
                                             uint32_t kofs, bool tail) {
  constexpr int SL = FM * FN;
#pragma unroll
  for (int q = 0; q < SL; ++q) {
    acc[q / FN][q % FN] = Op::mma(fa[q / FN], fb[q % FN], acc[q / FN][q % FN]);
    if (q < FM)
      na[q] = *reinterpret_cast<const typename Op::frag*>(pa + q * 32 * kBK);
    else if (q < FM + FN)
      nb[q - FM] = *reinterpret_cast<const typename Op::frag*>(pb + (q - FM) * 32 * kBK);
    if constexpr (CP) {
#pragma unroll
      for (int c = 0; c < Panel::PER_WAVE; ++c)
        if ((c * SL) / Panel::PER_WAVE == q) d.issue_one(dst, wave_u, c, kofs, tail);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// One substep of the ring loop: as above, with quarter X of the copies of
// one whole stage (A's NA blocks, then B's) spread over the slots.
template <class Op, int FM, int FN, int X, class PA, class PB>
__device__ __forceinline__ void ring_rows_substep(typename Op::acc (&acc)[FM][FN],
                                                  const typename Op::frag* fa,
                                                  const typename Op::frag* fb,
                                                  typename Op::frag* na, typename Op::frag* nb,
                                                  const uint16_t* pa, const uint16_t* pb,
                                                  const PA& da, const PB& db, uint16_t* da_dst,
                                                  uint16_t* db_dst, int wave_u, uint32_t kofs,
                                                  bool tail) {
  constexpr int SL = FM * FN, CN = PA::PER_WAVE + PB::PER_WAVE, RD = FM + FN;
  constexpr int C0 = (X * CN + 3) / 4, C1 = ((X + 1) * CN + 3) / 4;  // this quarter's copies
#pragma unroll
  for (int q = 0; q < SL; ++q) {
    acc[q / FN][q % FN] = Op::mma(fa[q / FN], fb[q % FN], acc[q / FN][q % FN]);
#pragma unroll
    for (int r = 0; r < RD; ++r) {
      if ((RD > SL ? (r * SL) / RD : r) != q) continue;
      if (r < FM)
        na[r] = *reinterpret_cast<const typename Op::frag*>(pa + r * 32 * kBK);
      else
        nb[r - FM] = *reinterpret_cast<const typename Op::frag*>(pb + (r - FM) * 32 * kBK);
    }
#pragma unroll
    for (int c = C0; c < C1; ++c) {
      if (((c - C0) * SL) / (C1 - C0) != q) continue;
      if (c < PA::PER_WAVE)
        da.issue_one(da_dst, wave_u, c, kofs, tail);
      else
        db.issue_one(db_dst, wave_u, c - PA::PER_WAVE, kofs, tail);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Lane l, register r of accumulator block (i, j) is row 8*(r/4) + 4*(l/32)
// + r%4 and column l%32 of the block.  Stored from registers: through LDS, in
// vectors of four, the 256x256 tile took 3 to 10% longer (8192^3 int8 449
// against 428 us).  scl: the tile's scales in LDS (loaded at the kernel's
// start, one per thread: fetched from memory between the stores they cost 28
// us per 256x256 tile, half of a K = 4096 main loop).
template <class Op, int BM, int BN, bool GATE, int EPI, bool FULL>
__device__ __forceinline__ void rows_epilogue(const RowsParams& p,
                                              typename Op::acc (&acc)[BM / 64][BN / 64],
                                              const float* scl, int m0, int n0, int wm, int wn,
                                              int lane, int ks) {
  constexpr bool I8 = std::is_same<Op, OpI8>::value;
  constexpr bool SCALED = I8 && EPI != kRowsPart;
  constexpr int FM = BM / 64, FN = BN / 64;
  const int h = lane >> 5, lc = lane & 31;
  const int rl = wm * (BM / 2) + 4 * h;   // lane's first row in the tile
  const int cl = wn * (BN / 2) + lc;      // lane's first tile column
  const int nout = GATE ? p.F : p.N;
  // lane's first output column
  const int c0 = n0 + (GATE ? wn * (BN / 4) + lc : cl);
  float sb[FN];
  if constexpr (SCALED) {
#pragma unroll
    for (int j = 0; j < FN; ++j) sb[j] = scl[BM + cl + 32 * j];
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float4 sa = make_float4(1.f, 1.f, 1.f, 1.f);
      if constexpr (SCALED)
        sa = *reinterpret_cast<const float4*>(scl + rl + i * 32 + 8 * q);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 4 * q + e;
        const int row = m0 + rl + i * 32 + 8 * q + e;
        if (!FULL && row >= p.M) continue;
        const float s = e == 0 ? sa.x : e == 1 ? sa.y : e == 2 ? sa.z : sa.w;
        if constexpr (EPI == kRowsPart) {
          auto* o = static_cast<std::conditional_t<I8, int, float>*>(p.part) +
                    ((int64_t)ks * p.M + row) * p.N;
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            const int c = c0 + 32 * (GATE ? j / 2 : j);
            if (FULL || c < nout) o[(GATE && (j & 1) ? p.F : 0) + c] = acc[i][j][r];
          }
        } else if constexpr (GATE) {
          uint16_t* const o = static_cast<uint16_t*>(p.C) + (int64_t)row * p.ldc;
#pragma unroll
          for (int j = 0; j < FN / 2; ++j) {
            const int c = c0 + 32 * j;
            float g = (float)acc[i][2 * j][r], u = (float)acc[i][2 * j + 1][r];
            if constexpr (I8) {
              g = g * s * sb[2 * j];
              u = u * s * sb[2 * j + 1];
            }
            if (!FULL && c >= nout) continue;
            o[c] = to_bf16(act_times(g, u, p.act));
          }
        } else {
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            const int c = c0 + 32 * j;
            const float v = (float)acc[i][j][r] * s * sb[j];
            if (!FULL && c >= nout) continue;
            if constexpr (EPI == kRowsStoreBf16)
              static_cast<uint16_t*>(p.C)[(int64_t)row * p.ldc + c] = to_bf16(v);
            else
              static_cast<float*>(p.C)[(int64_t)row * p.ldc + c] = v;
          }
        }
      }
    }
}

// Words per row of a wave's 32-row buffer below: with 8 words of padding the
// two halves of a wave, which write four rows apart, use different halves of
// the banks.
template <int BN>
constexpr int keep_row() {
  return BN / 2 + 8;
}

// The gated epilogue of bf16 operands that also keeps g and u, 32 rows at a
// time through LDS words of the wave's own (st): each accumulator is used in
// one place, where three outputs from registers ran the 256x256 tile out of
// them, and the three rows leave in vectors of four.
template <int BM, int BN>
__device__ __forceinline__ void keep_epilogue(const RowsParams& p,
                                              const f32x16_t (&acc)[BM / 64][BN / 64], float* st,
                                              int row0, int n0, int wn, int lane) {
  constexpr int FM = BM / 64, FN = BN / 64, LD = keep_row<BN>();
  constexpr int NO = BN / 4;                   // outputs per row of the wave's block
  constexpr int LPR = NO / 4, RPI = 64 / LPR;  // lanes per row, rows per pass
  const int h = lane >> 5, lc = lane & 31;
  const int o = (lane % LPR) * 4;              // this lane's four outputs on the way out
  const int rc = (o >> 5) * 64 + (o & 31);     // their gates' columns; u is 32 behind
  const int c = n0 + wn * NO + o;
  const int n = p.F - c;                       // of which so many exist
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        st[(8 * (r >> 2) + 4 * h + (r & 3)) * LD + j * 32 + lc] = acc[i][j][r];
    wave_lds_order();
#pragma unroll
    for (int q = 0; q < 32 / RPI; ++q) {
      const int rl = q * RPI + lane / LPR, row = row0 + i * 32 + rl;
      const float4 a = *reinterpret_cast<const float4*>(st + rl * LD + rc);
      const float4 b = *reinterpret_cast<const float4*>(st + rl * LD + rc + 32);
      if (row >= p.M || n <= 0) continue;
      const float g[4] = {a.x, a.y, a.z, a.w}, u[4] = {b.x, b.y, b.z, b.w};
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act_times(g[e], u[e], p.act);
      put4(static_cast<uint16_t*>(p.C) + (int64_t)row * p.ldc + c, v, n);
      float* const w = p.gu + (int64_t)row * p.ldgu + c;
      put4(w, g, n);
      put4(w + p.F, u, n);
    }
    wave_lds_order();
  }
}

// The linear epilogue, 32 rows at a time through LDS words of the wave's own,
// as above: rows enter and leave in vectors of four (a residual read from the
// accumulators' layout takes a request for every 32 values).  A wave whose
// block lies inside the output takes U rows of lanes at a time, their loads
// ahead of the first use; others test each value.
//
// The code is kept small: all of it is run once per tile, from a cold
// instruction cache.  (Unrolled over the blocks of 32 rows it was 75 KB, and a
// 4096 x 12288 x 5120 product took 437 us, not 403.)  So the blocks are a loop,
// with the accumulators, which only constants can index, chosen by a switch.
template <int BM, int BN>
__device__ __forceinline__ void linear_epilogue(const RowsParams& p,
                                                const f32x16_t (&acc)[BM / 64][BN / 64], float* st,
                                                int row0, int col0, int lane) {
  constexpr int FM = BM / 64, FN = BN / 64, LD = keep_row<BN>();
  constexpr int LPR = BN / 8, RPI = 64 / LPR, NQ = 32 / RPI;  // lanes per row, rows per pass
  constexpr int U = 4;
  static_assert(NQ % U == 0 && RPI * NQ == 32, "whole passes");
  const int h = lane >> 5, lc = lane & 31;
  const int cl = 4 * (lane % LPR), c = col0 + cl;  // this lane's four columns
  const int n = p.N - c;                           // of which so many exist
  const int rl = lane / LPR;
  const bool idle = rl >= RPI;  // (192 columns: 24 lanes a row, 16 left over)
  const bool full = row0 + BM / 2 <= p.M && col0 + BN / 2 <= p.N;
  float b[4];
  linear_bias4(p, c, n, b);
  auto stage = [&](const f32x16_t (&a)[FN]) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        st[(8 * (r >> 2) + 4 * h + (r & 3)) * LD + j * 32 + lc] = a[j][r];
  };
#pragma unroll 1
  for (int i = 0; i < FM; ++i) {
    if (i == 0) stage(acc[0]);
    if constexpr (FM > 1)
      if (i == 1) stage(acc[1]);
    if constexpr (FM > 2)
      if (i == 2) stage(acc[2]);
    if constexpr (FM > 3)
      if (i == 3) stage(acc[3]);
    wave_lds_order();
    const int row = row0 + i * 32 + rl;
    const float* const src = st + rl * LD + cl;
    if (idle) {
    } else if (full) {
#pragma unroll 1
      for (int q = 0; q < NQ; q += U) {
        float4 v[U];
        float r[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) linear_res4<true>(p, row + (q + u) * RPI, c, 4, r[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
          v[u] = *reinterpret_cast<const float4*>(src + (q + u) * RPI * LD);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float e[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
          linear_put4<true>(p, row + (q + u) * RPI, c, 4, e, b, r[u]);
        }
      }
    } else {
#pragma unroll 1
      for (int q = 0; q < NQ; q += U) {
        float r[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int at = row + (q + u) * RPI;
          linear_res4<false>(p, at, c, at < p.M ? n : 0, r[u]);
        }
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
          const int at = row + (q + u) * RPI;
          const float4 v = *reinterpret_cast<const float4*>(src + (q + u) * RPI * LD);
          if (at >= p.M || n <= 0) continue;
          const float e[4] = {v.x, v.y, v.z, v.w};
          // (r[u], which only constants can index)
          float ru[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ru[i] = r[0][i];
#pragma unroll
            for (int k = 1; k < U; ++k) ru[i] = u == k ? r[k][i] : ru[i];
          }
          linear_put4<false>(p, at, c, n, e, b, ru);
        }
      }
    }
    wave_lds_order();
  }
}

// ONCE: B is loaded non-temporally (one row of tiles only).
template <class Op, int BM, int BN, bool GATE, int EPI, bool ONCE>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(RowsParams p) {
  constexpr bool SCALED = std::is_same<Op, OpI8>::value && EPI != kRowsPart;
  constexpr int FM = BM / 64, FN = BN / 64;
  constexpr int NT = GATE ? BN / 2 : BN;       // output columns per tile
  constexpr int SA = BM * kBK, SB = BN * kBK;  // panel sizes in 16-bit units
  static_assert(!GATE || FN % 2 == 0, "gate pairs");
  static_assert((BM == 256 && BN >= 192) || BM <= 128, "one of the two schedules");
  // two A and three B panels, or the ring
  __shared__ __attribute__((aligned(16)))
  uint16_t lds[BM <= 128 ? ring_rows<BM, BN>() * (SA + SB) : 2 * SA + 3 * SB];

  const int lane = threadIdx.x & 63;
  const int wave_u = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave_u >> 1, wn = wave_u & 1;
  const int h = lane >> 5, lc = lane & 31;
  int tile, ks, tm, tn;
  xcd_remap(blockIdx.x, p.tilesM * p.tilesN * p.split, p.split, tile, ks);
  tile_coords(tile, p.tilesM, p.tilesN, p.groupM, tm, tn);
  const int m0 = tm * BM, n0 = p.col0 + tn * NT;
  const int kb = ks * p.kchunk, kend = min(p.K, kb + p.kchunk);
  const int nk = (kend - kb + kRowBytes - 1) / kRowBytes;
  const bool partial = ((kend - kb) & (kRowBytes - 1)) != 0;

  typename Op::acc acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  RowsPanel<BM, false> da;
  RowsPanel<BN, GATE, ONCE ? kNonTemporal : 0> db;
  da.init(p.A, p.lda, p.M, m0, kb, kend, wave_u, lane);
  db.init(p.B, p.ldb, GATE ? p.F : p.N, n0, kb, kend, wave_u, lane);

  // the scales of tile row and tile column threadIdx.x, for the epilogue
  float sa_t = 0.f, sb_t = 0.f;
  if constexpr (SCALED) {
    const int t = threadIdx.x;
    sa_t = p.scale_a[min(m0 + t, p.M - 1)];
    if constexpr (GATE)
      sb_t = p.scale_b[((t & 32) ? p.F : 0) + min(n0 + (t >> 6) * 32 + (t & 31), p.F - 1)];
    else
      sb_t = p.scale_b[min(n0 + t, p.N - 1)];
  }

  const int a_base = (wm * (BM / 2) + lc) * kBK;
  const int b_base = (wn * (BN / 2) + lc) * kBK;
  int xo[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) xo[s] = ((2 * s + h) ^ swz(lc)) << 3;

  // k-steps past the end re-read k-step 0 into a buffer that is never
  // multiplied, which keeps the copy counts, and so the waits, uniform
  auto kof = [nk](int t) { return (uint32_t)((t < nk ? t : 0) * kRowBytes); };
  auto tail = [nk, partial](int t) { return partial && (t == nk - 1 || (t > nk - 1 && nk == 1)); };
  constexpr int NA = RowsPanel<BM, false>::PER_WAVE, NB = RowsPanel<BN, GATE>::PER_WAVE;
  typename Op::frag fa[2][FM], fb[2][FN];
  // fragments of substep 0 of the first k-step
  auto read_first = [&](const uint16_t* a, const uint16_t* b) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
      fa[0][i] = *reinterpret_cast<const typename Op::frag*>(a + a_base + xo[0] + i * 32 * kBK);
#pragma unroll
    for (int j = 0; j < FN; ++j)
      fb[0][j] = *reinterpret_cast<const typename Op::frag*>(b + b_base + xo[0] + j * 32 * kBK);
  };
  if constexpr (BM <= 128) {
    // Ring of S stages: after the barrier of k-step kt its stage is free,
    // and the copies of k-step kt + S go there, a quarter in each of the next
    // four substeps.  A small tile's k-step is short (4 or 8 matrix
    // instructions per substep), so it takes several in flight to cover the
    // memory's latency.
    constexpr int S = ring_rows<BM, BN>(), CN = NA + NB;
    auto stA = [&](int g) { return lds + g * (SA + SB); };
#pragma unroll
    for (int g = 0; g < S - 1; ++g) {
      da.issue(stA(g), wave_u, kof(g), tail(g));
      db.issue(stA(g) + SA, wave_u, kof(g), tail(g));
    }
    constexpr int C1 = (CN + 3) / 4;  // the first quarter of stage S - 1
    static_assert(C1 <= NA, "copies of A");
#pragma unroll
    for (int c = 0; c < C1; ++c) da.issue_one(stA(S - 1), wave_u, c, kof(S - 1), tail(S - 1));
    __builtin_amdgcn_s_waitcnt(waitcnt_imm((S - 2) * CN + C1, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_first(lds, lds + SA);
    int cur = 0;  // kt % S
    for (int kt = 0; kt < nk; ++kt) {
      const int nxt = cur + 1 == S ? 0 : cur + 1, prv = cur == 0 ? S - 1 : cur - 1;
      const uint16_t* ac = stA(cur) + a_base;
      const uint16_t* bc = stA(cur) + SA + b_base;
      const uint16_t* an = stA(nxt) + a_base;
      const uint16_t* bn = stA(nxt) + SA + b_base;
      uint16_t* dp = stA(prv);
      const uint32_t kp = kof(kt - 1 + S), kn = kof(kt + S);
      const bool tp = tail(kt - 1 + S), tn2 = tail(kt + S);
      __builtin_amdgcn_sched_barrier(0);
      ring_rows_substep<Op, FM, FN, 1>(acc, fa[0], fb[0], fa[1], fb[1], ac + xo[1], bc + xo[1], da,
                                       db, dp, dp + SA, wave_u, kp, tp);
      ring_rows_substep<Op, FM, FN, 2>(acc, fa[1], fb[1], fa[0], fb[0], ac + xo[2], bc + xo[2], da,
                                       db, dp, dp + SA, wave_u, kp, tp);
      ring_rows_substep<Op, FM, FN, 3>(acc, fa[0], fb[0], fa[1], fb[1], ac + xo[3], bc + xo[3], da,
                                       db, dp, dp + SA, wave_u, kp, tp);
      // k-step kt+1 landed (own copies: all but the S-2 stages after it;
      // other waves': the barrier) and this wave's reads of k-step kt are
      // done, so after the barrier its stage is free
      __builtin_amdgcn_s_waitcnt(waitcnt_imm((S - 2) * CN, 0));
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      uint16_t* dc = stA(cur);
      ring_rows_substep<Op, FM, FN, 0>(acc, fa[1], fb[1], fa[0], fb[0], an + xo[0], bn + xo[0], da,
                                       db, dc, dc + SA, wave_u, kn, tn2);
      cur = nxt;
    }
  } else {
    uint16_t* const abuf = lds;           // two A panels
    uint16_t* const bbuf = lds + 2 * SA;  // three B panels
    da.issue(abuf, wave_u, kof(0), tail(0));
    db.issue(bbuf, wave_u, kof(0), tail(0));
    db.issue(bbuf + SB, wave_u, kof(1), tail(1));
    da.issue(abuf + SA, wave_u, kof(1), tail(1));
    // k-step 0 landed (own copies; other waves': the barrier)
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(NA + NB, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_first(abuf, bbuf);
    int b3 = 0;  // kt % 3
    for (int kt = 0; kt < nk; ++kt) {
      const int b3n = b3 == 2 ? 0 : b3 + 1;  // (kt + 1) % 3
      const int b3p = b3 == 0 ? 2 : b3 - 1;  // (kt + 2) % 3, the buffer k-step kt-1 used
      const uint16_t* ac = abuf + (kt & 1) * SA + a_base;
      const uint16_t* bc = bbuf + b3 * SB + b_base;
      const uint16_t* an = abuf + ((kt + 1) & 1) * SA + a_base;
      const uint16_t* bn = bbuf + b3n * SB + b_base;
      const uint32_t k2 = kof(kt + 2);
      const bool t2 = tail(kt + 2);
      __builtin_amdgcn_sched_barrier(0);
      rows_substep<Op, FM, FN, true>(acc, fa[0], fb[0], fa[1], fb[1], ac + xo[1], bc + xo[1], db,
                                     bbuf + b3p * SB, wave_u, k2, t2);
      rows_substep<Op, FM, FN, false>(acc, fa[1], fb[1], fa[0], fb[0], ac + xo[2], bc + xo[2], db,
                                      bbuf, wave_u, k2, t2);
      rows_substep<Op, FM, FN, false>(acc, fa[0], fb[0], fa[1], fb[1], ac + xo[3], bc + xo[3], db,
                                      bbuf, wave_u, k2, t2);
      // A(kt+1) and B(kt+1) landed (own copies: all but the NB just issued;
      // other waves': the barrier) and this wave's reads of k-step kt are
      // done, so after the barrier A(kt)'s buffer is free for A(kt+2)
      __builtin_amdgcn_s_waitcnt(waitcnt_imm(NB, 0));
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      rows_substep<Op, FM, FN, true>(acc, fa[1], fb[1], fa[0], fb[0], an + xo[0], bn + xo[0], da,
                                     abuf + (kt & 1) * SA, wave_u, k2, t2);
      b3 = b3n;
    }
  }
  // the trailing re-reads must land before the LDS is reused or released
  wait_dma();
  __syncthreads();
  if constexpr (EPI == kRowsGatedKeep) {
    constexpr int kWave = 32 * keep_row<BN>();
    static_assert(4 * kWave * 4 <= (int)sizeof(lds), "the waves' buffers fit");
    keep_epilogue<BM, BN>(p, acc, reinterpret_cast<float*>(lds) + wave_u * kWave,
                          m0 + wm * (BM / 2), n0, wn, lane);
  } else if constexpr (EPI == kRowsLinear) {
    constexpr int kWave = 32 * keep_row<BN>();
    static_assert(4 * kWave * 4 <= (int)sizeof(lds), "the waves' buffers fit");
    linear_epilogue<BM, BN>(p, acc, reinterpret_cast<float*>(lds) + wave_u * kWave,
                            m0 + wm * (BM / 2), n0 + wn * (BN / 2), lane);
  } else {
    float* const scl = reinterpret_cast<float*>(lds);  // BM row scales, BN column scales
    if constexpr (SCALED) {
      if ((int)threadIdx.x < BM) scl[threadIdx.x] = sa_t;
      if ((int)threadIdx.x < BN) scl[BM + threadIdx.x] = sb_t;
      __syncthreads();
    }
    // A wave whose whole block lies inside the output stores without tests.
    const bool full = m0 + BM <= p.M && n0 + NT <= (GATE ? p.F : p.N);
    if (full)
      rows_epilogue<Op, BM, BN, GATE, EPI, true>(p, acc, scl, m0, n0, wm, wn, lane, ks);
    else
      rows_epilogue<Op, BM, BN, GATE, EPI, false>(p, acc, scl, m0, n0, wm, wn, lane, ks);
  }
}

template <class Op, int BM, int BN, bool GATE, int EPI>
hipError_t launch_one(const RowsParams& p, hipStream_t s) {
  const dim3 grid(p.tilesM * p.tilesN * p.split), block(kThreads);
  // (one row of 64-row tiles: only gated products, whole in K, come here)
  if constexpr (BM == 64 && GATE && EPI != kRowsPart) {
    if (p.tilesM == 1 && streams_past_cache(p))
      return enqueue(rows_kernel<Op, BM, BN, GATE, EPI, true>, grid, block, s, p);
  }
  return enqueue(rows_kernel<Op, BM, BN, GATE, EPI, false>, grid, block, s, p);
}

// (the K dimension is split for the smaller tiles only)
template <int BM, int BN>
hipError_t launch_tile(int type, int epi, bool gate, const RowsParams& p, hipStream_t s) {
  if (epi == kRowsPart) {
    if constexpr (BM <= 128) {
      if (type == kRowsI8)
        return gate ? launch_one<OpI8, BM, BN, true, kRowsPart>(p, s)
                    : launch_one<OpI8, BM, BN, false, kRowsPart>(p, s);
      return gate ? launch_one<OpBf16, BM, BN, true, kRowsPart>(p, s)
                  : launch_one<OpBf16, BM, BN, false, kRowsPart>(p, s);
    }
  } else if (type == kRowsI8) {
    if (gate && epi == kRowsGated) return launch_one<OpI8, BM, BN, true, kRowsGated>(p, s);
    if (!gate && epi == kRowsStoreBf16) return launch_one<OpI8, BM, BN, false, kRowsStoreBf16>(p, s);
    if (!gate && epi == kRowsStoreF32) return launch_one<OpI8, BM, BN, false, kRowsStoreF32>(p, s);
  } else if (gate && epi == kRowsGated) {
    return p.gu != nullptr ? launch_one<OpBf16, BM, BN, true, kRowsGatedKeep>(p, s)
                           : launch_one<OpBf16, BM, BN, true, kRowsGated>(p, s);
  } else if (!gate && epi == kRowsLinear) {
    return launch_one<OpBf16, BM, BN, false, kRowsLinear>(p, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_rows_gemm(int type, int tile, int epi, bool gate, const RowsParams& p,
                            hipStream_t s) {
  if (tile == kRows256) return launch_tile<256, 256>(type, epi, gate, p, s);
  if (tile == kRows256x192)
    return type == kRowsBf16 && !gate && epi == kRowsLinear
               ? launch_one<OpBf16, 256, 192, false, kRowsLinear>(p, s)
               : hipErrorInvalidValue;
  if (tile == kRows128x256) return launch_tile<128, 256>(type, epi, gate, p, s);
  if (tile == kRows64) return launch_tile<64, 128>(type, epi, gate, p, s);
  return launch_tile<128, 128>(type, epi, gate, p, s);
}

}  // namespace tgemm
