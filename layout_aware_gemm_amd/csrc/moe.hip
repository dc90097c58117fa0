// A mixture-of-experts layer for few tokens (up to kMoeTokens per pass):
//   l = x . R                      (64-bit sums)
//   ids, p: the top-k of l, softmax weights
//   y[t] = sum_j p[t][j] (act(g) u) . W2[e_j]^T,  [g | u] = x[t] . W1[e_j]^T
// With a few tokens each expert that is hit serves a handful of rows, so the
// layer is bound by streaming the hit experts' weights from HBM once.
//
// Logits: one workgroup per expert and eight tokens, products and sums in 64
// bits, so that which experts a token takes depends on no order of summation.
// Choice: one workgroup per token; an expert's place is the number of experts
// before it (larger logit, or equal and lower index), counted from LDS.
// No list of experts is built in memory: a workgroup of the products finds its
// expert's tokens by a scan of the ids (at most 1024).
//
// The products are those of the few-row kernel (rows_skinny.hip): the weight's
// rows take the matrix instruction's row side, the tokens its columns; a wave
// loads whole 128-byte runs of its rows and turns them around in LDS words of
// its own.  Gate and up: a workgroup takes 16 or 32 outputs of one expert, its
// waves share the K steps.  Down: a workgroup takes 16 columns of y and goes
// through the experts, each wave through runs of K steps of its own; a token's
// sums collect in LDS words of the wave, and the waves' sums are added in
// order.  Few columns: the experts are split over workgroups, and a last
// kernel adds their sums.  Nothing depends on timing.
#include "ffn.h"
#include "gemm_kernel.h"
#include "row_vec.h"

namespace tgemm {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;  // bytes of K per row and step
constexpr int kMoeAssign = kMoeTokens * kMoeTop;

__device__ __forceinline__ f32x4_t mma16(const i32x4_t& a, const i32x4_t& b, const f32x4_t& c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
#else
  return c;
#endif
}

// ---- routing -----------------------------------------------------------------

// A wave's sums of T = 1 or 8 values per lane; lane l returns that of value
// l * T / 64.  (Eight values: each exchange halves what a lane still holds.)
template <int T>
__device__ __forceinline__ double wave_sums(double (&s)[T]) {
  const int lane = threadIdx.x & 63;
  double v = s[0];
  if constexpr (T == 8) {
    double h[4], q[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool up = (lane & 32) != 0;
      h[i] = (up ? s[4 + i] : s[i]) + __shfl_xor(up ? s[i] : s[4 + i], 32, 64);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool up = (lane & 16) != 0;
      q[i] = (up ? h[2 + i] : h[i]) + __shfl_xor(up ? h[i] : h[2 + i], 16, 64);
    }
    const bool up = (lane & 8) != 0;
    v = (up ? q[1] : q[0]) + __shfl_xor(up ? q[0] : q[1], 8, 64);
  }
#pragma unroll
  for (int o = 32 / T; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// T = 1 or 8 tokens per workgroup.
template <class R, int T>
__global__ void __launch_bounds__(256) moe_logits_kernel(MoeParams p) {
  __shared__ double buf[4][T];
  const int e = blockIdx.x, t0 = (int)blockIdx.y * T;
  const R* const r = static_cast<const R*>(p.router) + (int64_t)e * p.ldr;
  double s[T];
#pragma unroll
  for (int t = 0; t < T; ++t) s[t] = 0.0;
  for (int64_t c = (int64_t)threadIdx.x * 8; c < p.K; c += 2048) {
    const typename Vec8<R>::type w = load8(r, c, p.K);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if (t0 + t >= p.M) break;
      const u16x8_any x = load8(p.x + (int64_t)(t0 + t) * p.ldx, c, p.K);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[t] = fma((double)value(x, i), (double)value(w, i), s[t]);
    }
  }
  const double v = wave_sums<T>(s);
  const int lane = threadIdx.x & 63, t = lane * T / 64;
  if ((lane & (64 / T - 1)) == 0) buf[threadIdx.x >> 6][t] = v;
  __syncthreads();
  const int i = threadIdx.x;
  if (i < T && t0 + i < p.M)
    p.logits[(int64_t)(t0 + i) * p.E + e] = ((buf[0][i] + buf[1][i]) + buf[2][i]) + buf[3][i];
}

// Ordered like the logits, NaN above all.
__device__ __forceinline__ uint64_t logit_key(double l) {
  const uint64_t b = (uint64_t)__double_as_longlong(l);
  if ((b & 0x7fffffffffffffffull) > 0x7ff0000000000000ull) return ~0ull;
  // (-0 is +0)
  if (b == 0x8000000000000000ull) return 0x8000000000000000ull;
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

// The logit of a key (a NaN for every NaN, 0 for -0).
__device__ __forceinline__ double key_logit(uint64_t k) {
  return __longlong_as_double((long long)(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}

// One workgroup per token, one thread per expert.
__global__ void __launch_bounds__(kMoeExperts) moe_choose_kernel(MoeParams p) {
  __shared__ __attribute__((aligned(16))) uint64_t key[kMoeExperts];
  __shared__ double chosen[kMoeTop];
  __shared__ float part[16][1];
  const int t = blockIdx.x, i = threadIdx.x;
  const double l = i < p.E ? p.logits[(int64_t)t * p.E + i] : 0.0;
  const uint64_t mine = logit_key(l);
  if (i < p.E) key[i] = mine;
  __syncthreads();
  int rank = 0;
  if (i < p.E) {
#pragma unroll 8
    for (int j = 0; j < p.E; ++j) {
      const uint64_t k = key[j];
      rank += (k > mine || (k == mine && j < i)) ? 1 : 0;
    }
    if (rank < p.top) {
      chosen[rank] = l;
      p.ids[(int64_t)t * p.top + rank] = i;
    }
  }
  __syncthreads();
  const double top = chosen[0];
  float total[1] = {0.f};
  if (p.renormalize) {
    for (int j = 0; j < p.top; ++j) total[0] += expf((float)(chosen[j] - top));
  } else {
    if (i < p.E) total[0] = expf((float)(l - top));
    group_sum(total, part);
  }
  if (i < p.top)
    p.weights[(int64_t)t * p.top + i] =
        p.scale * (expf((float)(chosen[i] - top)) / total[0]);
}

// ---- weights' rows -----------------------------------------------------------

// Rows of K elements from which lanes read 16-byte chunks, zeros past K.
// AL: base and strides on 16-byte boundaries and K a multiple of 8; NT:
// non-temporal.
template <bool AL, bool NT>
struct ChunkRows {
  const char* base;
  int kb;  // bytes of K
#if defined(__HIP_DEVICE_COMPILE__)
  __amdgpu_buffer_rsrc_t rs;
#endif
  __device__ __forceinline__ void init(const char* b, int k_bytes) {
    base = b;
    kb = k_bytes;
#if defined(__HIP_DEVICE_COMPILE__)
    // (2^31 - 1 bytes, which no row of a workgroup passes: the host checks
    // the strides; a chunk past K takes an offset past it and reads as zero)
    if constexpr (AL)
      rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(b), (short)0, 0x7fffffff, 0x00020000);
#endif
  }
  __device__ __forceinline__ i32x4_t load(uint32_t row_off, int k) const {
    i32x4_t v = {0, 0, 0, 0};
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (AL) {
      const uint32_t ko = k < kb ? (uint32_t)k : 0x80000000u;
      v = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                          rs, (int)(row_off + ko), 0, NT ? kNonTemporal : 0));
    } else {
      const char* const s = base + row_off + k;
      if (k + 16 <= kb) {
        const u16x8_any a = *reinterpret_cast<const u16x8_any*>(s);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (int)a.w[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + 2 * i < kb)
            v[i >> 1] |= (int)((uint32_t)reinterpret_cast<const uint16_t*>(s)[i] << (16 * (i & 1)));
      }
    }
#endif
    return v;
  }
};

// ---- gate and up -------------------------------------------------------------

// The choice of up to kRouteSmall experts' logits (all tokens together) by the
// workgroup itself, in the place of moe_choose_kernel: ids into LDS, and by one
// workgroup, with the weights, into memory.
constexpr int kRouteSmall = 1024;

struct SmallRoute {
  __attribute__((aligned(16))) uint64_t key[kRouteSmall];
  double chosen[8 * kMoeTop];
  int ids[8 * kMoeTop];
};

__device__ __forceinline__ void choose_here(const MoeParams& p, SmallRoute& r, int threads,
                                            bool write) {
  const int n = p.M * p.E, A = p.M * p.top;
  for (int i = threadIdx.x; i < n; i += threads) r.key[i] = logit_key(p.logits[i]);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += threads) {
    const int t = i / p.E, e = i - t * p.E;
    const uint64_t mine = r.key[i];
    const uint64_t* const row = r.key + t * p.E;
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < p.E; ++j) rank += (row[j] > mine || (row[j] == mine && j < e)) ? 1 : 0;
    if (rank < p.top) {
      r.ids[t * p.top + rank] = e;
      r.chosen[t * p.top + rank] = key_logit(mine);
    }
  }
  __syncthreads();
  if (!write) return;
  for (int a = threadIdx.x; a < A; a += threads) {
    const int t = a / p.top;
    const double top = r.chosen[t * p.top];
    float total = 0.f;
    if (p.renormalize)
      for (int j = 0; j < p.top; ++j) total += expf((float)(r.chosen[t * p.top + j] - top));
    else
      for (int j = 0; j < p.E; ++j) total += expf((float)(key_logit(r.key[t * p.E + j]) - top));
    p.ids[a] = r.ids[a];
    p.weights[a] = p.scale * (expf((float)(r.chosen[a] - top)) / total);
  }
}

// With fewer choices than experts, blockIdx.y stands for the expert of that
// choice, and the workgroup is idle if an earlier choice has the same; else for
// that expert.  TB groups of 8 tokens at a time, 16 outputs, W waves.  ROUTE: the
// workgroup makes the choice itself.
template <int TB, int W, bool ROUTE, bool AL, bool NT>
__global__ void __launch_bounds__(W * 64) moe_up_kernel(MoeParams p) {
  constexpr int NB = 2, MB = (TB + 1) / 2;  // blocks of 16 weight rows: gate, up
  constexpr int ROWS = NB * 16 + TB * 8, STAGE = ROWS * 8, RED = NB * MB * 64;
  __shared__ i32x4_t lds[W * (STAGE > RED ? STAGE : RED)];
  __shared__ uint16_t list[kMoeAssign];
  __shared__ int s_n, s_first;
  static_assert(!ROUTE || sizeof(SmallRoute) <= sizeof(lds), "the choice fits");

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int slot = blockIdx.y, A = p.M * p.top;
  const int32_t* ids = p.ids;
  if constexpr (ROUTE) {
    SmallRoute& r = *reinterpret_cast<SmallRoute*>(lds);
    choose_here(p, r, W * 64, blockIdx.x == 0 && slot == 0);
    ids = r.ids;
  }
  const int e = __builtin_amdgcn_readfirstlane(A < p.E ? ids[slot] : slot);
  if (e < 0 || e >= p.E) return;

  const int n0 = blockIdx.x * 16;
  const int kb = (int)p.K * 2, steps = (kb + kStep - 1) / kStep;
  const int lc = lane & 7, lr = lane >> 3;
  const char* const w1 = reinterpret_cast<const char*>(p.w1 + (int64_t)e * p.sw1);
  ChunkRows<AL, NT> rw[2];
  ChunkRows<AL, false> rx;
  const int ld = (int)p.ldw1 * 2;
  // (a block past the last output repeats it)
  const int b0 = min(n0, p.F - 1);
  rw[0].init(w1 + (int64_t)b0 * ld, kb);
  rw[1].init(w1 + ((int64_t)p.F + b0) * ld, kb);
  rx.init(reinterpret_cast<const char*>(p.x), kb);
  uint32_t woff[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) woff[b] = (uint32_t)((min(n0 + b * 8 + lr, p.F - 1) - b0) * ld);
  i32x4_t wv[2 * NB], av[TB];
  auto load_w = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < 2 * NB; ++b) wv[b] = rw[b / 2].load(woff[b % 2], s * kStep + lc * 16);
  };
  // a single token's workgroups all have work: the weight's first steps need
  // not wait for the list
  const bool early = p.M == 1 && wave < steps;
  if (early) load_w(wave);

  if (threadIdx.x == 0) s_n = 0, s_first = A;
  __syncthreads();
  // this expert's choices (their order decides nothing: each token's sums are
  // its own)
  for (int a = threadIdx.x; a < A; a += W * 64) {
    if (ids[a] != e) continue;
    list[atomicAdd(&s_n, 1)] = (uint16_t)a;
    atomicMin(&s_first, a);
  }
  __syncthreads();
  const int n = __builtin_amdgcn_readfirstlane(s_n);
  if (n == 0 || (A < p.E && s_first != slot)) return;

  // staged row R holds its chunk c at c ^ swz(R)
  i32x4_t* const st = lds + wave * STAGE;
  int wr[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) wr[q] = lr * 8 + (lc ^ swz(8 * q + lr));
  const int r = lane & 15, g = lane >> 4;
  const int ar = TB == 1 ? (r & 7) : r;
  int fo[2], ao[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    fo[s] = r * 8 + ((4 * s + g) ^ swz(r));
    ao[s] = NB * 128 + ar * 8 + ((4 * s + g) ^ swz(ar));
  }

  for (int t0 = 0; t0 < n; t0 += TB * 8) {
    const int tb = (min(n - t0, TB * 8) + 7) / 8;  // groups of 8 tokens in use
    f32x4_t acc[MB][NB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[m][b] = f32x4_t{0, 0, 0, 0};
    uint32_t aoff[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t)
      aoff[t] = (uint32_t)((list[min(t0 + t * 8 + lr, n - 1)] / p.top) * ((int)p.ldx * 2));
    auto load_x = [&](int s) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < TB; ++t)
        if (t < tb) av[t] = rx.load(aoff[t], s * kStep + lc * 16);
    };
    if (wave < steps) {
      if (t0 > 0 || !early) load_w(wave);
      load_x(wave);
    }
    for (int s = wave; s < steps; s += W) {
#pragma unroll
      for (int b = 0; b < 2 * NB; ++b) st[b * 64 + wr[b & 1]] = wv[b];
#pragma unroll
      for (int t = 0; t < TB; ++t)
        if (t < tb) st[NB * 128 + t * 64 + wr[t & 1]] = av[t];
      wave_lds_order();
      if (s + W < steps) {
        load_w(s + W);
        load_x(s + W);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        i32x4_t wf[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) wf[b] = st[b * 128 + fo[q]];
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          if (2 * m >= tb) continue;
          const i32x4_t af = st[m * 128 + ao[q]];
#pragma unroll
          for (int b = 0; b < NB; ++b) acc[m][b] = mma16(wf[b], af, acc[m][b]);
        }
      }
      wave_lds_order();
    }
    __syncthreads();  // the staged rows become the sums' buffer
    f32x4_t* const red = reinterpret_cast<f32x4_t*>(lds);
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int b = 0; b < NB; ++b) red[wave * RED + (m * NB + b) * 64 + lane] = acc[m][b];
    __syncthreads();
    for (int t = threadIdx.x; t < MB * 64; t += W * 64) {
      const int l = t & 63, m = t >> 6;
      const int col = m * 16 + (l & 15);  // which of the tokens
      if (t0 + col >= n || (TB == 1 && col >= 8)) continue;
      f32x4_t a = red[m * NB * 64 + l], u = red[(m * NB + 1) * 64 + l];
#pragma unroll
      for (int w = 1; w < W; ++w) {
        a += red[w * RED + m * NB * 64 + l];
        u += red[w * RED + (m * NB + 1) * 64 + l];
      }
      const int c0 = n0 + 4 * (l >> 4);
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = c0 + i < p.F ? act_times(a[i], u[i], p.act) : 0.f;
      // (rows of h are padded with zeros to ldh, a multiple of 64)
      put4(p.h + (int64_t)list[t0 + col] * p.ldh + c0, v, 4);
    }
    if (t0 + TB * 8 < n) __syncthreads();  // the buffer becomes staged rows again
  }
}

// ---- down --------------------------------------------------------------------

// 16 columns of y, TB groups of 8 tokens of an expert at a time, TMAX tokens in
// all, W waves.  blockIdx.y: which share of the experts that are hit.
template <int TB, int TMAX, int W, bool AL, bool NT>
__global__ void __launch_bounds__(W * 64) moe_down_kernel(MoeParams p) {
  constexpr int MB = (TB + 1) / 2, STAGE = (16 + TB * 8) * 8;
  constexpr int LD = 17;  // floats per token's 16 sums
  __shared__ i32x4_t lds[W * STAGE];
  __shared__ float sums[W * TMAX * LD];
  __shared__ uint16_t order[kMoeAssign];           // choices, by expert
  __shared__ uint16_t first[kMoeExperts], count[kMoeExperts], hit[kMoeExperts];
  __shared__ int cnt[kMoeExperts];
  __shared__ int s_hits;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int A = p.M * p.top;
  for (int i = threadIdx.x; i < p.E; i += W * 64) cnt[i] = 0;
  for (int i = threadIdx.x; i < W * TMAX * LD; i += W * 64) sums[i] = 0.f;
  __syncthreads();
  for (int a = threadIdx.x; a < A; a += W * 64) {
    const int e = p.ids[a];
    if (e >= 0 && e < p.E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (wave == 0) {
    // 16 experts per lane at most: sums of counts and of hits before them
    const int per = (p.E + 63) / 64, i0 = lane * per;
    int c = 0, h = 0;
    for (int i = i0; i < min(p.E, i0 + per); ++i) c += cnt[i], h += cnt[i] > 0;
    int cs = c, hs = h;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int cu = __shfl_up(cs, o, 64), hu = __shfl_up(hs, o, 64);
      if (lane >= o) cs += cu, hs += hu;
    }
    if (lane == 63) s_hits = hs;
    cs -= c;
    hs -= h;
    for (int i = i0; i < min(p.E, i0 + per); ++i) {
      const int k = cnt[i];
      first[i] = (uint16_t)cs;
      count[i] = (uint16_t)k;
      if (k > 0) hit[hs++] = (uint16_t)i;
      cnt[i] = cs;
      cs += k;
    }
  }
  __syncthreads();
  for (int a = threadIdx.x; a < A; a += W * 64) {
    const int e = p.ids[a];
    if (e >= 0 && e < p.E) order[atomicAdd(&cnt[e], 1)] = (uint16_t)a;
  }
  __syncthreads();
  const int hits = __builtin_amdgcn_readfirstlane(s_hits);
  const int h0 = (int)((int64_t)hits * blockIdx.y / gridDim.y);
  const int h1 = (int)((int64_t)hits * (blockIdx.y + 1) / gridDim.y);

  const int n0 = blockIdx.x * 16;
  const int kb = (int)p.F * 2, steps = (kb + kStep - 1) / kStep;
  const int runs = (steps + p.run - 1) / p.run;  // of K steps per expert
  const int lc = lane & 7, lr = lane >> 3;
  const int ld = (int)p.ldw2 * 2;
  uint32_t woff[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) woff[b] = (uint32_t)((min(n0 + b * 8 + lr, (int)p.K - 1) - n0) * ld);
  i32x4_t* const st = lds + wave * STAGE;
  float* const own = sums + wave * TMAX * LD;
  int wr[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) wr[q] = lr * 8 + (lc ^ swz(8 * q + lr));
  const int r = lane & 15, g = lane >> 4;
  const int ar = TB == 1 ? (r & 7) : r;
  int fo[2], ao[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    fo[s] = r * 8 + ((4 * s + g) ^ swz(r));
    ao[s] = 128 + ar * 8 + ((4 * s + g) ^ swz(ar));
  }

  // The wave's place: run `it` of the share's (expert, run) pairs, step s of
  // it, tokens from t0 of the expert's n.
  struct Place {
    int it, s, send, t0, n, base, e;
  };
  auto begin = [&](Place& q, int it) __attribute__((always_inline)) {
    q.it = it;
    if (it >= (h1 - h0) * runs) return;
    const int i = it / runs, c = it - i * runs;
    const int e = __builtin_amdgcn_readfirstlane((int)hit[h0 + i]);
    q.e = e;
    q.s = c * p.run;
    q.send = min(steps, q.s + p.run);
    q.t0 = 0;
    q.n = __builtin_amdgcn_readfirstlane((int)count[e]);
    q.base = __builtin_amdgcn_readfirstlane((int)first[e]);
  };
  i32x4_t wv[2], av[TB];
  auto load = [&](const Place& q) __attribute__((always_inline)) {
    const int k = q.s * kStep + lc * 16;
    ChunkRows<AL, NT> rw;
    rw.init(reinterpret_cast<const char*>(p.w2 + (int64_t)q.e * p.sw2) + (int64_t)n0 * ld, kb);
#pragma unroll
    for (int b = 0; b < 2; ++b) wv[b] = rw.load(woff[b], k);
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      if (q.t0 + t * 8 >= q.n) continue;
      const int a = order[q.base + min(q.t0 + t * 8 + lr, q.n - 1)];
      av[t] = *reinterpret_cast<const i32x4_t*>(reinterpret_cast<const char*>(p.h) +
                                                ((int64_t)a * p.ldh * 2 + k));
    }
  };
  f32x4_t acc[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) acc[m] = f32x4_t{0, 0, 0, 0};
  const int items = (h1 - h0) * runs;
  Place cur = {};
  begin(cur, wave);
  if (cur.it < items) load(cur);
  while (cur.it < items) {
#pragma unroll
    for (int b = 0; b < 2; ++b) st[b * 64 + wr[b]] = wv[b];
#pragma unroll
    for (int t = 0; t < TB; ++t)
      if (cur.t0 + t * 8 < cur.n) st[128 + t * 64 + wr[t & 1]] = av[t];
    wave_lds_order();
    Place nxt = cur;
    if (++nxt.s == nxt.send) {
      nxt.s = (cur.it % runs) * p.run;
      nxt.t0 += TB * 8;
      if (nxt.t0 >= nxt.n) begin(nxt, cur.it + W);
    }
    if (nxt.it < items) load(nxt);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const i32x4_t wf = st[fo[q]];
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        if (cur.t0 + m * 16 >= cur.n) continue;
        acc[m] = mma16(wf, st[m * 128 + ao[q]], acc[m]);
      }
    }
    wave_lds_order();
    if (nxt.it != cur.it || nxt.t0 != cur.t0) {
      // these tokens' sums of the run
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const int col = m * 16 + (lane & 15);
        if (cur.t0 + col < cur.n && !(TB == 1 && col >= 8)) {
          const int a = order[cur.base + cur.t0 + col];
          const float w = p.weights[a];
          float* const o = own + (a / p.top) * LD + 4 * (lane >> 4);
          // (added, not set: a token may have chosen an expert twice)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            __hip_atomic_fetch_add(o + i, w * acc[m][i], __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_WORKGROUP);
        }
        acc[m] = f32x4_t{0, 0, 0, 0};
      }
    }
    cur = nxt;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.M * 16; i += W * 64) {
    const int t = i >> 4, c = i & 15;
    if (n0 + c >= p.K) continue;
    float v = sums[t * LD + c];
#pragma unroll
    for (int w = 1; w < W; ++w) v += sums[(w * TMAX + t) * LD + c];
    if (gridDim.y == 1)
      p.y[(int64_t)t * p.ldy + n0 + c] = to_bf16(v);
    else
      p.part[((int64_t)blockIdx.y * p.M + t) * p.K + n0 + c] = v;
  }
}

// y = the shares' sums, in order, four columns per thread.
__global__ void __launch_bounds__(256) moe_add_kernel(MoeParams p, int shares, int per_row) {
  const int t = (int)(blockIdx.x / per_row);
  const int c = ((int)(blockIdx.x % per_row) * 256 + (int)threadIdx.x) * 4;
  const int n = min(4, (int)p.K - c);
  if (n <= 0) return;
  float a[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < shares; ++s) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    get4(p.part + ((int64_t)s * p.M + t) * p.K + c, v, n);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] += v[i];
  }
  put4(p.y + (int64_t)t * p.ldy + c, a, n);
}

int slots_of(const MoeParams& p) { return p.M * p.top < p.E ? p.M * p.top : p.E; }

// The down product of few weights (48 MB) for up to 8 tokens runs on workgroups
// of 16 waves and one share of the experts where that gives 128 workgroups:
// what half the compute units lose is less than a launch to add shares (8
// experts 2048 x 1024: 11.5 us whole; 8 waves 16.1 whole, in 4 shares 9.4 and
// 3.3 for the sums).
bool down_small(const MoeParams& p) {
  return p.M <= 8 && (int64_t)slots_of(p) * p.F * p.K * 2 <= int64_t(48) << 20;
}

// Shares of the experts in the down product: enough workgroups of 16 columns
// for two per compute unit (128 experts 2048 x 768, 64 tokens, 1 / 2 / 4 / 8
// shares: 161 / 94 / 68 / 75 us).
int shares_of(const MoeParams& p) {
  const int blocks = ceil_div(p.K, 16), slots = slots_of(p);
  const int want = ceil_div(down_small(p) ? 128 : 512, blocks);
  return want < slots ? want : slots;
}

// The up product's workgroups make the choice of experts themselves where there
// are few logits, and few workgroups to repeat it.
bool routes_in_up(const MoeParams& p) {
  return p.router != nullptr && p.M <= 8 && p.M * p.E <= kRouteSmall &&
         p.ldh / 16 * slots_of(p) <= 1024;
}

template <int TB, int W, bool AL, bool NT>
hipError_t launch_up(const MoeParams& p, hipStream_t s) {
  const dim3 grid((unsigned)(p.ldh / 16), slots_of(p)), block(W * 64);
  if constexpr (TB == 1) {
    if (routes_in_up(p)) return enqueue(moe_up_kernel<TB, W, true, AL, NT>, grid, block, s, p);
  }
  return enqueue(moe_up_kernel<TB, W, false, AL, NT>, grid, block, s, p);
}

template <int TB, int TMAX, int W, bool AL, bool NT>
hipError_t launch_down(MoeParams p, hipStream_t s) {
  const int steps = ceil_div((int64_t)p.F * 2, kStep), shares = shares_of(p);
  // runs of up to 8 K steps, fewer where they would not go round the waves, and
  // even ones: a wave takes every W-th (12 steps as 8 + 4 74 us, as 6 + 6 68)
  const int even = ceil_div((int64_t)slots_of(p) * steps, shares * W);
  p.run = ceil_div(steps, ceil_div(steps, even < 8 ? even : 8));
  const dim3 grid(ceil_div(p.K, 16), shares), block(W * 64);
  return enqueue(moe_down_kernel<TB, TMAX, W, AL, NT>, grid, block, s, p);
}

template <bool AL, bool NT>
hipError_t launch_products(const MoeParams& p, hipStream_t s) {
  // Tokens at a time: an expert with more than that reads its weights again
  // (from the cache), so a few experts that are hit often do not decide.
  const bool few = p.M <= 8, many = (int64_t)p.M * p.top > (int64_t)12 * p.E;
  // Waves per workgroup of the up product: four for up to 32 K steps, which
  // have less to add up (2048 x 768, 64 tokens of 128 experts: 8 / 4 waves 136 /
  // 128 us; 4096 x 13824, 13 tokens of 8 experts: 266 / 276).
  const bool narrow = p.K <= 32 * kStep / 2;
  hipError_t e;
  if (few)
    e = narrow ? launch_up<1, 4, AL, NT>(p, s) : launch_up<1, 8, AL, NT>(p, s);
  else if (many)
    e = launch_up<8, 4, AL, NT>(p, s);
  else
    e = narrow ? launch_up<2, 4, AL, NT>(p, s) : launch_up<2, 8, AL, NT>(p, s);
  if (e != hipSuccess) return e;
  if (few)
    e = down_small(p) ? launch_down<1, 16, 16, AL, NT>(p, s) : launch_down<1, 16, 8, AL, NT>(p, s);
  else if (p.M <= 16)
    e = launch_down<2, 16, 8, AL, NT>(p, s);
  else
    e = many ? launch_down<8, 64, 8, AL, NT>(p, s) : launch_down<2, 64, 8, AL, NT>(p, s);
  const int shares = shares_of(p);
  if (e != hipSuccess || shares == 1) return e;
  const int per_row = ceil_div(p.K, 1024);
  return enqueue(moe_add_kernel, dim3((unsigned)((int64_t)p.M * per_row)), dim3(256), s, p, shares,
                 per_row);
}

inline bool aligned16(const void* p, int64_t a, int64_t b) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(2 * a) | (uintptr_t)(2 * b)) & 15) == 0;
}

}  // namespace

MoeSpace moe_space(const MoeParams& p) {
  const size_t logits = p.router != nullptr ? (size_t)p.M * p.E * sizeof(double) : 0;
  const size_t h = (size_t)p.M * p.top * p.ldh * 2;
  const int shares = shares_of(p);
  const size_t part = shares > 1 ? (size_t)shares * p.M * p.K * sizeof(float) : 0;
  return {logits, h, part};
}

hipError_t launch_moe(const MoeParams& p, hipStream_t s) {
  if (p.router != nullptr) {
    const bool one = p.M == 1;
    const dim3 grid(p.E, one ? 1 : ceil_div(p.M, 8)), block(256);
    hipError_t e =
        p.router_f32
            ? enqueue(one ? moe_logits_kernel<float, 1> : moe_logits_kernel<float, 8>, grid, block,
                      s, p)
            : enqueue(one ? moe_logits_kernel<uint16_t, 1> : moe_logits_kernel<uint16_t, 8>, grid,
                      block, s, p);
    if (e == hipSuccess && !routes_in_up(p))
      e = enqueue(moe_choose_kernel, dim3(p.M), dim3(ceil_div(p.E, 64) * 64), s, p);
    if (e != hipSuccess) return e;
  }
  const bool al = aligned16(p.x, p.ldx, p.K) && aligned16(p.w1, p.ldw1, p.sw1) &&
                  aligned16(p.w2, p.ldw2, p.sw2) && p.F % 8 == 0;
  const bool nt = (int64_t)slots_of(p) * p.F * p.K * 6 >= kCacheShare;
  if (!al) return launch_products<false, false>(p, s);
  return nt ? launch_products<true, true>(p, s) : launch_products<true, false>(p, s);
}

}  // namespace tgemm
