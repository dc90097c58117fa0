// A mixture-of-experts layer for few tokens (up to kMoeTokens per pass):
//   l = x . R                      (64-bit sums)
//   ids, p: the top-k of l, softmax weights
//   y[t] = sum_j p[t][j] (act(g) u) . W2[e_j]^T,  [g | u] = x[t] . W1[e_j]^T
// With a few tokens each expert that is hit serves a handful of rows, so the
// layer is bound by streaming the hit experts' weights from HBM once.
//
// Logits: one workgroup per expert and eight tokens, products and sums in 64
// bits, so that which experts a token takes depends on no order of summation.
// Choice: an expert's place is the number of experts before it (larger logit, or
// equal and lower index), counted from LDS: by a workgroup per token, or for few
// logits by each workgroup of the up product itself, a launch less.  No list of
// experts is built in memory: a workgroup of the products finds its expert's
// tokens by a scan of the ids (at most 1024).
//
// The products are those of the few-row kernel (rows_skinny.hip): the weight's
// rows take the matrix instruction's row side, the tokens its columns; a wave
// loads whole 128-byte runs of its rows and turns them around in LDS words of
// its own.  Up: a workgroup takes 16 outputs (gate and up) of one expert, its
// waves share the K steps, and their sums meet in LDS in wave order.  Down, two
// ways: a workgroup takes 16 columns of y and all experts that are hit, its waves
// runs of K steps of them (few tokens and weights); or 32 to 64 columns of one
// expert, as up, a row of sums per choice in memory, and a last kernel adds a
// token's choices by their weights, in order.  Nothing depends on timing.
//
// h = act(g) u is kept as the sum of two bf16 values, 16 bits in all: rounded to
// one it would be half of y's error.  The matrix instruction's 16 columns hold
// eight tokens' high and low parts, so that for up to 8 tokens the second part
// is free, and the weights are read once in any case.
//
// Measured (MI355X): 13 tokens on 2 of 8 experts 4096 x 13824 (2.7 GB of weights)
// 418 us, 6.5 TB/s; 64 tokens on 8 of 128 experts 2048 x 768 (1.2 GB) 214 us; one
// token on 8 of 64 experts 2048 x 1024 (100 MB) 30 us, three launches.
#include "chunk_rows.h"
#include "ffn.h"
#include "gemm_kernel.h"
#include "row_vec.h"

namespace tgemm {
namespace {

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

// The choices of expert e into list, by the whole workgroup; their number, and in
// s_first the first of them.  (Their order there decides nothing: each choice's
// sums are its own.)
__device__ __forceinline__ int expert_tokens(const MoeParams& p, const int32_t* ids, int e,
                                             int threads, uint16_t* list, int& s_n, int& s_first) {
  const int A = p.M * p.top;
  if (threadIdx.x == 0) s_n = 0, s_first = A;
  __syncthreads();
  for (int a = threadIdx.x; a < A; a += threads) {
    if (ids[a] != e) continue;
    list[atomicAdd(&s_n, 1)] = (uint16_t)a;
    atomicMin(&s_first, a);
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(s_n);
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

  const int n = expert_tokens(p, ids, e, W * 64, list, s_n, s_first);
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
      float v[4], low[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = c0 + i < p.F ? act_times(a[i], u[i], p.act) : 0.f;
        low[i] = v[i] - from_bf16(to_bf16(v[i]));
        // (an infinite or NaN h has no second part)
        if (!(fabsf(low[i]) <= 3.402823466e38f)) low[i] = 0.f;
      }
      // (rows of h are padded with zeros to ldh, a multiple of 64; the second
      // parts follow the first ones)
      uint16_t* const o = p.h + (int64_t)list[t0 + col] * p.ldh + c0;
      put4(o, v, 4);
      put4(o + (int64_t)A * p.ldh, low, 4);
    }
    if (t0 + TB * 8 < n) __syncthreads();  // the buffer becomes staged rows again
  }
}

// ---- down --------------------------------------------------------------------

// Few weights and up to 8 tokens: a workgroup takes 16 columns of y and goes
// through all the experts that are hit, each of its 16 waves through runs of K
// steps of its own; a token's sums collect in LDS words of the wave, and the
// waves' sums are added in order.  A token that lists an expert more than once
// takes one column of that expert, multiplied by its weights one by one.
constexpr int kSmallWaves = 16;

template <bool AL, bool NT>
__global__ void __launch_bounds__(kSmallWaves * 64) moe_down_small_kernel(MoeParams p) {
  constexpr int W = kSmallWaves, STAGE = 16 * 8;
  constexpr int LD = 17;  // floats per token's 16 sums
  __shared__ i32x4_t lds[W * STAGE];
  __shared__ float sums[W * 8 * LD];
  constexpr int kChoices = 8 * kMoeTop;
  __shared__ int32_t ids[kChoices];
  __shared__ float weight[kChoices];
  // A token's first choice of an expert stands for all of them (same: bit j for
  // its choice j).  The first of these of all tokens is the expert's leader: its
  // tokens are the `count` entries of order from 8 leader on.
  __shared__ uint16_t same[kChoices], count[kChoices], order[kChoices * 8], hit[kChoices];
  __shared__ uint8_t leads[kChoices];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int A = p.M * p.top, a = threadIdx.x;
  static_assert(kChoices == 128 && kChoices <= W * 64, "a thread per choice, in two waves");
  if (a < A) {
    ids[a] = p.ids[a];
    weight[a] = p.weights[a];
  }
  for (int i = threadIdx.x; i < W * 8 * LD; i += W * 64) sums[i] = 0.f;
  __syncthreads();
  if (a < kChoices) {
    bool lead = false;
    if (a < A) {
      const int e = ids[a], own = a / p.top;
      int leader = A, before = 0, n = 0;
      uint32_t mask = 0;
      for (int t = 0; t < p.M; ++t) {
        uint32_t m = 0;
        for (int k = 0; k < p.top; ++k) m |= ids[t * p.top + k] == e ? 1u << k : 0u;
        if (m == 0) continue;
        if (n++ == 0) leader = t * p.top + __builtin_ctz(m);
        before += t < own ? 1 : 0;
        if (t == own) mask = m;
      }
      if (e >= 0 && e < p.E && (mask & ((1u << (a - own * p.top)) - 1)) == 0) {
        lead = leader == a;
        same[a] = (uint16_t)mask;
        order[leader * 8 + before] = (uint16_t)a;
        if (lead) count[a] = (uint16_t)n;
      }
    }
    leads[a] = lead;
  }
  __syncthreads();
  // the leaders in order (each wave counts them, the first two list them)
  const uint64_t lead0 = __ballot(leads[lane] != 0), lead1 = __ballot(leads[lane + 64] != 0);
  const int hits0 = __popcll(lead0), hits = hits0 + __popcll(lead1);
  if (a < kChoices && leads[a])
    hit[(wave ? hits0 : 0) + __popcll((wave ? lead1 : lead0) & ((1ull << lane) - 1))] = (uint16_t)a;
  __syncthreads();

  const int n0 = blockIdx.x * 16;
  const int kb = (int)p.F * 2, steps = (kb + kStep - 1) / kStep;
  const int runs = (steps + p.run - 1) / p.run;  // of K steps per expert
  const int lc = lane & 7, lr = lane >> 3;
  const int ld = (int)p.ldw2 * 2;
  uint32_t woff[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) woff[b] = (uint32_t)((min(n0 + b * 8 + lr, (int)p.K - 1) - n0) * ld);
  i32x4_t* const st = lds + wave * STAGE;
  float* const own = sums + wave * 8 * LD;
  int wr[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) wr[q] = lr * 8 + (lc ^ swz(8 * q + lr));
  const int r = lane & 15, g = lane >> 4;
  int fo[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) fo[s] = r * 8 + ((4 * s + g) ^ swz(r));
  // the lane's part of h: token r & 7 of a group, its first or second part
  const char* const hp = reinterpret_cast<const char*>(p.h) +
                         ((r >> 3) ? (int64_t)A * p.ldh * 2 : 0) + g * 16;

  // The wave's place: (expert, run) pair `it`, step s of it; the expert's tokens,
  // n <= 8 of them, from `base` in the order.
  const int items = hits * runs;
  struct Place {
    int it, s, send, n, base, e;
  };
  auto begin = [&](Place& q, int it) __attribute__((always_inline)) {
    q.it = it;
    if (it >= items) return;
    const int i = it / runs, c = it - i * runs;
    const int l = __builtin_amdgcn_readfirstlane((int)hit[i]);
    q.e = __builtin_amdgcn_readfirstlane(ids[l]);
    q.s = c * p.run;
    q.send = min(steps, q.s + p.run);
    q.n = __builtin_amdgcn_readfirstlane((int)count[l]);
    q.base = l * 8;
  };
  i32x4_t wv[2], av[2];
  auto load = [&](const Place& q) __attribute__((always_inline)) {
    const int k = q.s * kStep + lc * 16;
    ChunkRows<AL, NT> rw;
    rw.init(reinterpret_cast<const char*>(p.w2 + (int64_t)q.e * p.sw2) + (int64_t)n0 * ld, kb);
#pragma unroll
    for (int b = 0; b < 2; ++b) wv[b] = rw.load(woff[b], k);
    // (straight into the matrix instruction's layout: these lines are shared by
    // all workgroups, and come from the cache)
    const int a = order[q.base + min(r & 7, q.n - 1)];
    const char* const s = hp + ((int64_t)a * p.ldh * 2 + q.s * kStep);
    av[0] = *reinterpret_cast<const i32x4_t*>(s);
    av[1] = *reinterpret_cast<const i32x4_t*>(s + 64);
  };
  f32x4_t acc = {0, 0, 0, 0};
  Place cur = {};
  begin(cur, wave);
  if (cur.it < items) load(cur);
  while (cur.it < items) {
#pragma unroll
    for (int b = 0; b < 2; ++b) st[b * 64 + wr[b]] = wv[b];
    const i32x4_t af[2] = {av[0], av[1]};
    wave_lds_order();
    Place nxt = cur;
    if (++nxt.s == nxt.send) begin(nxt, cur.it + W);
    if (nxt.it < items) load(nxt);
#pragma unroll
    for (int q = 0; q < 2; ++q) acc = mma16(st[fo[q]], af[q], acc);
    wave_lds_order();
    if (nxt.it != cur.it) {
      // these tokens' sums of the run, of both parts
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += __shfl_xor(acc[i], 8, 64);
      if (r < 8 && r < cur.n) {
        const int a = order[cur.base + r], t = a / p.top;
        float* const o = own + t * LD + 4 * g;
        f32x4_t v = {o[0], o[1], o[2], o[3]};
        for (uint32_t m = same[a]; m != 0; m &= m - 1)
          v += weight[t * p.top + __builtin_ctz(m)] * acc;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = v[i];
      }
      acc = f32x4_t{0, 0, 0, 0};
    }
    cur = nxt;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.M * 16; i += W * 64) {
    const int t = i >> 4, c = i & 15;
    if (n0 + c >= p.K) continue;
    float v = sums[t * LD + c];
#pragma unroll
    for (int w = 1; w < W; ++w) v += sums[(w * 8 + t) * LD + c];
    p.y[(int64_t)t * p.ldy + n0 + c] = to_bf16(v);
  }
}

// Other calls: a workgroup takes 16 NB columns of one expert, its waves share the
// K steps, and each choice's row of sums goes to memory, [M * top][K], for
// moe_weigh_kernel.  TB groups of 8 tokens at a time; blockIdx.y as in
// moe_up_kernel.
template <int TB, int NB, int W, bool AL, bool NT>
__global__ void __launch_bounds__(W * 64) moe_down_rows_kernel(MoeParams p) {
  constexpr int STAGE = NB * 16 * 8, RED = TB * NB * 64;
  __shared__ i32x4_t lds[W * (STAGE > RED ? STAGE : RED)];
  __shared__ uint16_t list[kMoeAssign];
  __shared__ int s_n, s_first;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int slot = blockIdx.y, A = p.M * p.top;
  const int e = __builtin_amdgcn_readfirstlane(A < p.E ? p.ids[slot] : slot);
  if (e < 0 || e >= p.E) return;
  const int n = expert_tokens(p, p.ids, e, W * 64, list, s_n, s_first);
  if (n == 0 || (A < p.E && s_first != slot)) return;

  const int n0 = blockIdx.x * 16 * NB;
  const int kb = (int)p.F * 2, steps = (kb + kStep - 1) / kStep;
  const int lc = lane & 7, lr = lane >> 3;
  const int ld = (int)p.ldw2 * 2;
  ChunkRows<AL, NT> rw;
  rw.init(reinterpret_cast<const char*>(p.w2 + (int64_t)e * p.sw2) + (int64_t)n0 * ld, kb);
  uint32_t woff[2 * NB];
#pragma unroll
  for (int b = 0; b < 2 * NB; ++b)
    woff[b] = (uint32_t)((min(n0 + b * 8 + lr, (int)p.K - 1) - n0) * ld);
  i32x4_t* const st = lds + wave * STAGE;
  int wr[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) wr[q] = lr * 8 + (lc ^ swz(8 * q + lr));
  const int r = lane & 15, g = lane >> 4;
  int fo[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) fo[s] = r * 8 + ((4 * s + g) ^ swz(r));
  const char* const hp = reinterpret_cast<const char*>(p.h) +
                         ((r >> 3) ? (int64_t)A * p.ldh * 2 : 0) + g * 16;

  for (int t0 = 0; t0 < n; t0 += TB * 8) {
    f32x4_t acc[TB][NB];
    int64_t hoff[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      hoff[t] = (int64_t)list[min(t0 + t * 8 + (r & 7), n - 1)] * p.ldh * 2;
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[t][b] = f32x4_t{0, 0, 0, 0};
    }
    i32x4_t wv[2 * NB], av[TB][2];
    auto load = [&](int s) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < 2 * NB; ++b) wv[b] = rw.load(woff[b], s * kStep + lc * 16);
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        if (t0 + t * 8 >= n) continue;
        const char* const a = hp + (hoff[t] + s * kStep);
        av[t][0] = *reinterpret_cast<const i32x4_t*>(a);
        av[t][1] = *reinterpret_cast<const i32x4_t*>(a + 64);
      }
    };
    if (wave < steps) load(wave);
    for (int s = wave; s < steps; s += W) {
#pragma unroll
      for (int b = 0; b < 2 * NB; ++b) st[b * 64 + wr[b & 1]] = wv[b];
      i32x4_t af[TB][2];
#pragma unroll
      for (int t = 0; t < TB; ++t) af[t][0] = av[t][0], af[t][1] = av[t][1];
      wave_lds_order();
      if (s + W < steps) load(s + W);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        i32x4_t wf[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) wf[b] = st[b * 128 + fo[q]];
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          if (t0 + t * 8 >= n) continue;
#pragma unroll
          for (int b = 0; b < NB; ++b) acc[t][b] = mma16(wf[b], af[t][q], acc[t][b]);
        }
      }
      wave_lds_order();
    }
    __syncthreads();  // the staged rows become the sums' buffer
    f32x4_t* const red = reinterpret_cast<f32x4_t*>(lds);
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        f32x4_t v = acc[t][b];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += __shfl_xor(v[i], 8, 64);
        red[wave * RED + (t * NB + b) * 64 + lane] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < RED; i += W * 64) {
      const int l = i & 63, q = i >> 6, t = q / NB, b = q % NB;
      const int col = t * 8 + (l & 15), c0 = n0 + b * 16 + 4 * (l >> 4);
      const int m = min(4, (int)p.K - c0);
      if ((l & 15) >= 8 || t0 + col >= n || m <= 0) continue;
      f32x4_t a = red[i];
#pragma unroll
      for (int w = 1; w < W; ++w) a += red[w * RED + i];
      const float v[4] = {a[0], a[1], a[2], a[3]};
      put4(p.part + (int64_t)list[t0 + col] * p.K + c0, v, m);
    }
    if (t0 + TB * 8 < n) __syncthreads();  // the buffer becomes staged rows again
  }
}

// y = the choices' rows by their weights, in order, four columns per thread.
__global__ void __launch_bounds__(256) moe_weigh_kernel(MoeParams p, int per_row) {
  const int t = (int)(blockIdx.x / per_row);
  const int c = ((int)(blockIdx.x % per_row) * 256 + (int)threadIdx.x) * 4;
  const int n = min(4, (int)p.K - c);
  if (n <= 0) return;
  float a[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = t * p.top; j < (t + 1) * p.top; ++j) {
    const int e = p.ids[j];
    if (e < 0 || e >= p.E) continue;
    const float w = p.weights[j];
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    get4(p.part + (int64_t)j * p.K + c, v, n);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = fmaf(w, v[i], a[i]);
  }
  put4(p.y + (int64_t)t * p.ldy + c, a, n);
}

int slots_of(const MoeParams& p) { return p.M * p.top < p.E ? p.M * p.top : p.E; }

// The down product of few weights (48 MB) for up to 8 tokens, on at least 32
// workgroups per token: what idle compute units and the short runs lose is then
// less than a launch to add up the choices.  Whole layer in us in a graph, small
// kernel / the other and the sums, F = 768, 2 of 16 experts unless noted.  At the
// edge: 1 token K = 1024 14.3 / 16.7, 2 tokens 1024 18.2 / 19.5, 3 tokens 1536 23.5
// / 24.0, 4 tokens 2048 (all of 8 experts) 31.3 / 32.3, 8 tokens 4096 (F = 512, all
// of 8) 36.1 / 39.4.  Before it: 3 tokens 1024 21.6 / 20.9, 6 tokens 2048 (all of 8)
// 33.9 / 33.1, 8 tokens 2048 (all of 8) 37.1 / 35.0, 8 tokens 2048 (2 of 64) 47.6 /
// 42.2.  Past 48 MB the sides change with the shape (8 tokens 8192 x 2048, 2 of 8
// 140 / 146; 4 tokens 4096 x 1408 51.6 / 50.4; 8 tokens 2048 x 1024, 8 of 64 117 /
// 106).
bool down_small(const MoeParams& p) {
  return p.M <= 8 && p.K >= 512 * p.M &&
         (int64_t)slots_of(p) * p.F * p.K * 2 <= int64_t(48) << 20;
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

template <bool AL, bool NT>
hipError_t launch_down_small(MoeParams p, hipStream_t s) {
  const int steps = ceil_div((int64_t)p.F * 2, kStep);
  // even runs of up to 8 K steps, fewer where they would not go round the waves
  const int even = ceil_div((int64_t)slots_of(p) * steps, kSmallWaves);
  p.run = ceil_div(steps, ceil_div(steps, even < 8 ? even : 8));
  return enqueue(moe_down_small_kernel<AL, NT>, dim3(ceil_div(p.K, 16)), dim3(kSmallWaves * 64), s,
                 p);
}

template <int TB, int NB, int W, bool AL, bool NT>
hipError_t launch_down_rows(const MoeParams& p, hipStream_t s) {
  return enqueue(moe_down_rows_kernel<TB, NB, W, AL, NT>,
                 dim3(ceil_div(p.K, 16 * NB), slots_of(p)), dim3(W * 64), s, p);
}

template <bool AL, bool NT>
hipError_t launch_products(const MoeParams& p, hipStream_t s) {
  // Tokens at a time: an expert with more than that reads its weights again
  // (from the cache), so a few experts that are hit often do not decide.
  const bool few = p.M <= 8, many = (int64_t)p.M * p.top > (int64_t)12 * p.E;
  // Waves per workgroup of the up product: four for up to 32 K steps, which
  // have less to add up (2048 x 768, 64 tokens of 128 experts: 8 / 4 waves 136 /
  // 128 us; 4096 x 13824, 13 tokens of 8 experts: 266 / 276).  Whole layers between
  // these, 8 of 64 experts, 8 / 4 waves: 8 tokens, F = 1024, K = 1024 64.0 / 64.9,
  // 1536 76.0 / 75.0, 2048 102 / 103, 2560 117 / 120, 4096 184 / 190; 24 tokens, F =
  // 768, 1024 67.3 / 65.2, 2048 113 / 113, 2560 131 / 133, 4096 196 / 199; one token
  // even to 4096, 62.9 / 69.4 at 6144.
  const bool narrow = p.K <= 32 * kStep / 2;
  hipError_t e;
  if (few)
    e = narrow ? launch_up<1, 4, AL, NT>(p, s) : launch_up<1, 8, AL, NT>(p, s);
  else if (many)
    e = launch_up<8, 4, AL, NT>(p, s);
  else
    e = narrow ? launch_up<2, 4, AL, NT>(p, s) : launch_up<2, 8, AL, NT>(p, s);
  if (e != hipSuccess) return e;
  if (down_small(p)) return launch_down_small<AL, NT>(p, s);
  // Tokens at a time and columns (in 16s) of the down product: h costs a
  // workgroup as much as NB / 2 times its columns of weights for each group of
  // tokens.  Us, 1 x 2 (8 waves) / 1 x 4 / 2 x 4 / 4 x 4: one token, 2 of 8 experts
  // 4096 x 13824 36 / 51; 13 tokens, the same 137 / 133 / 135 / 136; 64 tokens, 8
  // of 128 2048 x 768 75 / 68 / 70 / 84; 40 tokens, 2 of 8 4096 x 4096 86 / 82 / 54
  // / 55; 32 tokens, 8 of 8 208 / 197 / 101 / 66.
  e = few ? launch_down_rows<1, 2, 8, AL, NT>(p, s)
          : many ? launch_down_rows<4, 4, 4, AL, NT>(p, s) : launch_down_rows<2, 4, 4, AL, NT>(p, s);
  if (e != hipSuccess) return e;
  const int per_row = ceil_div(p.K, 1024);
  return enqueue(moe_weigh_kernel, dim3((unsigned)((int64_t)p.M * per_row)), dim3(256), s, p,
                 per_row);
}

inline bool aligned16(const void* p, int64_t a, int64_t b) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(2 * a) | (uintptr_t)(2 * b)) & 15) == 0;
}

}  // namespace

MoeSpace moe_space(const MoeParams& p) {
  const size_t logits = p.router != nullptr ? (size_t)p.M * p.E * sizeof(double) : 0;
  const size_t h = (size_t)p.M * p.top * p.ldh * 4;
  const size_t part = down_small(p) ? 0 : (size_t)p.M * p.top * p.K * sizeof(float);
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
