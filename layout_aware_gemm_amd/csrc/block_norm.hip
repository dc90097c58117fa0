// The norms around a residual sum, forward and backward.
//   p = y ry wp  (or y),     ry = 1 / sqrt(mean y^2 + eps)
//   s = h + a p,             a  = scale * gate (a gate row serves M / G rows)
//   n = s rs wn,             rs = 1 / sqrt(mean s^2 + eps)
// s stays in fp32 between its sum and the norm; only its stored copy is
// rounded.  Means of squares are summed in 64 bits: squares of bf16 values
// overflow fp32 from 1.8e19 on.
//
// Gradient, for dn and ds (of s from its other uses), with e = dn wn and the
// normed rows s' = s rs, y' = y ry:
//   t   = ds + rs (e - s' sum(e s') / K)         dh = t
//   dwn = sum_m dn s'
//   dgate = sum over the gate's rows of scale t p
//   f   = a t wp,  dy = ry (f - y' sum(f y') / K),  dwp = sum_m a t y'
// Only s' and y' enter sums and products (their squares are at most K): rs^3, ry^3
// or y s would leave fp32 for rows whose squares do.  s is computed again from
// y, h and the kept factors, in fp32, as the forward had it: read back in bf16 its
// rounding would be the error of dwn.  sum(f y') follows from sums of known terms,
//   sum(f y') = sum(q (ds + rs e)) - (rs / K) sum(e s') sum(q s'),  q = a wp y',
// so a row takes one reduction, not two in a chain.
//
// Bound: HBM bandwidth.  A row stays in registers between its reduction and
// its results, so each element moves once: 8 bytes forward (bf16), 12
// backward.  Measured: 8192 x 4096 53 us forward (5.1 TB/s, a large copy's
// rate), 87 us backward (4.6 TB/s) and 7 us for the sums.  The gradients of the
// weights are kept per column in registers while a workgroup works through its
// rows; the workgroups' sums are added in order by a second kernel (no atomics:
// the same bits every time).
#include "ffn.h"
#include "row_vec.h"

namespace tgemm {
namespace {

// a, the factor of p, for 8 columns
template <bool GATE>
__device__ __forceinline__ void gate8(const u16x8_any& g, float scale, float (&a)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = GATE ? scale * value(g, i) : scale;
}

// V chunks of 8 elements per thread.
template <int V, class T, bool POST, bool GATE>
__global__ void __launch_bounds__(V == 4 ? 512 : 1024) block_norm_kernel(BlockNormParams p) {
  __shared__ double sums[2][16][1];
  const int row = blockIdx.x, W = blockDim.x;
  const int64_t K = p.K;
  const uint16_t* const y = p.y + (int64_t)row * p.ldy;
  const T* const h = static_cast<const T*>(p.h) + (int64_t)row * p.ldh;
  const uint16_t* const gate = GATE ? p.gate + (int64_t)(row / p.rows_per_gate) * p.ldgate : nullptr;
  u16x8_any yv[V], wv[POST ? V : 1], gv[GATE ? V : 1], nv[V];
  float s[V][8];
  double ss[1] = {0.0};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t c = ((int64_t)v * W + threadIdx.x) * 8;
    yv[v] = load8(y, c, K);
    const typename Vec8<T>::type hv = load8(h, c, K);
    if constexpr (POST) wv[v] = load8(p.post, c, K);
    if constexpr (GATE) gv[v] = load8(gate, c, K);
    nv[v] = load8(p.weight, c, K);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[v][i] = value(hv, i);
      if constexpr (POST) {
        const double d = (double)value(yv[v], i);
        ss[0] = fma(d, d, ss[0]);
      }
    }
  }
  float ry = 1.f;
  if constexpr (POST) {
    group_sum(ss, sums[0]);
    ry = (float)(1.0 / sqrt(ss[0] / (double)K + (double)p.eps));
    ss[0] = 0.0;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a[8];
    gate8<GATE>(gv[GATE ? v : 0], p.scale, a);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float q = value(yv[v], i);
      if constexpr (POST) q = q * ry * value(wv[v], i);
      s[v][i] = fmaf(a[i], q, s[v][i]);
      ss[0] = fma((double)s[v][i], (double)s[v][i], ss[0]);
    }
    const int64_t c = ((int64_t)v * W + threadIdx.x) * 8;
    if (c < K) put8(static_cast<T*>(p.s) + (int64_t)row * p.lds, c, K, s[v]);
  }
  group_sum(ss, sums[1]);
  const float rs = (float)(1.0 / sqrt(ss[0] / (double)K + (double)p.eps));
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t c = ((int64_t)v * W + threadIdx.x) * 8;
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = s[v][i] * rs * value(nv[v], i);
    if (c < K) put8(p.n + (int64_t)row * p.ldn, c, K, o);
  }
  if (p.rstd != nullptr && threadIdx.x == 0) {
    p.rstd[row] = rs;
    if constexpr (POST) p.rstd[(int64_t)p.M + row] = ry;
  }
}

// Partial sums of a workgroup, rows of K floats: dwn, dwp, and the gate's for
// the group that begins before its rows and the one that ends after them.
struct PartRows {
  int post, head, tail, count;
};
__host__ __device__ inline PartRows part_rows(bool post, bool gate) {
  PartRows r = {1, 1 + (post ? 1 : 0), 2 + (post ? 1 : 0), 1 + (post ? 1 : 0) + (gate ? 2 : 0)};
  return r;
}

// A thread's sums over rows of its columns' gradients, 8 per chunk: in
// registers, or (LDS) in words of its own there.
template <int V, bool LDS, int THREADS>
struct ColumnSums {
  float r[LDS ? 1 : V][8];
  static constexpr int kWords = LDS ? V * 2 * THREADS : 1;  // float4

  __device__ __forceinline__ void clear(float4* m) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (LDS) {
        m[(2 * v) * THREADS + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
        m[(2 * v + 1) * THREADS + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[v][i] = 0.f;
      }
    }
  }
  // a * b to the sum of the chunk's element i; those of a chunk in LDS wait in
  // r[0] for done.
  __device__ __forceinline__ void fma_to(int v, int i, float a, float b) {
    if constexpr (LDS)
      r[0][i] = a * b;
    else
      r[v][i] = fmaf(a, b, r[v][i]);
  }
  __device__ __forceinline__ void done(float4* m, int v) {
    if constexpr (LDS) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float4& w = m[(2 * v + q) * THREADS + threadIdx.x];
        const float4 o = w;
        w = make_float4(o.x + r[0][4 * q], o.y + r[0][4 * q + 1], o.z + r[0][4 * q + 2],
                        o.w + r[0][4 * q + 3]);
      }
    }
  }
  __device__ __forceinline__ void get(const float4* m, int v, float (&x)[8]) const {
    if constexpr (LDS) {
      const float4 a = m[(2 * v) * THREADS + threadIdx.x];
      const float4 b = m[(2 * v + 1) * THREADS + threadIdx.x];
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
      x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = r[v][i];
    }
  }
};

// The inputs of one row, as they are stored.
template <int V, class T>
struct GradRow {
  u16x8_any y[V], dn[V];
  typename Vec8<T>::type h[V], ds[V];
};

// 8 elements of a row, in and out; WHOLE: its length is a multiple of 8.  (Bytes
// in 32 bits: a row's address then stays in scalar registers, the lane's place
// in one vector register for all rows.)
template <bool WHOLE, class P>
__device__ __forceinline__ auto row8(const P* p, uint32_t c, int64_t K) {
  if constexpr (WHOLE) {
    typename Vec8<P>::type v = {};
    if (c < K)
      v = *reinterpret_cast<const typename Vec8<P>::type*>(reinterpret_cast<const char*>(p) +
                                                           (uint32_t)(c * sizeof(P)));
    return v;
  } else {
    return load8(p, c, K);
  }
}
template <bool WHOLE, class P>
__device__ __forceinline__ void put_row8(P* p, uint32_t c, int64_t K, const float (&f)[8]) {
  if constexpr (WHOLE)
    p = reinterpret_cast<P*>(reinterpret_cast<char*>(p) + (uint32_t)(c * sizeof(P)));
  if (c >= K) return;
  if constexpr (WHOLE)
    put8(p, 0, 8, f);
  else
    put8(p, c, K, f);
}

// Keeps a vector packed: the compiler would hold its eight unpacked values from
// one use to the next, in twice the registers.
__device__ __forceinline__ void stay_packed(u16x8_any& v) {
#if defined(__HIP_DEVICE_COMPILE__)
  uint32_t a = v.w[0], b = v.w[1], c = v.w[2], d = v.w[3];
  asm volatile("" : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
  v = u16x8_any{{a, b, c, d}};
#endif
}

// Workgroup b takes rows b * p.per_group .. of its p.per_group.  The next row's
// loads are issued before the reduction of this one; the weights stay in
// registers, the gate while its group lasts.  One chunk per thread: up to 1024
// threads and 128 registers.  With a post-norm and a gate, and for four chunks
// (K past 8192; 512 threads, 256 registers), the sums of the two weights move to
// LDS; where the rest does not fit either (AHEAD false), the weights and dn are
// read when they are used, and no row ahead.
template <int V>
constexpr int bwd_threads() {
  return V == 4 ? 512 : 1024;
}

template <int V, class T, bool POST, bool GATE, bool WHOLE>
__global__ void __launch_bounds__(bwd_threads<V>()) block_norm_bwd_kernel(BlockNormGradParams p) {
  typedef ColumnSums<V, V == 4 || (POST && GATE), bwd_threads<V>()> Wide;
  // registers for the weights and the next row
  constexpr bool AHEAD =
      V < 4 && (!POST || !GATE || (WHOLE && std::is_same<T, uint16_t>::value));
  __shared__ float sums[2][bwd_threads<V>() / 64][3];
  __shared__ __attribute__((aligned(16))) float4 m_an[Wide::kWords];
  __shared__ __attribute__((aligned(16))) float4 m_ap[POST ? Wide::kWords : 1];
  const int W = blockDim.x;
  const int64_t K = p.K;
  const float rk = 1.f / (float)K;
  // (up to 2^31 - 1 rows: the last group's end and the rows of rstd pass 32 bits)
  const int first = (int)blockIdx.x * p.per_group, end = first + min(p.per_group, p.M - first);
  constexpr PartRows R = {1, 1 + (POST ? 1 : 0), 2 + (POST ? 1 : 0),
                          1 + (POST ? 1 : 0) + (GATE ? 2 : 0)};
  float* const part = p.part + (int64_t)blockIdx.x * R.count * K;
  auto col = [&](int v) __attribute__((always_inline)) {
    return (uint32_t)(v * W + (int)threadIdx.x) * 8;
  };
  auto load = [&](GradRow<V, T>& r, int row) __attribute__((always_inline)) {
    const uint16_t* const y = p.y + (int64_t)row * p.ldy;
    const uint16_t* const dn = p.dn + (int64_t)row * p.lddn;
    const T* const h = static_cast<const T*>(p.h) + (int64_t)row * p.ldh;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t c = col(v);
      r.y[v] = row8<WHOLE>(y, c, K);
      r.dn[v] = row8<WHOLE>(dn, c, K);
      r.h[v] = row8<WHOLE>(h, c, K);
      r.ds[v] = {};
      if (p.ds != nullptr)
        r.ds[v] = row8<WHOLE>(static_cast<const T*>(p.ds) + (int64_t)row * p.ldds, c, K);
    }
  };
  Wide an, ap;
  ColumnSums<V, false, bwd_threads<V>()> ag;
  an.clear(m_an);
  if constexpr (POST) ap.clear(m_ap);
  if constexpr (GATE) ag.clear(nullptr);
  u16x8_any wn[V], wp[POST ? V : 1], gv[GATE ? V : 1];
  if constexpr (AHEAD) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      wn[v] = row8<WHOLE>(p.weight, col(v), K);
      if constexpr (POST) wp[v] = row8<WHOLE>(p.post, col(v), K);
    }
  }
  GradRow<V, T> next;
  if constexpr (AHEAD) load(next, first);
  int held = -1;  // the group whose gate is in gv
  for (int row = first; row < end; ++row) {
    const int grp = GATE ? row / p.rows_per_gate : 0;
    const uint16_t* const gate = GATE ? p.gate + (int64_t)grp * p.ldgate : nullptr;
    const float rs = p.rstd[row], ry = POST ? p.rstd[(int64_t)p.M + row] : 1.f;
    if constexpr (GATE && AHEAD) {
      if (grp != held) {
        held = grp;
#pragma unroll
        for (int v = 0; v < V; ++v) gv[v] = row8<WHOLE>(gate, col(v), K);
      }
    }
    GradRow<V, T> cur;
    if constexpr (AHEAD) {
      cur = next;
      if (row + 1 < end) load(next, row + 1);
    } else {
      load(cur, row);
    }
    float s[V][8], t[V][8];        // s: s rs
    float q[3] = {0.f, 0.f, 0.f};  // sum e s, sum q (ds + rs e), sum q s
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float a[8];
      if constexpr (AHEAD) {
        stay_packed(wn[v]);
        if constexpr (POST) stay_packed(wp[v]);
        if constexpr (GATE) stay_packed(gv[v]);
      } else {
        __builtin_amdgcn_sched_barrier(0);
        wn[v] = row8<WHOLE>(p.weight, col(v), K);
        if constexpr (POST) wp[v] = row8<WHOLE>(p.post, col(v), K);
        if constexpr (GATE) gv[v] = row8<WHOLE>(gate, col(v), K);
      }
      gate8<GATE>(gv[GATE ? v : 0], p.scale, a);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float yi = POST ? value(cur.y[v], i) * ry : value(cur.y[v], i);
        float pi = yi;
        if constexpr (POST) pi = yi * value(wp[v], i);
        s[v][i] = fmaf(a[i], pi, value(cur.h[v], i)) * rs;
        const float e = value(cur.dn[v], i) * value(wn[v], i);
        t[v][i] = fmaf(rs, e, value(cur.ds[v], i));
        q[0] = fmaf(e, s[v][i], q[0]);
        if constexpr (POST) {
          const float w = a[i] * value(wp[v], i) * yi;
          q[1] = fmaf(w, t[v][i], q[1]);
          q[2] = fmaf(w, s[v][i], q[2]);
        }
      }
    }
    group_sum(q, sums[row & 1]);
    const float k = rs * (q[0] * rk);            // of s in t
    const float ky = fmaf(-k, q[2], q[1]) * rk;  // of y ry in f
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t c = col(v);
      float a[8], o[8];
      stay_packed(cur.y[v]);
      if constexpr (AHEAD) {
        stay_packed(cur.dn[v]);
        if constexpr (POST) stay_packed(wp[v]);
        if constexpr (GATE) stay_packed(gv[v]);
      } else {
        __builtin_amdgcn_sched_barrier(0);
        cur.dn[v] = row8<WHOLE>(p.dn + (int64_t)row * p.lddn, c, K);
        if constexpr (POST) wp[v] = row8<WHOLE>(p.post, c, K);
        if constexpr (GATE) gv[v] = row8<WHOLE>(gate, c, K);
      }
      gate8<GATE>(gv[GATE ? v : 0], p.scale, a);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float yi = POST ? value(cur.y[v], i) * ry : value(cur.y[v], i);
        t[v][i] = fmaf(-k, s[v][i], t[v][i]);
        an.fma_to(v, i, value(cur.dn[v], i), s[v][i]);
        const float u = a[i] * t[v][i];
        if constexpr (POST) {
          const float w = value(wp[v], i);
          ap.fma_to(v, i, u, yi);
          if constexpr (GATE) ag.fma_to(v, i, p.scale * t[v][i], yi * w);
          o[i] = ry * fmaf(-ky, yi, u * w);
        } else {
          if constexpr (GATE) ag.fma_to(v, i, p.scale * t[v][i], yi);
          o[i] = u;
        }
      }
      an.done(m_an, v);
      if constexpr (POST) ap.done(m_ap, v);
      put_row8<WHOLE>(static_cast<T*>(p.dh) + (int64_t)row * p.lddh, c, K, t[v]);
      put_row8<WHOLE>(p.dy + (int64_t)row * p.lddy, c, K, o);
    }
    if constexpr (GATE) {
      // the group's last row here: a whole group's sums are final
      if (row + 1 == end || (row + 1) % p.rows_per_gate == 0) {
        const bool before = grp * p.rows_per_gate < first;
        const bool after = (row + 1) % p.rows_per_gate != 0;
        float* const o = !before && !after ? p.dgate + (int64_t)grp * K
                                           : part + (before ? R.head : R.tail) * K;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float x[8];
          ag.get(nullptr, v, x);
          put_row8<WHOLE>(o, col(v), K, x);
        }
        ag.clear(nullptr);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float x[8];
    an.get(m_an, v, x);
    put_row8<WHOLE>(part, col(v), K, x);
    if constexpr (POST) {
      ap.get(m_ap, v, x);
      put_row8<WHOLE>(part + R.post * K, col(v), K, x);
    }
  }
}

// The workgroups' partial sums added, 64 columns per workgroup: job 0 dwn, then
// dwp, then the gate's groups that more than one workgroup shared (a group's
// first workgroup holds it as its tail, the others as their heads).  These have
// a job per group, or (by_end: more groups than workgroups) one for each
// workgroup but the last, which takes the group that begins there and goes on.
constexpr int kSumThreads = 1024;

__global__ void __launch_bounds__(kSumThreads) block_norm_sum_kernel(BlockNormGradParams p,
                                                                     int groups, int cblocks,
                                                                     int post, int gate,
                                                                     int by_end) {
  constexpr int NG = kSumThreads / 64;
  __shared__ float s[NG][64];
  const PartRows R = part_rows(post != 0, gate != 0);
  const int job = (int)(blockIdx.x / cblocks);
  const int l = (int)threadIdx.x & 63, g = (int)threadIdx.x >> 6;
  const int64_t c = (int64_t)(blockIdx.x % cblocks) * 64 + l;
  int w0 = 0, w1 = groups;  // the workgroups to add up
  int row = job, row0 = job;  // their row of partials, and the first one's
  float* out = job == 0 ? p.dweight : p.dpost;
  if (job > post) {
    int64_t grp = job - 1 - post;
    if (by_end) {
      const int64_t end = (grp + 1) * p.per_group, begin = end - p.per_group;
      grp = (end - 1) / p.rows_per_gate;
      if (grp * p.rows_per_gate < begin) return;  // (an earlier workgroup's)
    }
    w0 = (int)(grp * p.rows_per_gate / p.per_group);
    w1 = (int)(((grp + 1) * p.rows_per_gate - 1) / p.per_group) + 1;
    if (w1 - w0 == 1) return;  // (written whole)
    row = R.head;
    // (a group may begin with its workgroup, and is its tail then too)
    row0 = R.tail;
    out = p.dgate + grp * p.K;
  }
  const int per = (w1 - w0 + NG - 1) / NG;
  float a = 0.f;
  if (c < p.K) {
    const int e = min(w1, w0 + (g + 1) * per);
#pragma unroll 8
    for (int w = w0 + g * per; w < e; ++w)
      a += p.part[((int64_t)w * R.count + (w == w0 ? row0 : row)) * p.K + c];
  }
  s[g][l] = a;
  __syncthreads();
  if (g != 0 || c >= p.K) return;
#pragma unroll
  for (int i = 1; i < NG; ++i) a += s[i][l];
  out[c] = a;
}

// The fewest whole waves that hold a row in V chunks per thread.
int threads_of(int64_t K, int V) {
  const int64_t chunks = (K + 7) / 8;
  return (int)((chunks + 64 * V - 1) / (64 * V)) * 64;
}

template <int V, class T>
hipError_t launch_fwd(const BlockNormParams& p, hipStream_t s) {
  const dim3 grid(p.M), block(threads_of(p.K, V));
  if (p.post != nullptr)
    return enqueue(p.gate != nullptr ? block_norm_kernel<V, T, true, true>
                                     : block_norm_kernel<V, T, true, false>,
                   grid, block, s, p);
  return enqueue(p.gate != nullptr ? block_norm_kernel<V, T, false, true>
                                   : block_norm_kernel<V, T, false, false>,
                 grid, block, s, p);
}

template <int V, class T, bool WHOLE>
hipError_t launch_bwd(const BlockNormGradParams& p, int groups, hipStream_t s) {
  const dim3 grid(groups), block(threads_of(p.K, V));
  if (p.post != nullptr)
    return enqueue(p.gate != nullptr ? block_norm_bwd_kernel<V, T, true, true, WHOLE>
                                     : block_norm_bwd_kernel<V, T, true, false, WHOLE>,
                   grid, block, s, p);
  return enqueue(p.gate != nullptr ? block_norm_bwd_kernel<V, T, false, true, WHOLE>
                                   : block_norm_bwd_kernel<V, T, false, false, WHOLE>,
                 grid, block, s, p);
}

// Chunks per thread of the forward kernel.  Few rows: as few as possible, the
// call is latency.  Many: workgroups of about four waves (8192 x 5120, two /
// three / four chunks per thread: 77.9 / 67.8 / 69.8 us, 5.0 TB/s at best).
template <class T>
hipError_t launch_fwd_v(const BlockNormParams& p, hipStream_t s) {
  const int64_t chunks = (p.K + 7) / 8;
  const int64_t v = p.M < 512 ? (chunks + 1023) / 1024 : (chunks + 255) / 256;
  if (v <= 1) return launch_fwd<1, T>(p, s);
  if (v <= 2) return launch_fwd<2, T>(p, s);
  if (v <= 3) return launch_fwd<3, T>(p, s);
  return launch_fwd<4, T>(p, s);
}

// Chunks per thread of the backward kernel: one, while a workgroup holds the row
// so.
int bwd_chunks(int64_t K) { return K <= 8 * bwd_threads<1>() ? 1 : 4; }

template <class T>
hipError_t launch_bwd_v(const BlockNormGradParams& p, int groups, hipStream_t s) {
  const bool one = bwd_chunks(p.K) == 1;
  if (p.K % 8 == 0)
    return one ? launch_bwd<1, T, true>(p, groups, s) : launch_bwd<4, T, true>(p, groups, s);
  return one ? launch_bwd<1, T, false>(p, groups, s) : launch_bwd<4, T, false>(p, groups, s);
}

// Rows per workgroup of the backward kernel: one workgroup for each that the
// compute units hold at once, two each up to K = 4096 (8 waves) and one past it.
// Fewer rows each hide no more of a row's latency, and every workgroup writes
// its sums, which are then read once more (us, both kernels, with 256 / 512 /
// 1024 workgroups, post-norm and gate: 8192 x 512 50 / 33 / 38, 4096 x 2048 39 /
// 31 / 39, 8192 x 4096 112 / 96 / 120 (768), 2048 x 8192 54 / 65 / 91, 2048 x
// 13824 114 / 133 / 169).
int64_t per_group(int64_t M, int64_t K) {
  const int64_t groups = K <= 4096 ? 512 : 256;
  return ceil_div(M, M < groups ? M : groups);
}

}  // namespace

constexpr int64_t kNormMaxK = 16384;

bool block_norm_fits(int64_t M, int64_t K) {
  const int64_t chunks = (K + 7) / 8;
  return K <= kNormMaxK &&
         M * (chunks < 1024 ? (chunks + 63) / 64 * 64 : 1024) < (int64_t(1) << 32);
}

// (the sums have at most 2 + 511 jobs of 256 workgroups)
bool block_norm_bwd_fits(int64_t K) { return K <= kNormMaxK; }

size_t block_norm_bwd_bytes(int64_t M, int64_t K, bool post, bool gate) {
  const int64_t groups = ceil_div(M, per_group(M, K));
  return (size_t)(groups * part_rows(post, gate).count * K) * sizeof(float);
}

hipError_t launch_block_norm(const BlockNormParams& p, bool f32, hipStream_t s) {
  return f32 ? launch_fwd_v<float>(p, s) : launch_fwd_v<uint16_t>(p, s);
}

hipError_t launch_block_norm_bwd(BlockNormGradParams p, bool f32, hipStream_t s) {
  p.per_group = (int)per_group(p.M, p.K);
  const int groups = ceil_div(p.M, p.per_group);
  const hipError_t e =
      f32 ? launch_bwd_v<float>(p, groups, s) : launch_bwd_v<uint16_t>(p, groups, s);
  if (e != hipSuccess) return e;
  const int post = p.post != nullptr, gate = p.gate != nullptr;
  const int cblocks = ceil_div(p.K, 64);
  // groups of whole rows of one workgroup need no second pass
  const bool shared = gate && p.per_group % p.rows_per_gate != 0;
  const int gates = p.M / p.rows_per_gate, by_end = gates >= groups;
  const int jobs = 1 + post + (!shared ? 0 : by_end ? groups - 1 : gates);
  return enqueue(block_norm_sum_kernel, dim3((unsigned)(jobs * cblocks)), dim3(kSumThreads), s, p,
                 groups, cblocks, post, gate, by_end);
}

}  // namespace tgemm
