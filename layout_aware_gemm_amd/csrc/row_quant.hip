// Rows to 8-bit codes with one scale each, after an optional residual sum
// and RMS norm:
//   h = bf16(x + residual),  t = h * w,  T = max |t|,
//   scale = T / (127 sqrt(mean h^2 + eps)),  q = round(127 t / T).
// The codes are those of y / scale, y = t / sqrt(mean h^2 + eps): the norm's
// factor cancels, so they depend on exact products of bf16 values and on the
// row's maximum alone.  They are the correctly rounded quotients (ties to
// even): the candidate from a reciprocal is checked by its remainder, which
// fp32 holds exactly (127 t has 23 bits), so the same row gives the same
// codes whatever the order of the sums.  The mean of squares is summed in
// 64 bits: squares of bf16 values overflow fp32 from 1.8e19 on.
//
// One workgroup per row; the row stays in registers between the reduction
// and the codes, so each element moves once: 7 bytes per element with a
// residual, 3 without.  Bound: HBM bandwidth.
#include "ffn.h"
#include "row_vec.h"

namespace tgemm {
namespace {

// The row's constants for its codes.
struct RowCode {
  int shift;   // exponent that brings T into [1/2, 1)
  float top;   // T scaled so
  float rcp;   // about 127 / top
  bool none;   // the codes are 0: T = 0, or the row holds NaN or infinity
};

// The code of t in bits 0..7.
__device__ __forceinline__ uint32_t code_of(float t, const RowCode& c) {
#if defined(__HIP_DEVICE_COMPILE__)
  const float s = __builtin_amdgcn_ldexpf(t, c.shift);
  float k = rintf(s * c.rcp);
  const float rem = fmaf(-k, c.top, 127.f * s);  // exact
  // move to the neighbour when the remainder passes half of T, or is
  // exactly half and the candidate is odd (half is never 0, so one unit
  // below its bits is the next smaller value)
  const uint32_t half = __float_as_uint(0.5f * c.top) - ((uint32_t)(int)k & 1u);
  if ((__float_as_uint(rem) & 0x7fffffffu) > half) k += copysignf(1.f, rem);
  return (uint32_t)(int)k & 0xffu;
#else
  (void)t, (void)c;
  return 0;
#endif
}

__device__ __forceinline__ void wave_sum_max(double& ss, uint32_t& mx) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    ss += __shfl_xor(ss, o, 64);
    const uint32_t m = __shfl_xor(mx, o, 64);
    mx = m > mx ? m : mx;
  }
}

// Reduce over the workgroup (in wave order), then the row's constants.
template <bool NORM>
__device__ __forceinline__ RowCode row_code(const RowQuantParams& p, int row, double ss,
                                            uint32_t mx) {
  wave_sum_max(ss, mx);
  const int waves = (int)blockDim.x >> 6;
  if (waves > 1) {
    __shared__ double s_ss[16];
    __shared__ uint32_t s_mx[16];
    if ((threadIdx.x & 63) == 0) {
      s_ss[threadIdx.x >> 6] = ss;
      s_mx[threadIdx.x >> 6] = mx;
    }
    __syncthreads();
    ss = s_ss[0];
    mx = s_mx[0];
    for (int w = 1; w < waves; ++w) {
      ss += s_ss[w];
      mx = s_mx[w] > mx ? s_mx[w] : mx;
    }
  }
  RowCode c;
  const bool bad = mx >= 0x7f800000u;  // infinity or NaN
  c.none = bad || mx == 0;
  const float top = __uint_as_float(mx);
  if (threadIdx.x == 0) {
    double s = (double)top / 127.0;
    if constexpr (NORM) s /= sqrt(ss / (double)p.K + (double)p.eps);
    p.scale[row] = bad ? __uint_as_float(0x7fc00000u) : mx == 0 ? 0.f : (float)s;
  }
#if defined(__HIP_DEVICE_COMPILE__)
  c.shift = -__builtin_amdgcn_frexp_expf(top);
  c.top = __builtin_amdgcn_frexp_mantf(top);
#else
  c.shift = 0;
  c.top = top;
#endif
  c.rcp = 127.f / c.top;
  return c;
}

// |t| of the 8 elements into the maximum (as integers: NaN above infinity
// above every finite value) and h^2 into the sum.
template <bool NORM>
__device__ __forceinline__ void accumulate(const u16x8_any& h, const u16x8_any& w, double& ss,
                                           uint32_t& mx) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float t = (i & 1) ? hi_f(h.w[i >> 1]) : lo_f(h.w[i >> 1]);
    if constexpr (NORM) {
      const double d = (double)t;
      ss = fma(d, d, ss);
      t *= (i & 1) ? hi_f(w.w[i >> 1]) : lo_f(w.w[i >> 1]);
    }
    const uint32_t a = __float_as_uint(t) & 0x7fffffffu;
    mx = a > mx ? a : mx;
  }
}

template <bool NORM>
__device__ __forceinline__ u8x8_any codes8(const u16x8_any& h, const u16x8_any& w,
                                           const RowCode& c) {
  u8x8_any o;
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    uint32_t v = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 4 * d + e;
      float t = (i & 1) ? hi_f(h.w[i >> 1]) : lo_f(h.w[i >> 1]);
      if constexpr (NORM) t *= (i & 1) ? hi_f(w.w[i >> 1]) : lo_f(w.w[i >> 1]);
      v |= code_of(t, c) << (8 * e);
    }
    o.w[d] = c.none ? 0u : v;
  }
  return o;
}

__device__ __forceinline__ void store_codes(int8_t* p, int64_t c, int64_t n, const u8x8_any& v) {
  if (c + 8 <= n) {
    *reinterpret_cast<u8x8_any*>(p + c) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) p[c + i] = (int8_t)(v.w[i >> 2] >> ((i & 3) * 8));
  }
}

__device__ __forceinline__ u16x8_any add8(const u16x8_any& x, const u16x8_any& r) {
  u16x8_any h;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h.w[i] = pack_bf16x2(lo_f(x.w[i]) + lo_f(r.w[i]), hi_f(x.w[i]) + hi_f(r.w[i]));
  return h;
}

// V chunks of 8 elements per thread: rows of up to 8 V blockDim.x.
// (x, residual and sum may be the same rows: a thread writes only what it
// has read itself.)
template <int V, bool NORM, bool RES>
__global__ void __launch_bounds__(1024) row_quant_kernel(RowQuantParams p) {
  const int row = blockIdx.x, T = blockDim.x;
  const uint16_t* x = p.x + (int64_t)row * p.ldx;
  u16x8_any h[V], w[NORM ? V : 1];
  double ss = 0.0;
  uint32_t mx = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t c = ((int64_t)v * T + threadIdx.x) * 8;
    h[v] = u16x8_any{{0, 0, 0, 0}};
    if constexpr (NORM) w[v] = h[v];
    if (c < p.K) {
      h[v] = load8(x, c, p.K);
      if constexpr (NORM) w[v] = load8(p.weight, c, p.K);
      if constexpr (RES) h[v] = add8(h[v], load8(p.residual + (int64_t)row * p.ldr, c, p.K));
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t c = ((int64_t)v * T + threadIdx.x) * 8;
    if constexpr (RES) {
      if (c < p.K) store8(p.sum + (int64_t)row * p.lds, c, p.K, h[v]);
    }
    accumulate<NORM>(h[v], w[NORM ? v : 0], ss, mx);
  }
  const RowCode rc = row_code<NORM>(p, row, ss, mx);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t c = ((int64_t)v * T + threadIdx.x) * 8;
    if (c < p.K)
      store_codes(p.q + (int64_t)row * p.ldq, c, p.K, codes8<NORM>(h[v], w[NORM ? v : 0], rc));
  }
}

// Rows too long for registers: the second pass reads the row again.
template <bool NORM, bool RES>
__global__ void __launch_bounds__(1024) row_quant_long(RowQuantParams p) {
  const int row = blockIdx.x;
  const uint16_t* x = p.x + (int64_t)row * p.ldx;
  const uint16_t* again = RES ? p.sum + (int64_t)row * p.lds : x;
  double ss = 0.0;
  uint32_t mx = 0;
  u16x8_any w = {{0, 0, 0, 0}};
  for (int64_t c = threadIdx.x * 8; c < p.K; c += 8192) {
    u16x8_any h = load8(x, c, p.K);
    if constexpr (RES) {
      h = add8(h, load8(p.residual + (int64_t)row * p.ldr, c, p.K));
      store8(p.sum + (int64_t)row * p.lds, c, p.K, h);
    }
    if constexpr (NORM) w = load8(p.weight, c, p.K);
    accumulate<NORM>(h, w, ss, mx);
  }
  const RowCode rc = row_code<NORM>(p, row, ss, mx);
  for (int64_t c = threadIdx.x * 8; c < p.K; c += 8192) {
    const u16x8_any h = load8(again, c, p.K);
    if constexpr (NORM) w = load8(p.weight, c, p.K);
    store_codes(p.q + (int64_t)row * p.ldq, c, p.K, codes8<NORM>(h, w, rc));
  }
}

// The fewest whole waves that hold a row in V chunks per thread.
int threads_of(const RowQuantParams& p, int V) {
  const int64_t chunks = (p.K + 7) / 8;
  return (int)((chunks + 64 * V - 1) / (64 * V)) * 64;
}

hipError_t launch_quant8(const RowQuantParams& p, hipStream_t s) {
  return enqueue(row_quant_kernel<8, false, false>, dim3(p.M), dim3(threads_of(p, 8)), s, p);
}

template <int V>
hipError_t launch_v(const RowQuantParams& p, hipStream_t s) {
  const dim3 grid(p.M), block(threads_of(p, V));
  if (p.weight != nullptr && p.residual != nullptr)
    return enqueue(row_quant_kernel<V, true, true>, grid, block, s, p);
  if (p.weight != nullptr) return enqueue(row_quant_kernel<V, true, false>, grid, block, s, p);
  return enqueue(row_quant_kernel<V, false, false>, grid, block, s, p);
}

}  // namespace

// One workgroup per row, of at most 1024 threads: 2^32 - 1 in a launch.
bool row_quant_fits(const RowQuantParams& p) {
  const int64_t chunks = (p.K + 7) / 8;
  return p.M * (chunks < 1024 ? (chunks + 63) / 64 * 64 : 1024) < (int64_t(1) << 32);
}

// Chunks per thread.  Few rows: as few as possible, the call is latency.
// Many: workgroups of about four waves, which overlap best (us, MI355X:
// norm with residual 8192 x 5120, 1 / 2 / 3 / 4 chunks per thread 65.4 / 54.8
// / 53.2 / 58.5; codes alone 4096 x 13824, 2 / 4 / 8 chunks 44.9 / 38.0 /
// 36.1; norm 8 x 5120, 1 / 2 / 4 chunks 4.3 / 4.7 / 5.4).  Eight chunks of a
// norm's two inputs would not fit the registers of a full workgroup.
hipError_t launch_row_quant(const RowQuantParams& p, hipStream_t s) {
  const int64_t chunks = (p.K + 7) / 8;
  const int64_t v = p.M < 512 ? (chunks + 1023) / 1024 : (chunks + 255) / 256;
  if (v <= 1) return launch_v<1>(p, s);
  if (v <= 2) return launch_v<2>(p, s);
  if (v <= 3) return launch_v<3>(p, s);
  if (p.weight == nullptr) {
    if (v > 4 && chunks <= 8192) return launch_quant8(p, s);
    if (chunks <= 4096) return launch_v<4>(p, s);
    return enqueue(row_quant_long<false, false>, dim3(p.M), dim3(1024), s, p);
  }
  if (chunks <= 4096) return launch_v<4>(p, s);
  if (p.residual != nullptr)
    return enqueue(row_quant_long<true, true>, dim3(p.M), dim3(1024), s, p);
  return enqueue(row_quant_long<true, false>, dim3(p.M), dim3(1024), s, p);
}

}  // namespace tgemm
