// The gated product's two gradient products in one launch:
//   dX = G . W       [M][K],  G = dGU [M][2F], W [2F][K]     (NN)
//   dW = G^T . X     [2F][K], X [M][K]                       (TN)
// with 256x256 or 128x128 tiles on the library's NN and TN loops.
//
// Why one launch: dX has few, long tiles (K dimension 2F) and dW many short
// ones (K dimension M).  Alone, dX's last round leaves most compute units
// idle for a whole tile (4096 x 13824 x 5120: 320 tiles on 256 units, 1.38
// ms where 1.25 rounds of work would take 0.86); launched together with the
// longer tiles first, the short ones fill the gap.
//
// Edges need no loop of their own.  G lives in the workspace, padded: rows
// M .. round64(M) - 1 and columns 2F .. round64(2F) - 1 are zero, so the K
// dimension of either product is whole k-steps of G, and G's tiles may read
// on to whole tiles.  W and X are read through buffers that end with them:
// past their last row, the padded part of the K dimension, they read 0; past
// a row's end they read on into the next row, which only reaches output
// columns that are not stored.
#include "ffn.h"
#include "gemm_kernel.h"

namespace tgemm {
namespace {

// Store a wave's block of a T x T tile, a quarter of it (accumulator layout
// as in the GEMM's epilogues) through LDS words of its own, 32 rows at a
// time: rows leave as 128 to 512 contiguous bytes, and each accumulator is
// used in one place only.  (Stored from registers under the tests for the
// edge and the type, they were copied out of the matrix cores' registers all
// at once, and some of them through scratch.)  With 8 words of padding per
// row the two halves of a wave, four rows apart, write to different halves of
// the banks.
template <int T>
constexpr int out_row() {
  return T / 2 + 8;
}

template <int T>
__device__ __forceinline__ void store_block(const GemmParams& p, void* C, int64_t ldc, bool f32,
                                            const f32x16_t (&acc)[T / 64][T / 64], float* st,
                                            int row0, int col0, int lane) {
  constexpr int F = T / 64, LD = out_row<T>();
  constexpr int LPR = T / 8, RPI = 64 / LPR;  // lanes per row, rows per pass on the way out
  const int h = lane >> 5, lc = lane & 31;
  const int cl = 4 * (lane % LPR), c = col0 + cl;  // this lane's four columns
  const int n = p.N - c;                           // of which so many exist
#pragma unroll
  for (int i = 0; i < F; ++i) {
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
      for (int j = 0; j < F; ++j)
        st[(8 * (r >> 2) + 4 * h + (r & 3)) * LD + j * 32 + lc] = acc[i][j][r];
    wave_lds_order();
#pragma unroll
    for (int q = 0; q < 32 / RPI; ++q) {
      const int rl = q * RPI + lane / LPR, row = row0 + i * 32 + rl;
      const float4 v = *reinterpret_cast<const float4*>(st + rl * LD + cl);
      if (row >= p.M || n <= 0) continue;
      const float e[4] = {v.x, v.y, v.z, v.w};
      const int64_t off = (int64_t)row * ldc + c;
      if (f32)
        put4(static_cast<float*>(C) + off, e, n);
      else
        put4(static_cast<uint16_t*>(C) + off, e, n);
    }
    wave_lds_order();
  }
}

// One tile of one product: dX (NN) or dW (TN).
template <int kT, bool DW>
__device__ __forceinline__ void grad_tile(const GemmParams& p, int bid, bool f32, uint16_t* lds) {
  constexpr int FM = kT / 64, FN = kT / 64, SA = kT * kBK;
  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int h = lane >> 5, lc = lane & 31;
  int tile, ks, tm, tn;
  xcd_remap(bid, p.tilesM * p.tilesN * p.splitk, p.splitk, tile, ks);
  tile_coords(tile, p.tilesM, p.tilesN, p.groupM, tm, tn);
  const int m0 = tm * kT, n0 = tn * kT;
  const int kbeg = ks * p.kchunk;
  const int nk = (min(p.K, kbeg + p.kchunk) - kbeg) / kBK;
  f32x16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  const int a_base = (wm * (kT / 2) + lc) * kBK;
  const int b_base = SA + (wn * (kT / 2) + lc) * kBK;
  int xo[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) xo[s] = ((2 * s + h) ^ swz(lc)) << 3;
  if constexpr (DW)
    reg2_mainloop<kT, kT, FM, FN, false, false, false, true>(p, m0, n0, kbeg, nk, lds, nullptr,
                                                             nullptr, nullptr, tid, a_base, b_base,
                                                             xo, acc);
  else
    mix_mainloop<kT, kT, FM, FN, true, false, true>(p, m0, n0, kbeg, nk, lds, lds + 3 * SA, tid,
                                                    wave, lane, a_base, b_base - SA, xo, acc);
  void* C = p.C;
  int64_t ldc = p.ldc;
  if (p.splitk > 1) {
    C = p.ws + (int64_t)ks * p.M * p.N;
    ldc = p.N;
    f32 = true;
  }
  __syncthreads();  // the stages become the rows' buffer
  store_block<kT>(p, C, ldc, f32, acc, reinterpret_cast<float*>(lds) + wave * 32 * out_row<kT>(),
                  m0 + wm * (kT / 2), n0 + wn * (kT / 2), lane);
}

// 64 columns of a sum over rows: four groups of rows, added in order.
__device__ __forceinline__ void column_sum(const ColumnSum& j, int b, float* s) {
  const int l = (int)threadIdx.x & 63, g = (int)threadIdx.x >> 6;
  const int64_t c = (int64_t)b * 64 + l;
  const int per = (j.rows + 3) / 4, end = min(j.rows, (g + 1) * per);
  float a = 0.f;
  if (c < j.cols) {
#pragma unroll 4
    for (int i = g * per; i < end; ++i) a += j.part[i * j.cols + c];
  }
  s[g * 64 + l] = a;
  __syncthreads();
  if (g == 0 && c < j.cols) j.out[c] = s[l] + s[64 + l] + s[128 + l] + s[192 + l];
}

// Workgroups 0 .. nfirst - 1 (a multiple of 8, so that a product's tiles
// keep their XCDs) take the product with the longer tiles, dW if wfirst.
// f32x, f32w: the output types (K chunks are fp32).  The workgroups after the
// products' ntiles take the column sums, in the compute units' last gaps.
template <int kT>
__global__ void __launch_bounds__(kThreads, kT == 128 ? 2 : 1) gated_bwd_kernel(GemmParams px, GemmParams pw,
                                                                int nfirst, int wfirst, int f32x,
                                                                int f32w, int ntiles, ColumnSum sum) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[5 * kT * kBK];
  const int b = blockIdx.x;
  if (b >= ntiles) {
    column_sum(sum, b - ntiles, reinterpret_cast<float*>(lds));
    return;
  }
  const bool w = (b < nfirst) == (wfirst != 0);
  const int l = b < nfirst ? b : b - nfirst;
  // (workgroups past a product's last tile are the padding to a multiple of 8)
  if (w) {
    if (l < pw.tilesM * pw.tilesN * pw.splitk) grad_tile<kT, true>(pw, l, f32w != 0, lds);
  } else {
    if (l < px.tilesM * px.tilesN * px.splitk) grad_tile<kT, false>(px, l, f32x != 0, lds);
  }
}

// Sums of the K chunks' partials [split][M][N] of up to two products in one
// launch, in ascending chunk order, four columns per thread.
struct SumJob {
  const float* ws;
  int split, M, N;
  void* C;
  int64_t ldc;
  int f32;
  int per_row;  // workgroups per row
};

__global__ void __launch_bounds__(kThreads) bwd_sum_kernel(SumJob x, SumJob w, int xblocks) {
  const bool second = (int)blockIdx.x >= xblocks;
  const SumJob& j = second ? w : x;
  const int b = second ? (int)blockIdx.x - xblocks : (int)blockIdx.x;
  const int row = b / j.per_row;
  const int c = ((b - row * j.per_row) * kThreads + (int)threadIdx.x) * 4;
  const int n = min(4, j.N - c);
  if (n <= 0) return;
  const int64_t slice = (int64_t)j.M * j.N;
  const float* p = j.ws + (int64_t)row * j.N + c;
  float a[4] = {0.f, 0.f, 0.f, 0.f};
  for (int q = 0; q < j.split; ++q, p += slice) {
    if (n == 4) {
      const x4_any<float> t = *reinterpret_cast<const x4_any<float>*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] += t.v[i];
    } else {
      for (int i = 0; i < n; ++i) a[i] += p[i];
    }
  }
  const int64_t o = (int64_t)row * j.ldc + c;
  if (j.f32)
    put4(static_cast<float*>(j.C) + o, a, n);
  else
    put4(static_cast<uint16_t*>(j.C) + o, a, n);
}

int64_t sum_job(const GemmParams& p, bool f32, SumJob* j) {
  *j = {p.ws, p.splitk, p.M, p.N, p.C, p.ldc, f32 ? 1 : 0, ceil_div(p.N, 4 * kThreads)};
  return p.splitk > 1 ? (int64_t)p.M * j->per_row : 0;
}

void set_split(GemmParams* p, int split) {
  const int steps = p->K / kBK;
  const int per = ceil_div(steps, split);
  p->kchunk = per * kBK;
  p->splitk = ceil_div(steps, per);
}

}  // namespace

int gated_bwd_plan(GemmParams* px, GemmParams* pw) {
  auto tiles = [&](int t) {
    double work = 0;  // k-steps of all tiles
    for (GemmParams* p : {px, pw}) {
      p->tilesM = ceil_div(p->M, t);
      p->tilesN = ceil_div(p->N, t);
      p->groupM = p->tilesM < 4 ? p->tilesM : (p->tilesM <= 8 ? p->tilesM : 4);
      work += (double)p->tilesM * p->tilesN * (p->K / kBK);
    }
    return work;
  };
  // Under 60 k-steps of 256x256 tiles per compute unit the smaller tiles win
  // (whole training steps, us, 256 against 128): 333 x 1000 x 520 (1.3) 45.3,
  // 31.0; 1000 x 2048 x 1024 (8) 72, 58; 768 x 4096 x 4096 (48) 232, 214; 128
  // x 13824 x 5120 (51) 345, 296.  Then they tie (1024 x 4096 x 4096, 64: 267,
  // 269; 256 x 13824 x 5120, 68: 412, 416) and lose (2048 x 8192 x 2048, 128:
  // 492, 540).
  double total = tiles(256);
  const int t = total < 60 * 256 ? 128 : 256;
  if (t == 128) total = tiles(128);
  // Split the K dimension of a product whose tiles are longer than an even
  // share of all the work (two small tiles run per compute unit), in chunks
  // of at least kMinSteps k-steps (333 x 1000 x 520: with 4, 6, 8 and 12 the
  // step takes 37, 31, 31 and 33 us; 64 x 512 x 256: 17.6, 18.6, 18.9, 23).
  constexpr int kMinSteps = 6;
  const double even = total / (t == 128 ? 512 : 256);
  const double share = even > kMinSteps ? even : kMinSteps;
  for (GemmParams* p : {px, pw}) {
    const double n = (p->K / kBK) / share;
    set_split(p, n < 1.5 ? 1 : n > 64 ? 64 : (int)(n + 0.5));
  }
  return t;
}

namespace {
int64_t grid_of(const GemmParams& p) { return (int64_t)p.tilesM * p.tilesN * p.splitk; }
}  // namespace

bool gated_bwd_fits(const GemmParams& px, const GemmParams& pw, int64_t sum_cols) {
  return grid_of(px) + grid_of(pw) + 8 + ceil_div(sum_cols, 64) <= kMaxWorkgroups;
}

hipError_t launch_gated_bwd(int tile, const GemmParams& px, const GemmParams& pw, bool f32x,
                            bool f32w, const ColumnSum& sum, hipStream_t s) {
  const int64_t nx = grid_of(px), nw = grid_of(pw);
  const int wfirst = pw.kchunk > px.kchunk;
  const int nfirst = (int)(((wfirst ? nw : nx) + 7) / 8 * 8);
  const int ntiles = (int)(nfirst + (wfirst ? nx : nw));
  const int sums = sum.part != nullptr ? ceil_div(sum.cols, 64) : 0;
  const dim3 grid((unsigned)(ntiles + sums)), block(kThreads);
  const hipError_t e = enqueue(tile == 128 ? gated_bwd_kernel<128> : gated_bwd_kernel<256>, grid,
                               block, s, px, pw, nfirst, wfirst, f32x ? 1 : 0, f32w ? 1 : 0, ntiles, sum);
  // Only a product of at most 341 tiles is split (its K is 1.5 shares or
  // more), so the sums' grid stays under 2^16 workgroups.
  SumJob jx, jw;
  const int64_t bx = sum_job(px, f32x, &jx), bw = sum_job(pw, f32w, &jw);
  if (e != hipSuccess || bx + bw == 0) return e;
  return enqueue(bwd_sum_kernel, dim3((unsigned)(bx + bw)), block, s, jx, jw, (int)bx);
}

}  // namespace tgemm
