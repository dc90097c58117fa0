// Host entries of the feed-forward operators: 8-bit products, gated and linear
// products and their gradients, the row quantiser.  Validation (validate.cpp),
// choice of kernel, workspace, launches.
#include "ffn.h"

#include <stdio.h>

#include "tgemm.h"

using namespace tgemm;

namespace tgemm {
namespace {

inline bool is_n(char t) { return t == 'N' || t == 'n'; }

int status_of(hipError_t e) { return e == hipSuccess ? TGEMM_OK : TGEMM_ERR_HIP; }

constexpr size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// The copy offsets of a tile (at most 256 rows) stay below 2^31 bytes.
inline bool stride_fits(int64_t ld_bytes) { return ld_bytes < (int64_t(1) << 23); }

// Kernel and tiles of a product whose operands are aligned.
struct RowsPlan {
  bool skinny;
  int tile;
  int tail;        // -1, or the tile of the output columns from tail_col on
  int tail_col;
};

inline int out_cols(int tile, bool gate) { return gate ? rows_tile_n(tile) / 2 : rows_tile_n(tile); }

// The tile grid over output columns col0 .. end - 1.
void set_tile(RowsParams* p, bool gate, int tile, int col0, int end) {
  p->col0 = col0;
  p->tilesM = ceil_div(p->M, rows_tile_m(tile));
  p->tilesN = ceil_div(end - col0, out_cols(tile, gate));
  p->groupM = p->tilesM < 4 ? p->tilesM : (p->tilesM <= 8 ? p->tilesM : 4);
}

// Time of a grid in us: rounds of 256 workgroups (one per compute unit), each
// a fixed part (the pipeline's fill, the epilogue) and the k-steps, plus the
// second pass over the partial sums of a split K.  A round of 128x128 tiles
// takes 6 us and 2.9 us per KB of K (gated 2048 wide, 128 rows: 1 KB 8.9, 2
// KB 11.5, 4 KB 18.2, 8 KB 29.4; plain 5120 x 13.5 KB 45), the other tiles
// 0.8 (64x128), 1.33 (128x256) and 1.95 (256x256) of it (gated 13824 x 5120,
// us for 64x128 / 128x128 / 128x256 / 256x256 tiles: 256 rows 101 / 66.9 /
// 51.4 / 65.0 int8, 170 / 114 / 89 / 121 bf16; 512 rows 163 / 123 / 92 / 70
// and 272 / 211 / 158 / 125).  256x192 tiles (linear products) take 0.89 of a
// 256x256 round (us, cold operands, as many rounds of either: 2047 x 5120 x
// 13824 262 / 294, one; 4096 x 6144 x 4096 184 / 204, two; 4096 x 9216 x 4096 277
// / 310, three).  A round more than 256x256 tiles, or than these and smaller
// ones in their last round, take is a loss (us, the smaller tiles first: 4096 x
// 15360 x 4096 451 / 436, five and four; 8192 x 9216 x 1024 211 / 202, six and
// five; 1979 x 9280 x 1024 74 / 60 and 1437 x 13120 x 4096 172 / 158, two and one
// with a tail).
double grid_cost(RowsParams* p, bool gate, int tile, int split, int col0, int end) {
  constexpr double cost[5] = {1.95, 1.33, 1.0, 0.8, 1.74};
  set_tile(p, gate, tile, col0, end);
  const double round = cost[tile] * (6 + 2.9e-3 * p->K / split);
  const double sums = split > 1 ? 4 + 1.7e-6 * split * p->M * p->N : 0;
  return (double)(((int64_t)p->tilesM * p->tilesN * split + 255) / 256) * round + sums;
}

// linear: 256x192 tiles may be used.
RowsPlan plan_rows(RowsParams* p, bool gate, bool linear) {
  // Few rows of A: the kernel that streams B.  From 17 rows on a gated
  // weight wide enough for 64x128 tiles on most of the chip is faster there
  // (us tiles / streaming, int8 then bf16: 13824 x 5120, 16 rows 29.3 / 28.4,
  // 49.6 / 52.5; 64 rows 32.7 / 36.1, 56.0 / 65.9; 11008 x 4096, 17 rows 18.1 /
  // 20.8, 38.2 / 43.2; 64 rows 19.9 / 24.4, 43.2 / 50.1), a smaller one is not
  // (8192 x 4096, 32 rows 15.3 / 13.1, 38.9 / 31.7), nor a plain one (32000 x
  // 4096 int8, 48 rows 33.6 / 32.5).
  RowsPlan r = {p->M <= kSkinnyRows, kRows256, -1, 0};
  p->split = 1;
  const int end = gate ? p->F : p->N;
  if (r.skinny && p->M > 16 && gate && p->F >= 160 * 64) {
    r.skinny = false;
    r.tile = kRows64;
    set_tile(p, gate, kRows64, 0, end);
  } else if (!r.skinny) {
    double best = grid_cost(p, gate, kRows256, 1, 0, end);
    // 256x256 tiles whose last round is short: give its columns to smaller
    // tiles, which need less than a whole round (a second launch: 4 us).
    // Gated products, us with and without: 513 x 13824 x 5120 102 / 115 int8,
    // 178 / 208 bf16; 4096 x 2100 x 5120 96 / 122, 166 / 213; 2047 x 13824 x
    // 5120, where the chip runs at its power limit, 278 / 279.
    const int cols = (int)((int64_t)p->tilesM * p->tilesN / 256 * 256 / p->tilesM);
    if (cols > 0 && cols < p->tilesN) {
      const int col = cols * out_cols(kRows256, gate);
      const double head = grid_cost(p, gate, kRows256, 1, 0, col) + 4;
      for (int t = kRows128x256; t <= kRows64; ++t) {
        const double c = head + grid_cost(p, gate, t, 1, col, end);
        if (c < best) {
          best = c;
          r.tail = t;
          r.tail_col = col;
        }
      }
    }
    if (linear) {
      const double c = grid_cost(p, gate, kRows256x192, 1, 0, end);
      if (c < best) {
        best = c;
        r.tile = kRows256x192;
        r.tail = -1;
      }
    }
    for (int t = kRows128x256; t <= kRows64; ++t) {
      const double c = grid_cost(p, gate, t, 1, 0, end);
      if (c < best) {
        best = c;
        r.tile = t;
        r.tail = -1;
        p->split = 1;
      }
      // Few small tiles: split K to give every compute unit a workgroup, in
      // chunks of at least 2048 bytes (5120 x 13824 int8: 128 rows, 128x128
      // tiles 45 us whole, 26 in 6 chunks with the second pass, 64x128 tiles
      // 23.5 in 3; 512 rows, 128x128 tiles 51.4 whole, 128x256 tiles 46.6 in 3).
      const int64_t fill = 256 / ((int64_t)p->tilesM * p->tilesN), by_k = p->K / 2048;
      const int split = (int)(fill < by_k ? fill : by_k);
      if (split < 2) continue;
      const double cs = grid_cost(p, gate, t, split, 0, end);
      if (cs < best) {
        best = cs;
        r.tile = t;
        r.tail = -1;
        p->split = split;
      }
    }
    set_tile(p, gate, r.tile, 0, r.tail < 0 ? end : r.tail_col);
  }
  p->kchunk = ceil_div(ceil_div(p->K, p->split), 128) * 128;
  p->split = ceil_div(p->K, p->kchunk);  // no empty chunks
  return r;
}

bool grid_fits(const RowsParams& p, const RowsPlan& r, bool gate) {
  // (the few-row kernel: at most one workgroup of 512 threads per 16 outputs)
  if (r.skinny) return ceil_div(gate ? p.F : p.N, 16) <= kMaxWorkgroups / 2;
  if (r.tail >= 0) {
    RowsParams q = p;
    set_tile(&q, gate, r.tail, r.tail_col, gate ? p.F : p.N);
    if ((int64_t)q.tilesM * q.tilesN > kMaxWorkgroups) return false;
  }
  if (p.split > 1 && !rows_finish_fits(p, gate)) return false;
  return (int64_t)p.tilesM * p.tilesN * p.split <= kMaxWorkgroups;
}

hipError_t launch_rows(int type, const RowsParams& p, const RowsPlan& r, int epi, bool gate,
                       hipStream_t s) {
  if (r.skinny) return launch_rows_skinny(type, epi, p, s);
  const int e = p.split > 1 ? (int)kRowsPart : epi;
  hipError_t h = launch_rows_gemm(type, r.tile, e, gate, p, s);
  if (h == hipSuccess && r.tail >= 0) {
    RowsParams q = p;
    set_tile(&q, gate, r.tail, r.tail_col, gate ? p.F : p.N);
    h = launch_rows_gemm(type, r.tail, e, gate, q, s);
  }
  return h != hipSuccess || p.split == 1 ? h : launch_rows_finish(type, epi, p, s);
}

void say_rows(const char* what, const RowsParams& p, const RowsPlan& r) {
  if (verbose())
    fprintf(stderr, "tgemm: %s M=%d N=%d K=%d bytes tile=%dx%d split=%d tail=%d\n", what, p.M, p.N,
            p.K, r.skinny ? 0 : rows_tile_m(r.tile), r.skinny ? 0 : rows_tile_n(r.tile), p.split,
            r.tail < 0 ? 0 : rows_tile_n(r.tail));
}

// ----------------------------------------------------------------------
// Workspace of one call.  bytes >= 0: the caller's buffer of that size (a
// call that needs more fails before anything is enqueued); bytes < 0: the
// library's own per-stream buffer, which a stream under capture does not
// get: a graph's memory is the caller's here.
// query set: report the need and launch nothing.
// ----------------------------------------------------------------------
struct CallSpace {
  void* ptr;
  int64_t bytes;
  int64_t* query;
};

constexpr int kQueried = 1;  // take_workspace: the need was reported

int take_workspace(const CallSpace& c, hipStream_t s, size_t need, Workspace* w) {
  if (c.query != nullptr) {
    *c.query = (int64_t)need;
    return kQueried;
  }
  if (need == 0) return TGEMM_OK;
  if (c.bytes >= 0) {
    if (c.ptr == nullptr || (size_t)c.bytes < need) return TGEMM_ERR_WORKSPACE_LIMIT;
    if ((reinterpret_cast<uintptr_t>(c.ptr) & 15) != 0) return TGEMM_ERR_INVALID_ARG;
    w->ptr = c.ptr;
    return TGEMM_OK;
  }
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  if (s != nullptr && hipStreamIsCapturing(s, &cs) == hipSuccess &&
      cs != hipStreamCaptureStatusNone)
    return TGEMM_ERR_WORKSPACE_LIMIT;
  return get_workspace(kWsCached, s, need, w);
}

// p holds everything but the operands' final addresses.  Operands that the
// direct-copy kernels cannot read in place -- not K-contiguous, or with
// rows off 16-byte boundaries -- are copied into the workspace first.
int run_i8(char ta, char tb, const void* A, int64_t lda, const void* B, int64_t ldb, RowsParams p,
           int epi, bool gate, const CallSpace& space, hipStream_t s) {
  const int K = p.K;
  const int Kp = ceil_div(K, 16) * 16;
  // (the stride of a single row is never used)
  if (is_n(ta) && p.M == 1) lda = Kp;
  if (!is_n(tb) && p.N == 1) ldb = Kp;
  const bool packA = !is_n(ta) || !rows_aligned(A, lda, K) || !stride_fits(lda);
  const bool packB = is_n(tb) || !rows_aligned(B, ldb, K) || !stride_fits(ldb);
  p.K = packA || packB ? Kp : K;
  const RowsPlan r = plan_rows(&p, gate, false);
  PackRows ca = {A, lda, is_n(ta), p.M, K, nullptr, p.M, Kp};
  PackRows cb = {B, ldb, !is_n(tb), p.N, K, nullptr, p.N, Kp};
  if (!grid_fits(p, r, gate) || (packA && !pack_rows_fits(ca, 1)) ||
      (packB && !pack_rows_fits(cb, 1)))
    return TGEMM_ERR_UNSUPPORTED;
  const size_t bytesA = packA ? round256((size_t)p.M * Kp) : 0;
  const size_t bytesB = packB ? round256((size_t)p.N * Kp) : 0;
  const size_t bytesP = p.split > 1 ? (size_t)p.split * p.M * p.N * sizeof(int) : 0;
  Workspace w;
  const int st = take_workspace(space, s, bytesA + bytesB + bytesP, &w);
  if (st != TGEMM_OK) return st;
  say_rows(gate ? "gated i8" : "i8", p, r);
  char* ws = static_cast<char*>(w.ptr);
  p.A = static_cast<const char*>(A);
  p.B = static_cast<const char*>(B);
  p.lda = lda;
  p.ldb = ldb;
  hipError_t e = hipSuccess;
  if (packA) {
    ca.out = ws;
    e = launch_pack_rows(ca, 1, s);
    p.A = ws;
    p.lda = Kp;
  }
  if (packB && e == hipSuccess) {
    cb.out = ws + bytesA;
    e = launch_pack_rows(cb, 1, s);
    p.B = ws + bytesA;
    p.ldb = Kp;
  }
  if (bytesP) p.part = ws + bytesA + bytesB;
  if (e == hipSuccess) e = launch_rows(kRowsI8, p, r, epi, gate, s);
  release_workspace(w);
  return status_of(e);
}

inline int64_t round_up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

// bf16 product, gated or linear: p holds everything but the operands and K.
// Operands that the kernels cannot read in place -- not
// K-contiguous, or with rows off 16-byte boundaries -- are copied into the
// workspace first.  (The copy costs a read and a write of the operand; the
// alternative, the library's GEMM in the operand's own layout, has to write
// and re-read the whole fp32 [M][2F] product instead, and runs rows off
// 16-byte boundaries at a third of the rate.)
int run_bf16(char ta, char tb, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb,
             RowsParams p, int epi, bool gate, const CallSpace& space, hipStream_t s) {
  const int64_t Kp = round_up(K, 8);
  if (Kp >= int64_t(1) << 30) return TGEMM_ERR_UNSUPPORTED;
  // (the stride of a single row is never used)
  if (is_n(ta) && p.M == 1) lda = Kp;
  if (!is_n(tb) && p.N == 1) ldb = Kp;
  // (a linear product of few rows reads rows of any alignment, if the weight is
  // K-contiguous)
  const bool any = !gate && p.M <= kSkinnyRows && !is_n(tb) && stride_fits(2 * ldb);
  const bool packA =
      !is_n(ta) || !(any || rows_aligned(A, 2 * lda, 2 * K)) || !stride_fits(2 * lda);
  const bool packB = is_n(tb) || !(any || rows_aligned(B, 2 * ldb, 2 * K)) || !stride_fits(2 * ldb);
  if ((packA || packB) && !stride_fits(2 * Kp)) return TGEMM_ERR_UNSUPPORTED;
  p.K = (int)(2 * (any ? K : Kp));
  const RowsPlan r = plan_rows(&p, gate, epi == kRowsLinear);
  PackRows ca = {A, lda, is_n(ta), p.M, (int)K, nullptr, p.M, Kp};
  PackRows cb = {B, ldb, !is_n(tb), p.N, (int)K, nullptr, p.N, Kp};
  if (!grid_fits(p, r, gate) || (packA && !pack_rows_fits(ca, 2)) ||
      (packB && !pack_rows_fits(cb, 2)))
    return TGEMM_ERR_UNSUPPORTED;
  const size_t bytesA = packA ? round256((size_t)p.M * Kp * 2) : 0;
  const size_t bytesB = packB ? round256((size_t)p.N * Kp * 2) : 0;
  const size_t bytesP = p.split > 1 ? (size_t)p.split * p.M * p.N * sizeof(float) : 0;
  Workspace w;
  const int st = take_workspace(space, s, bytesA + bytesB + bytesP, &w);
  if (st != TGEMM_OK) return st;
  say_rows(gate ? "gated bf16" : "linear", p, r);
  char* const ws = static_cast<char*>(w.ptr);
  p.A = static_cast<const char*>(A);
  p.B = static_cast<const char*>(B);
  p.lda = 2 * lda;
  p.ldb = 2 * ldb;
  hipError_t e = hipSuccess;
  if (packA) {
    ca.out = ws;
    e = launch_pack_rows(ca, 2, s);
    p.A = ws;
    p.lda = 2 * Kp;
  }
  if (packB && e == hipSuccess) {
    cb.out = ws + bytesA;
    e = launch_pack_rows(cb, 2, s);
    p.B = ws + bytesA;
    p.ldb = 2 * Kp;
  }
  if (bytesP) p.part = ws + bytesA + bytesB;
  if (e == hipSuccess) e = launch_rows(kRowsBf16, p, r, epi, gate, s);
  release_workspace(w);
  return status_of(e);
}

int run_gated(char ta, char tb, int64_t M, int64_t F, int64_t K, const void* A, int64_t lda,
              const void* B, int64_t ldb, int act, void* H, int64_t ldh, float* GU, int64_t ldgu,
              const CallSpace& space, hipStream_t s) {
  RowsParams p = {};
  p.M = (int)M;
  p.N = (int)(2 * F);
  p.F = (int)F;
  p.act = act;
  p.C = H;
  p.ldc = ldh;
  p.gu = GU;
  p.ldgu = ldgu;
  return run_bf16(ta, tb, K, A, lda, B, ldb, p, kRowsGated, true, space, s);
}

// The two gradient products of a bf16 product with N2 columns, given the
// gradient G [M][N2] of its sums: dA = G . op(B)^T and dB in one launch, which
// reads A and B as [M][K] and [N2][K] rows on 16-byte boundaries; others are
// copied first.  dB stored [K][N2] is the product with the operands exchanged,
// A^T . G; its first operand is then a zero-padded copy of A.
// grad(G, ldg, rows, part) enqueues the kernel that writes G into the
// workspace, zero-padded, and where db is set the partial column sums [strips]
// [N2], which the products' launch adds up there.
struct GradSource {
  bool fits;    // its grid is launchable
  float* db;
  int strips;
};

template <class Grad>
int run_backward(const char* what, char ta, char tb, int64_t M, int64_t N2, int64_t K,
                 const void* A, int64_t lda, const void* B, int64_t ldb, void* dA, int64_t ldda,
                 void* dB, int64_t lddb, bool f32, const GradSource& src, Grad&& grad,
                 const CallSpace& space, hipStream_t s) {
  const int64_t Kp = round_up(K, 8);
  const int64_t ldg = round_up(N2, 64), rows = round_up(M, 64);
  constexpr int64_t kLimit = int64_t(1) << 23;  // (32-bit copy offsets)
  if (Kp >= kLimit || ldg >= kLimit) return TGEMM_ERR_UNSUPPORTED;
  // (the stride of a single row is never used)
  if (is_n(ta) && M == 1) lda = Kp;
  if (!is_n(tb) && N2 == 1) ldb = Kp;
  const bool swap = is_n(tb);
  const bool packA = !is_n(ta) || swap || !rows_aligned(A, 2 * lda, 0) || lda >= kLimit;
  const bool packB = is_n(tb) || !rows_aligned(B, 2 * ldb, 0) || ldb >= kLimit;
  // tiles of 256 rows (columns) read on past the padding of G (and of A)
  const size_t bytesG = round256((size_t)(round_up(M, 256) * ldg + 256) * 2);
  const size_t bytesA = packA ? round256((size_t)(rows * Kp + 256) * 2) : 0;
  const size_t bytesB = packB ? round256((size_t)N2 * Kp * 2) : 0;
  GemmParams px = {}, pw = {};
  px.M = (int)M;
  px.N = (int)K;
  px.K = (int)ldg;
  px.kvb = (int)N2;
  px.lda = ldg;
  px.C = dA;
  px.ldc = ldda;
  pw.M = (int)(swap ? K : N2);
  pw.N = (int)(swap ? N2 : K);
  pw.K = (int)rows;
  pw.kvb = (int)M;
  pw.C = dB;
  pw.ldc = lddb;
  const int tile = gated_bwd_plan(&px, &pw);
  PackRows ca = {A, lda, is_n(ta), (int)M, (int)K, nullptr, (int)rows, Kp};
  PackRows cb = {B, ldb, !is_n(tb), (int)N2, (int)K, nullptr, (int)N2, Kp};
  const bool sums = src.db != nullptr;
  if (!gated_bwd_fits(px, pw, sums ? N2 : 0) || !src.fits || (packA && !pack_rows_fits(ca, 2)) ||
      (packB && !pack_rows_fits(cb, 2)))
    return TGEMM_ERR_UNSUPPORTED;
  const size_t bytesX =
      px.splitk > 1 ? round256((size_t)px.splitk * px.M * px.N * sizeof(float)) : 0;
  const size_t bytesW =
      pw.splitk > 1 ? round256((size_t)pw.splitk * pw.M * pw.N * sizeof(float)) : 0;
  const size_t bytesS = sums ? (size_t)src.strips * N2 * sizeof(float) : 0;
  Workspace w;
  const int st =
      take_workspace(space, s, bytesG + bytesA + bytesB + bytesX + bytesW + bytesS, &w);
  if (st != TGEMM_OK) return st;
  if (verbose())
    fprintf(stderr,
            "tgemm: %s backward %c%c M=%lld N=%lld K=%lld copies=%d,%d tile=%d split=%d,%d\n", what,
            ta, tb, (long long)M, (long long)N2, (long long)K, packA, packB, tile, px.splitk,
            pw.splitk);
  char* ws = static_cast<char*>(w.ptr);
  uint16_t* const G = reinterpret_cast<uint16_t*>(ws);
  ws += bytesG;
  float* const part =
      sums ? reinterpret_cast<float*>(ws + bytesA + bytesB + bytesX + bytesW) : nullptr;
  hipError_t e = grad(G, ldg, (int)rows, part);
  const void *Ar = A, *Br = B;  // [M][K], [2F][K] rows
  if (packA && e == hipSuccess) {
    ca.out = ws;
    e = launch_pack_rows(ca, 2, s);
    Ar = ws;
    lda = Kp;
  }
  ws += bytesA;
  if (packB && e == hipSuccess) {
    cb.out = ws;
    e = launch_pack_rows(cb, 2, s);
    Br = ws;
    ldb = Kp;
  }
  ws += bytesB;
  px.A = G;
  px.B = static_cast<const uint16_t*>(Br);
  px.ldb = ldb;
  px.ws = reinterpret_cast<float*>(ws);
  pw.A = swap ? static_cast<const uint16_t*>(Ar) : G;
  pw.lda = swap ? lda : ldg;
  pw.B = swap ? G : static_cast<const uint16_t*>(Ar);
  pw.ldb = swap ? ldg : lda;
  pw.ws = reinterpret_cast<float*>(ws + bytesX);
  if (e == hipSuccess) e = launch_gated_bwd(tile, px, pw, false, f32, {part, src.strips, N2, src.db}, s);
  release_workspace(w);
  return status_of(e);
}

// Gradient of the gated product, by way of dGU.
int run_gated_backward(char ta, char tb, int64_t M, int64_t F, int64_t K, const void* A,
                       int64_t lda, const void* B, int64_t ldb, const void* dH, int64_t lddh,
                       const void* GU, int64_t ldgu, bool gu_f32, int act, void* dA, int64_t ldda,
                       void* dB, int64_t lddb, bool f32, const CallSpace& space, hipStream_t s) {
  return run_backward(
      "gated", ta, tb, M, 2 * F, K, A, lda, B, ldb, dA, ldda, dB, lddb, f32,
      {gated_grad_fits(round_up(M, 64), F), nullptr, 0},
      [&](uint16_t* G, int64_t ldg, int rows, float*) {
        return launch_gated_grad(static_cast<const uint16_t*>(dH), lddh, GU, ldgu, gu_f32, (int)M,
                                 F, act, G, ldg, rows, ldg, s);
      },
      space, s);
}

// Gradient of the linear product, by way of dZ; db: its column sums.
int run_linear_backward(char ta, char tb, int64_t M, int64_t N, int64_t K, const void* A,
                        int64_t lda, const void* B, int64_t ldb, const void* dY, int64_t lddy,
                        const void* Z, int64_t ldz, bool z_f32, int act, void* dA, int64_t ldda,
                        void* dB, int64_t lddb, bool f32, float* db, const CallSpace& space,
                        hipStream_t s) {
  const int64_t rows = round_up(M, 64), cols = round_up(N, 64);
  return run_backward(
      "linear", ta, tb, M, N, K, A, lda, B, ldb, dA, ldda, dB, lddb, f32,
      {linear_grad_fits(rows, cols), db, ceil_div(rows, linear_grad_strip(rows, cols))},
      [&](uint16_t* G, int64_t ldg, int r, float* part) {
        return launch_linear_grad(static_cast<const uint16_t*>(dY), lddy, Z, ldz, z_f32, (int)M, N,
                                  act, G, ldg, r, ldg, part, s);
      },
      space, s);
}

// A mixture-of-experts layer, kMoeTokens rows of X at a time; p holds all but
// the rows' part and the workspace.
int run_moe(MoeParams p, int64_t M, const CallSpace& space, hipStream_t s) {
  p.ldh = round_up(p.F, 64);
  p.M = (int)(M < kMoeTokens ? M : kMoeTokens);
  MoeSpace need = moe_space(p);
  if (M > kMoeTokens && M % kMoeTokens != 0) {  // (the last rows, which may run otherwise)
    p.M = (int)(M % kMoeTokens);
    const MoeSpace last = moe_space(p);
    need = {need.logits > last.logits ? need.logits : last.logits, need.h > last.h ? need.h : last.h,
            need.part > last.part ? need.part : last.part};
  }
  const size_t bytesL = round256(need.logits), bytesH = round256(need.h);
  Workspace w;
  const int st = take_workspace(space, s, bytesL + bytesH + need.part, &w);
  if (st != TGEMM_OK) return st;
  if (verbose())
    fprintf(stderr, "tgemm: moe M=%lld K=%lld F=%d E=%d top=%d\n", (long long)M, (long long)p.K, p.F,
            p.E, p.top);
  char* const ws = static_cast<char*>(w.ptr);
  p.logits = reinterpret_cast<double*>(ws);
  p.h = reinterpret_cast<uint16_t*>(ws + bytesL);
  p.part = reinterpret_cast<float*>(ws + bytesL + bytesH);
  hipError_t e = hipSuccess;
  for (int64_t m = 0; m < M && e == hipSuccess; m += kMoeTokens) {
    p.M = (int)(M - m < kMoeTokens ? M - m : kMoeTokens);
    e = launch_moe(p, s);
    p.x += kMoeTokens * p.ldx;
    p.y += kMoeTokens * p.ldy;
    p.ids += kMoeTokens * p.top;
    p.weights += kMoeTokens * p.top;
  }
  release_workspace(w);
  return status_of(e);
}

// The workspace list allocates host memory; no exception leaves the library.
template <class Fn>
int no_throw(Fn&& fn) {
  try {
    return fn();
  } catch (...) {
    return TGEMM_ERR_NO_MEMORY;
  }
}

}  // namespace
}  // namespace tgemm

namespace {

// The operators' calls after validation, and their workspace queries.
int call_i8(char ta, char tb, int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda,
            const int8_t* B, int64_t ldb, const float* sa, const float* sb, void* C, int64_t ldc,
            int epi, int act, const CallSpace& space, void* stream) {
  const bool gate = epi == kRowsGated;
  RowsParams p = {};
  p.M = (int)M;
  p.N = (int)N;
  p.F = gate ? (int)(N / 2) : 0;
  p.K = (int)K;
  p.act = act;
  p.scale_a = sa;
  p.scale_b = sb;
  p.C = C;
  p.ldc = ldc;
  return no_throw([&] {
    return run_i8(ta, tb, A, lda, B, ldb, p, epi, gate, space,
                  reinterpret_cast<hipStream_t>(stream));
  });
}

// need, or the error that kept it from being found
int64_t queried(int st, int64_t need) { return st == kQueried ? need : st; }

// (a non-NULL address for the arguments a query does not take)
float g_any[1];

}  // namespace

extern "C" int tgemm_run_i8(char transA, char transB, int64_t M, int64_t N, int64_t K,
                            const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb,
                            const float* scale_a, const float* scale_b, void* C, int64_t ldc,
                            int epilogue, void* workspace, int64_t workspace_bytes, void* stream) {
  const int st = tgemm_validate_i8(transA, transB, M, N, K, A, lda, B, ldb, scale_a, scale_b, C,
                                   ldc, epilogue);
  if (st != TGEMM_OK) return st;
  return call_i8(transA, transB, M, N, K, A, lda, B, ldb, scale_a, scale_b, C, ldc,
                 epilogue == TGEMM_EPI_STORE_BF16 ? kRowsStoreBf16 : kRowsStoreF32, 0,
                 {workspace, workspace_bytes, nullptr}, stream);
}

extern "C" int64_t tgemm_i8_workspace_bytes(char transA, char transB, int64_t M, int64_t N,
                                            int64_t K, const int8_t* A, int64_t lda,
                                            const int8_t* B, int64_t ldb) {
  const int st = tgemm_validate_i8(transA, transB, M, N, K, A, lda, B, ldb, g_any, g_any, g_any, N,
                                   TGEMM_EPI_STORE_BF16);
  if (st != TGEMM_OK) return st;
  int64_t need = 0;
  return queried(call_i8(transA, transB, M, N, K, A, lda, B, ldb, nullptr, nullptr, nullptr, N,
                         kRowsStoreBf16, 0, {nullptr, 0, &need}, nullptr),
                 need);
}

extern "C" int tgemm_run_gated_i8(char transA, char transB, int64_t M, int64_t F, int64_t K,
                                  const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb,
                                  const float* scale_a, const float* scale_b, int activation,
                                  void* H, int64_t ldh, void* workspace, int64_t workspace_bytes,
                                  void* stream) {
  const int st = tgemm_validate_gated_i8(transA, transB, M, F, K, A, lda, B, ldb, scale_a, scale_b,
                                         activation, H, ldh);
  if (st != TGEMM_OK) return st;
  return call_i8(transA, transB, M, 2 * F, K, A, lda, B, ldb, scale_a, scale_b, H, ldh, kRowsGated,
                 activation, {workspace, workspace_bytes, nullptr}, stream);
}

extern "C" int64_t tgemm_gated_i8_workspace_bytes(char transA, char transB, int64_t M, int64_t F,
                                                  int64_t K, const int8_t* A, int64_t lda,
                                                  const int8_t* B, int64_t ldb) {
  const int st = tgemm_validate_gated_i8(transA, transB, M, F, K, A, lda, B, ldb, g_any, g_any,
                                         TGEMM_ACT_SILU, g_any, F);
  if (st != TGEMM_OK) return st;
  int64_t need = 0;
  return queried(call_i8(transA, transB, M, 2 * F, K, A, lda, B, ldb, nullptr, nullptr, nullptr, F,
                         kRowsGated, 0, {nullptr, 0, &need}, nullptr),
                 need);
}

extern "C" int tgemm_run_gated(char transA, char transB, int64_t M, int64_t F, int64_t K,
                               const void* A, int64_t lda, const void* B, int64_t ldb,
                               int activation, void* H, int64_t ldh, float* GU, int64_t ldgu,
                               void* workspace, int64_t workspace_bytes, void* stream) {
  const int st =
      tgemm_validate_gated(transA, transB, M, F, K, A, lda, B, ldb, activation, H, ldh, GU, ldgu);
  if (st != TGEMM_OK) return st;
  return no_throw([&] {
    return run_gated(transA, transB, M, F, K, A, lda, B, ldb, activation, H, ldh, GU, ldgu,
                     {workspace, workspace_bytes, nullptr}, reinterpret_cast<hipStream_t>(stream));
  });
}

extern "C" int64_t tgemm_gated_workspace_bytes(char transA, char transB, int64_t M, int64_t F,
                                               int64_t K, const void* A, int64_t lda,
                                               const void* B, int64_t ldb) {
  const int st = tgemm_validate_gated(transA, transB, M, F, K, A, lda, B, ldb, TGEMM_ACT_SILU,
                                      g_any, F, nullptr, 0);
  if (st != TGEMM_OK) return st;
  int64_t need = 0;
  return queried(no_throw([&] {
                   return run_gated(transA, transB, M, F, K, A, lda, B, ldb, 0, nullptr, F, nullptr,
                                    0, {nullptr, 0, &need}, nullptr);
                 }),
                 need);
}

extern "C" int tgemm_gated_grad(int64_t M, int64_t F, const void* dH, int64_t lddh, const void* GU,
                                int64_t ldgu, int gu_type, int activation, void* dGU,
                                int64_t lddgu, void* stream) {
  const int st =
      tgemm_validate_gated_grad(M, F, dH, lddh, GU, ldgu, gu_type, activation, dGU, lddgu);
  if (st != TGEMM_OK) return st;
  if (!gated_grad_fits(M, F)) return TGEMM_ERR_UNSUPPORTED;
  if (verbose())
    fprintf(stderr, "tgemm: gated grad M=%lld F=%lld\n", (long long)M, (long long)F);
  return status_of(launch_gated_grad(static_cast<const uint16_t*>(dH), lddh, GU, ldgu,
                                     gu_type == TGEMM_EPI_STORE_F32, (int)M, F, activation,
                                     static_cast<uint16_t*>(dGU), lddgu, (int)M, 2 * F,
                                     reinterpret_cast<hipStream_t>(stream)));
}

extern "C" int tgemm_run_gated_backward(char transA, char transB, int64_t M, int64_t F, int64_t K,
                                        const void* A, int64_t lda, const void* B, int64_t ldb,
                                        const void* dH, int64_t lddh, const void* GU, int64_t ldgu,
                                        int gu_type, int activation, void* dA, int64_t ldda, void* dB,
                                        int64_t lddb, int epilogue, void* workspace,
                                        int64_t workspace_bytes, void* stream) {
  const int st = tgemm_validate_gated_backward(transA, transB, M, F, K, A, lda, B, ldb, dH, lddh,
                                               GU, ldgu, gu_type, activation, dA, ldda, dB, lddb,
                                               epilogue);
  if (st != TGEMM_OK) return st;
  return no_throw([&] {
    return run_gated_backward(transA, transB, M, F, K, A, lda, B, ldb, dH, lddh, GU, ldgu,
                              gu_type == TGEMM_EPI_STORE_F32, activation, dA, ldda, dB, lddb,
                              epilogue == TGEMM_EPI_STORE_F32,
                              {workspace, workspace_bytes, nullptr},
                              reinterpret_cast<hipStream_t>(stream));
  });
}

extern "C" int64_t tgemm_gated_backward_workspace_bytes(char transA, char transB, int64_t M,
                                                        int64_t F, int64_t K, const void* A,
                                                        int64_t lda, const void* B, int64_t ldb) {
  const int64_t ldd = transB == 'N' || transB == 'n' ? 2 * F : K;
  const int st =
      tgemm_validate_gated_backward(transA, transB, M, F, K, A, lda, B, ldb, g_any, F, g_any, 2 * F,
                                    TGEMM_EPI_STORE_BF16, TGEMM_ACT_SILU, g_any, K, g_any, ldd,
                                    TGEMM_EPI_STORE_BF16);
  if (st != TGEMM_OK) return st;
  int64_t need = 0;
  return queried(no_throw([&] {
                   return run_gated_backward(transA, transB, M, F, K, A, lda, B, ldb, nullptr, F,
                                             nullptr, 2 * F, false, 0, nullptr, K, nullptr, ldd,
                                             false,
                                             {nullptr, 0, &need}, nullptr);
                 }),
                 need);
}

extern "C" int tgemm_run_linear(char transA, char transB, int64_t M, int64_t N, int64_t K,
                                const void* A, int64_t lda, const void* B, int64_t ldb,
                                const void* bias, int activation, const void* residual, int64_t ldr,
                                void* Y, int64_t ldy, int epilogue, void* Z, int64_t ldz,
                                int z_type, void* workspace, int64_t workspace_bytes,
                                void* stream) {
  const int st = tgemm_validate_linear(transA, transB, M, N, K, A, lda, B, ldb, bias, activation,
                                       residual, ldr, Y, ldy, epilogue, Z, ldz, z_type);
  if (st != TGEMM_OK) return st;
  RowsParams p = {};
  p.M = (int)M;
  p.N = (int)N;
  p.act = activation;
  p.C = Y;
  p.ldc = ldy;
  p.c_f32 = epilogue == TGEMM_EPI_STORE_F32;
  p.bias = static_cast<const uint16_t*>(bias);
  p.res = residual;
  p.ldr = ldr;
  p.z = Z;
  p.ldz = ldz;
  p.z_f32 = z_type == TGEMM_EPI_STORE_F32;
  return no_throw([&] {
    return run_bf16(transA, transB, K, A, lda, B, ldb, p, kRowsLinear, false,
                    {workspace, workspace_bytes, nullptr}, reinterpret_cast<hipStream_t>(stream));
  });
}

extern "C" int64_t tgemm_linear_workspace_bytes(char transA, char transB, int64_t M, int64_t N,
                                                int64_t K, const void* A, int64_t lda,
                                                const void* B, int64_t ldb) {
  const int st =
      tgemm_validate_linear(transA, transB, M, N, K, A, lda, B, ldb, nullptr, TGEMM_ACT_NONE,
                            nullptr, 0, g_any, N, TGEMM_EPI_STORE_BF16, nullptr, 0,
                            TGEMM_EPI_STORE_BF16);
  if (st != TGEMM_OK) return st;
  RowsParams p = {};
  p.M = (int)M;
  p.N = (int)N;
  int64_t need = 0;
  return queried(no_throw([&] {
                   return run_bf16(transA, transB, K, A, lda, B, ldb, p, kRowsLinear, false,
                                   {nullptr, 0, &need}, nullptr);
                 }),
                 need);
}

extern "C" int tgemm_run_linear_backward(char transA, char transB, int64_t M, int64_t N, int64_t K,
                                         const void* A, int64_t lda, const void* B, int64_t ldb,
                                         const void* dY, int64_t lddy, const void* Z, int64_t ldz,
                                         int z_type, int activation, void* dA, int64_t ldda,
                                         void* dB, int64_t lddb, int epilogue, float* dbias,
                                         void* workspace, int64_t workspace_bytes, void* stream) {
  const int st = tgemm_validate_linear_backward(transA, transB, M, N, K, A, lda, B, ldb, dY, lddy,
                                                Z, ldz, z_type, activation, dA, ldda, dB, lddb,
                                                epilogue, dbias);
  if (st != TGEMM_OK) return st;
  return no_throw([&] {
    return run_linear_backward(transA, transB, M, N, K, A, lda, B, ldb, dY, lddy, Z, ldz,
                               z_type == TGEMM_EPI_STORE_F32, activation, dA, ldda, dB, lddb,
                               epilogue == TGEMM_EPI_STORE_F32, dbias,
                               {workspace, workspace_bytes, nullptr},
                               reinterpret_cast<hipStream_t>(stream));
  });
}

extern "C" int64_t tgemm_linear_backward_workspace_bytes(char transA, char transB, int64_t M,
                                                         int64_t N, int64_t K, const void* A,
                                                         int64_t lda, const void* B, int64_t ldb) {
  const int64_t ldd = transB == 'N' || transB == 'n' ? N : K;
  const int st = tgemm_validate_linear_backward(
      transA, transB, M, N, K, A, lda, B, ldb, g_any, N, nullptr, 0, TGEMM_EPI_STORE_BF16,
      TGEMM_ACT_NONE, g_any, K, g_any, ldd, TGEMM_EPI_STORE_BF16, nullptr);
  if (st != TGEMM_OK) return st;
  int64_t need = 0;
  return queried(no_throw([&] {
                   return run_linear_backward(transA, transB, M, N, K, A, lda, B, ldb, nullptr, N,
                                              nullptr, 0, false, kActNone, nullptr, K, nullptr, ldd,
                                              false, g_any, {nullptr, 0, &need}, nullptr);
                 }),
                 need);
}

extern "C" int tgemm_rms_norm_i8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                 const void* weight, float eps, int64_t M, int64_t K, void* sum,
                                 int64_t lds, int8_t* q, int64_t ldq, float* scale, void* stream) {
  const int st = tgemm_validate_rms_norm_i8(x, ldx, residual, ldr, weight, eps, M, K, sum, lds, q,
                                            ldq, scale);
  if (st != TGEMM_OK) return st;
  const RowQuantParams p = {static_cast<const uint16_t*>(x), ldx,
                            static_cast<const uint16_t*>(residual), ldr,
                            static_cast<const uint16_t*>(weight), eps,
                            static_cast<uint16_t*>(sum), lds, q, ldq, scale, (int)M, K};
  if (!row_quant_fits(p)) return TGEMM_ERR_UNSUPPORTED;
  if (verbose())
    fprintf(stderr, "tgemm: rms norm i8 M=%lld K=%lld residual=%d\n", (long long)M, (long long)K,
            residual != nullptr);
  return status_of(launch_row_quant(p, reinterpret_cast<hipStream_t>(stream)));
}

extern "C" int tgemm_quantize_i8(const void* x, int64_t ldx, int64_t M, int64_t K, int8_t* q,
                                 int64_t ldq, float* scale, void* stream) {
  const int st = tgemm_validate_quantize_i8(x, ldx, M, K, q, ldq, scale);
  if (st != TGEMM_OK) return st;
  const RowQuantParams p = {static_cast<const uint16_t*>(x), ldx, nullptr, 0, nullptr, 0.f,
                            nullptr, 0, q, ldq, scale, (int)M, K};
  if (!row_quant_fits(p)) return TGEMM_ERR_UNSUPPORTED;
  if (verbose())
    fprintf(stderr, "tgemm: quantize i8 M=%lld K=%lld\n", (long long)M, (long long)K);
  return status_of(launch_row_quant(p, reinterpret_cast<hipStream_t>(stream)));
}

extern "C" int tgemm_block_norm(const void* y, int64_t ldy, const void* residual, int64_t ldr,
                                int stream_type, const void* post_weight, const void* gate,
                                int64_t ldgate, int64_t gates, float scale, const void* weight,
                                float eps, int64_t M, int64_t K, void* sum, int64_t lds, void* n,
                                int64_t ldn, float* rstd, void* stream) {
  const int st = tgemm_validate_block_norm(y, ldy, residual, ldr, stream_type, post_weight, gate,
                                           ldgate, gates, scale, weight, eps, M, K, sum, lds, n, ldn,
                                           rstd);
  if (st != TGEMM_OK) return st;
  if (!block_norm_fits(M, K)) return TGEMM_ERR_UNSUPPORTED;
  if (verbose())
    fprintf(stderr, "tgemm: block norm M=%lld K=%lld post=%d gates=%lld\n", (long long)M,
            (long long)K, post_weight != nullptr, (long long)(gate != nullptr ? gates : 0));
  const BlockNormParams p = {static_cast<const uint16_t*>(y), ldy, residual, ldr,
                             static_cast<const uint16_t*>(post_weight),
                             static_cast<const uint16_t*>(gate), ldgate,
                             gate != nullptr ? (int)(M / gates) : 1, scale,
                             static_cast<const uint16_t*>(weight), eps, sum, lds,
                             static_cast<uint16_t*>(n), ldn, rstd, (int)M, K};
  return status_of(launch_block_norm(p, stream_type == TGEMM_EPI_STORE_F32,
                                     reinterpret_cast<hipStream_t>(stream)));
}

extern "C" int64_t tgemm_block_norm_backward_workspace_bytes(int64_t M, int64_t K, int post,
                                                             int64_t gates) {
  if (M < 1 || K < 1 || gates < 0 || (gates > 0 && M % gates != 0)) return TGEMM_ERR_INVALID_ARG;
  if (M >= int64_t(1) << 31 || !block_norm_bwd_fits(K)) return TGEMM_ERR_UNSUPPORTED;
  return (int64_t)block_norm_bwd_bytes(M, K, post != 0, gates > 0);
}

extern "C" int tgemm_block_norm_backward(const void* dn, int64_t lddn, const void* ds, int64_t ldds,
                                         const void* y, int64_t ldy, const void* residual,
                                         int64_t ldr, int stream_type, const void* post_weight,
                                         const void* gate, int64_t ldgate, int64_t gates,
                                         float scale, const void* weight, const float* rstd,
                                         int64_t M, int64_t K, void* dresidual, int64_t lddr,
                                         void* dy, int64_t lddy, float* dweight, float* dpost,
                                         float* dgate, void* workspace, int64_t workspace_bytes,
                                         void* stream) {
  const int st = tgemm_validate_block_norm_backward(
      dn, lddn, ds, ldds, y, ldy, residual, ldr, stream_type, post_weight, gate, ldgate, gates,
      scale, weight, rstd, M, K, dresidual, lddr, dy, lddy, dweight, dpost, dgate);
  if (st != TGEMM_OK) return st;
  if (!block_norm_bwd_fits(K)) return TGEMM_ERR_UNSUPPORTED;
  return no_throw([&] {
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    Workspace w;
    const int sw = take_workspace({workspace, workspace_bytes, nullptr}, s,
                                  block_norm_bwd_bytes(M, K, post_weight != nullptr, gate != nullptr),
                                  &w);
    if (sw != TGEMM_OK) return sw;
    if (verbose())
      fprintf(stderr, "tgemm: block norm backward M=%lld K=%lld post=%d gates=%lld\n", (long long)M,
              (long long)K, post_weight != nullptr, (long long)(gate != nullptr ? gates : 0));
    const BlockNormGradParams p = {static_cast<const uint16_t*>(dn), lddn, ds, ldds,
                                   static_cast<const uint16_t*>(y), ldy, residual, ldr,
                                   static_cast<const uint16_t*>(post_weight),
                                   static_cast<const uint16_t*>(gate), ldgate,
                                   gate != nullptr ? (int)(M / gates) : 1, scale,
                                   static_cast<const uint16_t*>(weight), rstd, dresidual, lddr,
                                   static_cast<uint16_t*>(dy), lddy, dweight, dpost, dgate, (int)M,
                                   K, static_cast<float*>(w.ptr), 0};
    const hipError_t e = launch_block_norm_bwd(p, stream_type == TGEMM_EPI_STORE_F32, s);
    release_workspace(w);
    return status_of(e);
  });
}

extern "C" int tgemm_run_moe(int64_t M, int64_t K, int64_t F, int64_t E, int64_t top, const void* X,
                             int64_t ldx, const void* router, int64_t ldr, int router_type,
                             int renormalize, float scale, int32_t* ids, float* weights,
                             const void* W1, int64_t ldw1, int64_t sw1, const void* W2,
                             int64_t ldw2, int64_t sw2, int activation, void* Y, int64_t ldy,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  const int st = tgemm_validate_moe(M, K, F, E, top, X, ldx, router, ldr, router_type, renormalize,
                                    scale, ids, weights, W1, ldw1, sw1, W2, ldw2, sw2, activation, Y,
                                    ldy);
  if (st != TGEMM_OK) return st;
  MoeParams p = {};
  p.K = K;
  p.F = (int)F;
  p.E = (int)E;
  p.top = (int)top;
  p.x = static_cast<const uint16_t*>(X);
  p.ldx = M == 1 ? K : ldx;  // (the stride of a single row is never used)
  p.router = router;
  p.ldr = ldr;
  p.router_f32 = router_type == TGEMM_EPI_STORE_F32;
  p.renormalize = renormalize != 0;
  p.scale = scale;
  p.ids = ids;
  p.weights = weights;
  p.w1 = static_cast<const uint16_t*>(W1);
  p.ldw1 = ldw1;
  p.sw1 = E == 1 ? 0 : sw1;
  p.w2 = static_cast<const uint16_t*>(W2);
  p.ldw2 = K == 1 ? F : ldw2;
  p.sw2 = E == 1 ? 0 : sw2;
  p.act = activation;
  p.y = static_cast<uint16_t*>(Y);
  p.ldy = ldy;
  return no_throw([&] {
    return run_moe(p, M, {workspace, workspace_bytes, nullptr},
                   reinterpret_cast<hipStream_t>(stream));
  });
}

extern "C" int64_t tgemm_moe_workspace_bytes(int64_t M, int64_t K, int64_t F, int64_t E,
                                             int64_t top, int routed) {
  const int st = tgemm_validate_moe(M, K, F, E, top, g_any, K, routed ? g_any : nullptr, K,
                                    TGEMM_EPI_STORE_BF16, 1, 1.f, reinterpret_cast<int32_t*>(g_any),
                                    g_any, g_any, K, 2 * F * K, g_any, F, K * F, TGEMM_ACT_SILU,
                                    g_any, K);
  if (st != TGEMM_OK) return st;
  MoeParams p = {};
  p.K = K;
  p.F = (int)F;
  p.E = (int)E;
  p.top = (int)top;
  p.router = routed ? g_any : nullptr;
  int64_t need = 0;
  return queried(no_throw([&] { return run_moe(p, M, {nullptr, 0, &need}, nullptr); }), need);
}
