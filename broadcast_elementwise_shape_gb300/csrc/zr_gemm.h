// zr_gemm.h — plan of the tensor-core products behind the cross entropy of a
// linear head, and its launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "zr_internal.h"

namespace zr {

// The labels of the rows, int32 or int64: a row's index is split over the
// labels' dims (merged where they allow it, innermost first; mostly one).
struct RowLabels {
  const void* p;
  uint32_t i64, n;
  FastDiv div[kMaxDims];
  int64_t stride[kMaxDims];
};
#if defined(__CUDACC__)
__device__ __forceinline__ int64_t row_label(const RowLabels& l, uint32_t row) {
  int64_t off = 0;
  uint32_t i = 0;
#pragma unroll 1
  for (; i + 1 < l.n; ++i) {
    const uint32_t q = fd_div(l.div[i], row);
    off += int64_t(row - q * l.div[i].d) * l.stride[i];
    row = q;
  }
  off += int64_t(row) * l.stride[i];
  return l.i64 ? static_cast<const int64_t*>(l.p)[off]
               : int64_t(static_cast<const int32_t*>(l.p)[off]);
}
#endif

// One product out[m, n] = sum_k A[m, k] B[n, k] of bfloat16 operands, binary32
// accumulation.  K-major operands have k as their contiguous dim, MN-major ones
// m or n.  Each is a 4-d tensor map over (64 columns, rows, blocks of 64
// columns, parts), whose box is one stage's share, all parts of it: 64 columns
// of 128 or 256 rows (K-major), or 64 rows of two or four column blocks
// (MN-major).  One box per
// operand and stage: two of 8 KB instead of one of 16 KB cost MN-major products
// 12 % ([4096, 32000] x [32000, 1024]: 193 against 172 us).
// Parts: one, or the three that a binary32 operand is split into (zr_xent.cu),
// whose product is the sum of six; G of bfloat16 tensors may have two, whose
// product with one is the sum of both.
struct GemmProblem {
  CUtensorMap a, b;
  uint32_t m, n, k;
  uint32_t a_mn, b_mn;       // 1: MN-major
  uint32_t tn;               // tile width; the last tile of an MN-major B is
                             // as narrow as its boxes allow
  uint32_t m_tiles, n_tiles, n_kb;  // n_kb: 64-wide k blocks
  // Epilogue kEpiOut: k in `slices` parts of kb_slice blocks (the last one
  // shorter), each with tiles of its own whose results go to plane `slice` of
  // acc, `plane` elements apart; elsewhere one of all blocks.
  uint32_t slices, kb_slice;
  int64_t plane;
  uint32_t chunk;            // k blocks per accumulation in TMEM
  // Epilogues kEpiGrad and kEpiOut with tma_out: results leave through this map,
  // in boxes of 128 bytes by 32 rows.
  CUtensorMap c;
  uint32_t tma_out;
  // Epilogue kEpiOut: out = [acc_in +] product, in the operands' type with row
  // stride ldo; or to the binary32 array acc when acc_out.
  void* out;
  float* acc;
  int64_t ldo, lda;
  uint32_t acc_in, acc_out;
  // Epilogue kEpiOut: rows are those of the labels; left-out ones become 0
  // whatever the product and the factor are.
  uint32_t by_row;
};

enum GemmEpilogue : int {
  kEpiLse = 0,   // per row and half tile: maximum and sum of exponentials
  kEpiGrad = 1,  // scale * (exp(product - lse) - [column == label]) as bfloat16 parts,
                 // and the sums that the label's element is worked out from
  kEpiOut = 2    // the product itself
};

struct GemmPlan {
  GemmProblem pr[2];
  uint32_t n_prob, parts;    // parts: of both operands; 2: of G alone
  uint32_t tiles0, tiles;    // tiles of problem 0, of both
  uint32_t m_fast;           // consecutive tiles walk m first
  // Two problems' tiles over `workers` clusters (GemmWalk).
  uint32_t workers, head, extra, late_first;
  const float* out_scale;    // kEpiOut: multiplies the finished product, or null (1)
  // kEpiLse, kEpiGrad; kEpiOut by_row
  RowLabels labels;
  // kEpiLse
  uint32_t* ticket;          // set to 0
  float2* partial;           // [m][2 * n_tiles] (maximum, sum)
  float* at;                 // [m] product at the label; kEpiGrad: exp(product - lse) there
  // kEpiGrad
  const float* lse;          // [m]
  const float* row_scale;    // [m], or null (1)
  float* sums;               // [m][2 * n_tiles] sum of exp(product - lse) but for the label,
                             // whose element is stored as 0; or null
  int64_t ignore_index, vocab;
  int64_t label_base;        // column 0 of this product is this label
};

// The tiles of worker w, in order: its share of problem 0 round-robin, then of
// problem 1.  Problem 0's tiles may not divide evenly: the first `head`
// workers then have one more than the rest, which take `extra` tiles of
// problem 1 meanwhile (about as long as one of problem 0), before all walk the
// remaining ones round-robin, those that are ahead first.  Tiles that run at
// the same time are neighbours throughout, so they share operands in L2.
struct GemmWalk {
  uint32_t w, n0, j;
};
#if defined(__CUDACC__)
#define ZR_GEMM_HD __host__ __device__ __forceinline__
#else
#define ZR_GEMM_HD inline
#endif
ZR_GEMM_HD GemmWalk gemm_walk(const GemmPlan& p, uint32_t w) {
  GemmWalk g;
  g.w = w;
  g.n0 = w < p.tiles0 ? (p.tiles0 - w - 1) / p.workers + 1 : 0;
  g.j = 0;
  return g;
}
// The next tile, or p.tiles when there is none.
ZR_GEMM_HD uint32_t gemm_next(const GemmPlan& p, GemmWalk* g) {
  const uint32_t j = g->j++;
  if (j < g->n0) return g->w + j * p.workers;
  uint32_t k = j - g->n0;                     // k-th tile of problem 1
  const uint32_t rest = p.workers - p.head;   // workers with one tile fewer
  uint32_t l;
  if (g->w >= p.head && k < p.extra) {
    l = k * rest + (g->w - p.head);
  } else {
    if (g->w >= p.head) k -= p.extra;
    uint32_t at = g->w;
    if (p.late_first) at = at >= p.head ? at - p.head : at + rest;
    l = p.extra * rest + k * p.workers + at;
  }
  const uint32_t t = p.tiles0 + l;
  return t < p.tiles ? t : p.tiles;
}

// grid: CTAs (a multiple of cg); cg: CTAs per cluster, 1 or 2.  sum: chunks of
// k are added in registers (else every problem's chunk is its whole k); always
// with three parts.
cudaError_t launch_gemm(int epi, int cg, bool sum, const GemmPlan& p, unsigned grid, cudaStream_t s);

}  // namespace zr
