// zr_attn.h — plan of the causal attention and its launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "zr_internal.h"

namespace zr {

// A tensor [batch, token, head, element] (packed sequences: one batch).
struct AttnView {
  const void* p;
  int64_t batch, token, head, elem;  // strides in elements
};

struct AttnPlan {
  AttnView q, k, v, o, go;   // o: the output (forward: written)
  AttnView gq, gk, gv;       // gradients, written
  void* low;                 // dense over o's shape: o's rounding error, or null
  float* lse;                // dense over (batch, token, head), or null
  float* lse2;               // backward, workspace: lse * log2(e), [batch][head][row_pitch]
  float* delta;              // backward, workspace: sum of grad_out * out, likewise
  const int32_t* offsets;    // packed sequences: their `sequences` + 1 borders, or null
  uint32_t sequences;
  uint32_t batch, tokens, heads, kv_heads, group, dim;
  uint32_t row_pitch;        // tokens rounded up to 128
  uint32_t slots;            // tiles of one head, all sequences (packed: at most)
  uint32_t tile_rows;        // rows of a tile
  uint32_t splits;           // tensor cores, bfloat16: shares of a pair of query tiles' keys (forward),
                             // of a key tile's steps (backward), 1 to 8
  float* part;               // with splits > 1, workspace: [split][batch][token][head] of results, then of
                             // lse; backward [split][batch][token][kv head][grad_v, grad_k]
  uint32_t want;             // bit 0: grad_q, bits 1 and 2: grad_k, grad_v
  uint32_t vec;              // 16-byte reads of every operand
  uint32_t o_wide, low_wide; // tensor-core forward: 16-byte stores of o and low;
                             // backward, o_wide: 16-byte reads of o, low and go
  uint32_t g_wide;           // tensor-core backward: bits as `want`, of the gradients
  float scale, scale_log2;   // scale, scale * log2(e)
};

// Tensor maps of the tensor-core kernels: boxes of 64 elements x 128 tokens.
struct AttnMaps {
  CUtensorMap q, k, v, go;
};

// One tile of one sequence.
struct AttnTile {
  uint32_t batch, start, len, tile;  // rows [start, start + len) of `batch`; which tile of them
  bool live;
};

#if defined(__CUDACC__)
// The tile behind `slot`, by a whole warp.  Sequences of one length: the tiles
// with the most to see come first.  Packed ones are found by their borders,
// which are kept inside the tokens whatever they hold.
__device__ __forceinline__ AttnTile attn_tile(const AttnPlan& p, uint32_t slot, bool ascending) {
  AttnTile t;
  if (!p.offsets) {
    const uint32_t per = (p.tokens + p.tile_rows - 1) / p.tile_rows;
    const uint32_t rank = slot / p.batch;
    t.batch = slot - rank * p.batch;
    t.tile = ascending ? rank : per - 1 - rank;
    t.start = 0;
    t.len = p.tokens;
    t.live = rank < per;
    return t;
  }
  const uint32_t lane = threadIdx.x & 31;
  t.batch = 0;
  t.live = false;
  t.start = t.len = t.tile = 0;
  uint32_t before = 0;
  for (uint32_t base = 0; base < p.sequences; base += 32) {
    const uint32_t i = base + lane;
    int64_t lo = 0, hi = 0;
    if (i < p.sequences) {
      lo = p.offsets[i];
      hi = p.offsets[i + 1];
    }
    lo = lo < 0 ? 0 : lo > int64_t(p.tokens) ? int64_t(p.tokens) : lo;
    hi = hi < lo ? lo : hi > int64_t(p.tokens) ? int64_t(p.tokens) : hi;
    const uint32_t n = (uint32_t(hi - lo) + p.tile_rows - 1) / p.tile_rows;
    uint32_t sum = n;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= uint32_t(d)) sum += x;
    }
    const uint32_t end = before + sum;  // tiles up to and with sequence i
    const uint32_t mine = __ballot_sync(0xFFFFFFFFu, slot < end);
    if (mine) {
      const int src = __ffs(int(mine)) - 1;
      const uint32_t first = __shfl_sync(0xFFFFFFFFu, end - n, src), count = __shfl_sync(0xFFFFFFFFu, n, src);
      t.start = __shfl_sync(0xFFFFFFFFu, uint32_t(lo), src);
      t.len = __shfl_sync(0xFFFFFFFFu, uint32_t(hi - lo), src);
      t.tile = ascending ? slot - first : count - 1 - (slot - first);
      t.live = true;
      return t;
    }
    before = __shfl_sync(0xFFFFFFFFu, end, 31);
  }
  return t;
}
#endif

// es: bytes per element.
cudaError_t launch_attn_any_fwd(int es, const AttnPlan& p, cudaStream_t s);
// On the tensor cores, bfloat16, dim <= 128; p.tile_rows and p.slots for tiles of
// 256 queries.
cudaError_t launch_attn_fwd(const AttnPlan& p, const AttnMaps& maps, cudaStream_t s);
// The same of tiles of 128; after launch_attn_rows.
cudaError_t launch_attn_bwd(const AttnPlan& p, const AttnMaps& maps, cudaStream_t s);
cudaError_t launch_attn_any_bwd(int es, const AttnPlan& p, cudaStream_t s);
// launch_attn_split copies q, k, v (and go; count = 3 or 4) to rows that the maps
// are over: binary32 with dim <= 64 into parts, [part][batch][token][head][64]; bfloat16
// as they are, in rows of 64 or 128.  wide: bit i, 16-byte reads (binary32).
cudaError_t launch_attn_split(int es, const AttnPlan& p, uint16_t* const* out, uint32_t count, uint32_t wide,
                              cudaStream_t s);
// binary32, dim <= 64, in parts.  Tiles of 256 queries forward, of 128 backward.
cudaError_t launch_attn_f32_fwd(const AttnPlan& p, const AttnMaps& maps, cudaStream_t s);
cudaError_t launch_attn_f32_bwd(const AttnPlan& p, const AttnMaps& maps, cudaStream_t s);
// lse2 and delta of every row that a sequence holds.
cudaError_t launch_attn_rows(int es, const AttnPlan& p, cudaStream_t s);

}  // namespace zr
