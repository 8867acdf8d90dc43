// zr_attn_tc.cuh — what the tensor-core attention kernels share (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "zr_attn.h"
#include "zr_kernels.cuh"
#include "zr_tc.cuh"

namespace zr {

constexpr uint32_t kAtRows = 128;             // rows of a tile, queries or keys
constexpr uint32_t kAtBlock = kAtRows * 128;  // bytes of 64 elements of its rows

// Registers per thread from here on, by a whole warpgroup.  384 threads are
// launched with 168 each: 216 for two warpgroups and 72 for the third are as
// many (or 200 and 104), so the wait for them ends.
template <int N>
__device__ __forceinline__ void regs_give() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
static_assert(2 * 216 + 72 == 3 * 168 && 2 * 200 + 104 == 3 * 168, "registers");

// 64 elements (block * 64 on) of 128 tokens of a head, 128-byte swizzle; tokens
// and elements out of range read as zero.
__device__ __forceinline__ void at_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, uint32_t block,
                                        uint32_t head, uint32_t token, uint32_t batch) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(block * 64), "r"(head), "r"(token), "r"(batch)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// D += A B with A in tensor memory: 128 lanes, two bfloat16 k per column.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 columns of this warp's 32 TMEM lanes; tc_wait_store() before others read.
__device__ __forceinline__ void tc_store32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tc_wait_store() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// An operand tile [128 rows][DP] as blocks of 64 elements: K-major (k along the
// elements) block by block, MN-major (k along the rows) with the blocks as the
// leading offset.
__device__ __forceinline__ uint64_t at_desc(uint32_t addr, bool rows_are_k) {
  uint64_t d = uint64_t((addr & 0x3FFFFu) >> 4);
  d |= uint64_t(rows_are_k ? kAtBlock >> 4 : 1) << 16;
  d |= uint64_t(1024 >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}
// D binary32, A and B bfloat16; b_rows_k: B's k runs along its rows.
__device__ __forceinline__ constexpr uint32_t at_idesc(uint32_t n, bool b_rows_k) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(b_rows_k) << 16) | ((n >> 3) << 17) | ((kAtRows / 16) << 24);
}
// D[128, 128] = A B^T of two K-major tiles of DP elements.
template <int DP>
__device__ __forceinline__ void at_scores(uint32_t d, uint32_t a, uint32_t b) {
  const uint64_t da = at_desc(a, false), db = at_desc(b, false);
#pragma unroll
  for (uint32_t j = 0; j < DP / 16; ++j) {
    const uint64_t at = (j / 4) * (kAtBlock >> 4) + (j % 4) * 2;
    tc_mma<1>(d, da + at, db + at, at_idesc(128, false), j != 0);
  }
}
// D[128, DP] (+)= W B, W [128, 128] bfloat16 in tensor memory, B's k its rows.
template <int DP>
__device__ __forceinline__ void at_sum(uint32_t d, uint32_t w, uint32_t b, bool accumulate) {
  const uint64_t db = at_desc(b, true);
#pragma unroll
  for (uint32_t j = 0; j < kAtRows / 16; ++j)
    tc_mma_ts(d, w + j * 8, db + j * (2048 >> 4), at_idesc(DP, true), accumulate || j != 0);
}

// Zeroes the rows [from, 128) of a tile in shared memory by one warp: rows
// behind a packed sequence belong to others or to nobody, and what they hold
// must not meet a zero weight in a product (0 times NaN).
__device__ __forceinline__ void at_clear(uint32_t tile, uint32_t blocks, uint32_t from) {
  for (uint32_t b = 0; b < blocks; ++b)
    for (uint32_t i = from * 8 + (threadIdx.x & 31); i < kAtRows * 8; i += 32)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + b * kAtBlock + i * 16), "r"(0) : "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// Item `round` of this CTA: there and back over the list.
__device__ __forceinline__ uint32_t at_item(uint32_t round) {
  return round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// Stores a row's 32 results as bfloat16 at elements d0 on (of dim; wide: 8 at a
// time).
__device__ __forceinline__ void at_store_row(__nv_bfloat16* row, int64_t elem, bool wide, const float* v, uint32_t d0,
                                             uint32_t dim) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
      if (d0 + i < dim)
        *reinterpret_cast<uint4*>(row + d0 + i) = make_uint4(pack_bf16(v[i], v[i + 1]), pack_bf16(v[i + 2], v[i + 3]),
                                                             pack_bf16(v[i + 4], v[i + 5]), pack_bf16(v[i + 6], v[i + 7]));
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (d0 + i < dim) row[int64_t(d0 + i) * elem] = __float2bfloat16_rn(v[i]);
  }
}

}  // namespace zr
