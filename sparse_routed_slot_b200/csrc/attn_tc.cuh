// attn_tc.cuh -- what the tensor-core attention kernels share.
#pragma once

#include <cuda.h>

#include "attention.cuh"
#include "tc.cuh"
#include "tma_map.h"

namespace rsm {
namespace attn {

constexpr float kNegInf = -__builtin_inff();

RSM_DEV void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}

// Bounded waits. An expired wait is reported, and its warp stops; every other role of the block depends on
// some wait that then expires as well. (A shared flag read beside each wait would cost a third of it.)
RSM_DEV bool wait_one(uint64_t* bar, uint32_t parity) {
  if (tc::mbar_wait(bar, parity)) return true;
  raise_status(RSM_ERR_TIMEOUT);
  return false;
}
// The same decision in every lane of a warp.
RSM_DEV bool wait_warp(uint64_t* bar, uint32_t parity) { return __all_sync(kFull, wait_one(bar, parity)); }

// The lowest n bits of a word (n below 0: none, above 32: all).
RSM_DEV uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

RSM_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The largest of three.
RSM_DEV float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

RSM_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}

// NC fp32 columns of a thread's row in TMEM, times `scale`, as bf16 into row r of a tile that a tensor store
// takes (64-column blocks of 128 swizzled rows), from column `c0` of the tile on.
template <int NC> RSM_DEV void stage_row(unsigned char* tile, int r, int c0, uint32_t tmem, float scale) {
#pragma unroll 1
  for (int c = 0; c < NC; c += 32) {
    float x[32];
    tc::tmem_ld32(tmem + c, x);
    tc::tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
      const int k = (c0 + c + e) >> 3;
      *reinterpret_cast<uint4*>(tile + (k >> 3) * (128 * 128) + r * 128 + (((k & 7) ^ (r & 7)) << 4)) =
          make_uint4(pack_bf16(x[e] * scale, x[e + 1] * scale), pack_bf16(x[e + 2] * scale, x[e + 3] * scale),
                     pack_bf16(x[e + 4] * scale, x[e + 5] * scale), pack_bf16(x[e + 6] * scale, x[e + 7] * scale));
    }
  }
}
// What that rounding left, as bf16, into such a tile.
template <int NC> RSM_DEV void stage_row_low(unsigned char* tile, int r, uint32_t tmem, float scale) {
#pragma unroll 1
  for (int c = 0; c < NC; c += 32) {
    float x[32];
    tc::tmem_ld32(tmem + c, x);
    tc::tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      x[e] *= scale;
      x[e] -= __bfloat162float(__float2bfloat16_rn(x[e]));
    }
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
      const int k = (c + e) >> 3;
      *reinterpret_cast<uint4*>(tile + (k >> 3) * (128 * 128) + r * 128 + (((k & 7) ^ (r & 7)) << 4)) =
          make_uint4(pack_bf16(x[e], x[e + 1]), pack_bf16(x[e + 2], x[e + 3]), pack_bf16(x[e + 4], x[e + 5]),
                     pack_bf16(x[e + 6], x[e + 7]));
    }
  }
}
// The same columns straight to memory, 16 bytes at a time.
template <int NC> RSM_DEV void store_row(__nv_bfloat16* to, uint32_t tmem, float scale, int cols, bool live) {
#pragma unroll 1
  for (int c = 0; c < NC; c += 32) {
    float x[32];
    tc::tmem_ld32(tmem + c, x);
    tc::tmem_wait_ld();
    if (!live) continue;
#pragma unroll
    for (int e = 0; e < 32; e += 8)
      if (c + e < cols)
        *reinterpret_cast<uint4*>(to + c + e) =
            make_uint4(pack_bf16(x[e] * scale, x[e + 1] * scale), pack_bf16(x[e + 2] * scale, x[e + 3] * scale),
                       pack_bf16(x[e + 4] * scale, x[e + 5] * scale), pack_bf16(x[e + 6] * scale, x[e + 7] * scale));
  }
}
RSM_DEV void group_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

}  // namespace attn
}  // namespace rsm
