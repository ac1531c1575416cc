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

// Bounded wait of a whole warp. False: the wait expired here or somewhere else in the block.
RSM_DEV bool wait_ok(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (!tc::mbar_wait(bar, parity)) {
    *abort_flag = 1;
    raise_status(RSM_ERR_TIMEOUT);
  }
  return !__any_sync(kFull, *abort_flag != 0);
}

RSM_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

RSM_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}

}  // namespace attn
}  // namespace rsm
