// block_norm.cu -- the norms around a block, fused with its output gate and residual scale, and
// their gradients (rsm_block_norm_forward, rsm_block_norm_backward).
//
//   r1 = rsqrt(mean(y^2) + eps),  n = y r1 w_post,  h = res + scale n act(g)
//   r2 = rsqrt(mean(h^2) + eps),  x = h r2 w_pre
// and, with e = dx w_pre,
//   dH = dh + r2 e - h r2^3 mean(e h),  dres = dH,  du = scale dH
//   dg = du n act'(g),  f = du act(g) w_post,  dy = r1 f - y r1^3 mean(f y)
//   dw_post = sum_rows du act(g) y r1,  dw_pre = sum_rows dx h r2
// The cubes are never formed: h r2 and mean(e h) r2 are of the order of 1 and of e, where r2^3 is infinite for a
// row of zeros from eps = 1e-26 down.
// Everything is fp32, two values per instruction, between the loads and the stores; h is normalised before it
// is rounded, and the backward forms it again from its inputs, so no rounded value enters a sum.
//
// A row stays on the SM: TPR threads hold VEC * ITER values each, and the row crosses memory once (bound: HBM
// bandwidth). The row sums go over shuffles and, past one warp, one exchange in shared memory. In the backward
// each thread adds up its columns' weight gradients in registers over all of its rows; the blocks' sums are
// joined by a second kernel in a fixed order (no atomics: the result does not change from call to call).
//
// 2^25 values, us, forward / gradients (the copy rate: 51 / 82 bf16, 61 / 102 with fp32 y, 102 / 164 fp32):
//   d           64         128        1024       2048       2500         4096       8192
//   bf16        59 / 110   59 / 115   55 / 121   58 / 133  105 / 197    58 / 115   60 / 127
//   fp32 y      71 / 138   71 / 144   66 / 165   65 / 162  109 / 196    71 / 146   66 / 172
//   fp32       114 / 198  114 / 198  116 / 182  122 / 180  132 / 264   119 / 179  121 / 194
// What is left is the chain of three row sums in the gradients (two in the forward) and, where d is not a
// multiple of 8, bf16 pieces of 8 bytes. With the next row in registers instead of the ring (and 256 threads or
// more, a power of two, per block) the gradients of bf16 took 318, 173, 163, 173, 308, 190 and 235.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace rsm {

namespace {

// VEC values as they stand in memory (16 bytes, or 8, at a time).
template <typename T, int VEC> struct Raw {
  static constexpr int kWords = VEC * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  RSM_DEV void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  RSM_DEV void load(const T* p) {
    if constexpr (kWords == 2) {
      const uint2 t = *reinterpret_cast<const uint2*>(p);
      w[0] = t.x; w[1] = t.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 t = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
        w[i] = t.x; w[i + 1] = t.y; w[i + 2] = t.z; w[i + 3] = t.w;
      }
    }
  }
  // values 2 i and 2 i + 1
  RSM_DEV float2 operator[](int i) const {
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
};

template <typename T, int VEC> RSM_DEV void store_vec(T* p, const float2 (&x)[VEC / 2]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(x[i].x, x[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    if constexpr (VEC == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; i += 2)
      *reinterpret_cast<float4*>(p + 2 * i) = make_float4(x[i].x, x[i].y, x[i + 1].x, x[i + 1].y);
  }
}

// Sums of NV values over the TPR threads of a row (8, 16 or a multiple of 32; every thread of the block
// calls it). `buf` holds one value per warp and NV; successive calls alternate between two buffers,
// so one barrier per call is enough. The second stage reads the warps' sums four at a time.
template <int THREADS, int NV> RSM_DEV void row_sum(float (&v)[NV], int tpr, float (*buf)[32]) {
  if (THREADS <= 128 && tpr < 32) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      for (int o = tpr >> 1; o > 0; o >>= 1) v[k] += __shfl_xor_sync(kFull, v[k], o);
    return;
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) v[k] = warp_sum_f(v[k]);
  if (THREADS <= 128 && tpr == 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) buf[k][warp] = v[k];
  }
  __syncthreads();
  const int nw = tpr >> 5, w0 = nw < 4 ? warp & ~(nw - 1) : 0;  // (2, or a multiple of 4: then the row has the block)
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (nw == 2) {
      v[k] = buf[k][w0] + buf[k][w0 + 1];
    } else {
      float4 s = *reinterpret_cast<const float4*>(&buf[k][w0]);
      for (int w = 4; w < nw; w += 4) {
        const float4 t = *reinterpret_cast<const float4*>(&buf[k][w0 + w]);
        s.x += t.x; s.y += t.y; s.z += t.z; s.w += t.w;
      }
      v[k] = (s.x + s.y) + (s.z + s.w);
    }
  }
}

// The gate is a template argument: a test per element would cost as much as the arithmetic.
enum { kNoGate = 0, kSilu = 1, kSigmoid = 2 };

// act(g) and act'(g). The sigmoid is 1 / (1 + 2^(-g log2 e)) from the approximate exponential and reciprocal
// (2^-22 each, far below what the row sums and the stored types keep): with the exact ones the
// instructions, not the memory, set the pace. A gate of -100 gives 1 / inf = 0.
template <int GATE> RSM_DEV void activation(float2 g, float2& a, float2& slope) {
  if constexpr (GATE == kNoGate) {
    a = both(1.f);
    slope = both(0.f);
  } else {
    const float2 z = mul2(g, both(-1.4426950408889634f));
    float2 e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(z.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(z.y));
    e = add2(e, both(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(e.y));
    const float2 rest = fma2(s, both(-1.f), both(1.f));
    if constexpr (GATE == kSilu) {
      a = mul2(g, s);
      slope = fma2(a, rest, s);
    } else {
      a = s;
      slope = mul2(s, rest);
    }
  }
}

// Rows come through a ring in shared memory that every warp fills, and reads, for itself: no barrier, no
// registers for what is on its way, and a later pass reads again what an earlier one had. Lanes copy
// neighbouring 16 bytes: where a thread's piece has 32 (8 fp32 values), as two copies of its own it would take
// every sector twice (8 values of fp32 y with bf16 otherwise, 2^25 values: 89 us against 74).
template <typename TX, int VEC, int ITER, int THREADS> struct Slot {
  static constexpr int kPiece = VEC * (int)sizeof(TX), kChunk = kPiece < 16 ? kPiece : 16, kPer = kPiece / kChunk;
  static constexpr int kBytes = ITER * kPiece * THREADS;
  // Where chunk q of the warp's stands: pairs change places in every other group of eight, so that eight lanes
  // which read every second chunk meet all banks.
  static RSM_DEV int place(int i, int q) {
    if (kPer == 2) q ^= (q >> 3) & 1;
    return ((i * (THREADS / 32) + (int)(threadIdx.x >> 5)) * 32 * kPer + q) * kChunk;
  }
  // The thread's share of piece i of its warp's lanes in the row, of a row of d that starts at x + at; c is the
  // thread's column.
  static RSM_DEV void copy(unsigned char* slot, int i, const TX* x, int64_t at, int c, int d, bool there, int tpr) {
    const int lane = threadIdx.x & 31, lanes = THREADS > 128 ? 32 : min(tpr, 32), l = lane & (lanes - 1);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int q = lanes * k + l, col = c - l * VEC + q * (VEC / kPer);
      const bool in = there && col < d;
      const uint32_t to = (uint32_t)__cvta_generic_to_shared(slot + place(i, (lane - l) * kPer + q));
      const TX* from = x + (in ? at + col : 0);
      if constexpr (kChunk == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(in ? 8 : 0) : "memory");
    }
  }
  static RSM_DEV Raw<TX, VEC> read(const unsigned char* slot, int i) {
    Raw<TX, VEC> x;
    constexpr int kWords = kChunk / 4;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const unsigned char* at = slot + place(i, kPer * (threadIdx.x & 31) + k);
      if constexpr (kChunk == 16) {
        const uint4 t = *reinterpret_cast<const uint4*>(at);
        x.w[kWords * k] = t.x; x.w[kWords * k + 1] = t.y; x.w[kWords * k + 2] = t.z; x.w[kWords * k + 3] = t.w;
      } else {
        const uint2 t = *reinterpret_cast<const uint2*>(at);
        x.w[0] = t.x; x.w[1] = t.y;
      }
    }
    return x;
  }
};

// y, gate, residual and, for the gradients, dx and dh of one row after the other.
template <typename TY, typename T, int VEC, int ITER, int THREADS, bool BACK> struct Ring {
  using Y = Slot<TY, VEC, ITER, THREADS>;
  using X = Slot<T, VEC, ITER, THREADS>;
  static constexpr int kTensors = BACK ? 5 : 3;
  static constexpr int kStage = Y::kBytes + (kTensors - 1) * X::kBytes;
  // Blocks per SM: as many threads as the registers of a thread's values, weights and sums leave room for.
  static constexpr int kBlocks = (VEC * ITER <= 8 ? 768 : BACK ? 512 : 768) / THREADS;
  static constexpr int kFit = (232448 / kBlocks - 2048) / kStage;
  // (three stages: bf16, rows of 1024, 2^25 values: forward 65 us against 60, gradients 124 against 120)
  static constexpr int kStages = kFit < 2 ? 1 : 2;
  static constexpr int kBytes = kStages * kStage;
  static_assert(kBytes <= 232448 - 2048, "shared memory budget");
  // Rows behind the last one, columns behind d, and what is not given are zeros.
  template <class A> static RSM_DEV void fetch(unsigned char* ring, int stage, const A& a, int64_t row, int t, int tpr) {
    unsigned char* to = ring + stage * kStage;
    const bool there = row < a.rows;
    const int64_t at = there ? row * a.d : 0;
    __syncwarp();  // every lane has read its pieces of the stage
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int c = (t + i * tpr) * VEC;
      Y::copy(to, i, static_cast<const TY*>(a.y), at, c, a.d, there, tpr);
      auto tensor = [&](int k, const void* x) {
        X::copy(to + Y::kBytes + (k - 1) * X::kBytes, i, static_cast<const T*>(x ? x : a.residual), at, c, a.d, there && x, tpr);
      };
      if (a.gate) tensor(1, a.gate);
      tensor(2, a.residual);
      if constexpr (BACK) {
        tensor(3, a.dx);
        tensor(4, a.dh);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // Every lane's part of the oldest stage is there.
  static RSM_DEV void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
  }
  static RSM_DEV Raw<TY, VEC> y(const unsigned char* in, int i) { return Y::read(in, i); }
  static RSM_DEV Raw<T, VEC> x(const unsigned char* in, int k, int i) { return X::read(in + Y::kBytes + (k - 1) * X::kBytes, i); }
};
constexpr int kGate = 1, kResidual = 2, kDx = 3, kDh = 4;  // of the ring

// The blocks stay and take row after row; the next rows are on their way while this one is summed up and
// written (without that, the memory idles during the two row sums: 32768 rows of 2048, fp32 y, 236 us against
// 123 at the copy's rate).
template <typename TY, typename T, int VEC, int ITER, int THREADS, int GATE>
__global__ void __launch_bounds__(THREADS, Ring<TY, T, VEC, ITER, THREADS, false>::kBlocks)
    block_norm_kernel(const rsm_block_norm_args a, int tpr) {
  using R = Ring<TY, T, VEC, ITER, THREADS, false>;
  __shared__ __align__(16) float buf[2][32];
  extern __shared__ __align__(16) unsigned char ring[];
  const int rpb = blockDim.x / tpr;
  const int t = threadIdx.x % tpr;
  const int64_t step = (int64_t)gridDim.x * rpb;
  const float inv_d = 1.f / (float)a.d;
  int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr;
#pragma unroll
  for (int k = 0; k < R::kStages; ++k) R::fetch(ring, k, a, row + k * step, t, tpr);
  Raw<float, VEC> w1[ITER], w2[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int c = (t + i * tpr) * VEC;
    w1[i].zero(); w2[i].zero();
    if (c < a.d) {
      w1[i].load(a.w_post + c);
      if (a.w_pre) w2[i].load(a.w_pre + c);
    }
  }
  int stage = 0;
  // (every thread of the block makes the same number of rounds: the sums hold barriers)
  for (int64_t row0 = (int64_t)blockIdx.x * rpb; row0 < a.rows; row0 += step, row += step) {
    R::wait();
    const unsigned char* in = ring + stage * R::kStage;
    const bool live = row < a.rows;
    const int64_t base = row * a.d;
    float2 acc = both(0.f);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const Raw<TY, VEC> y = R::y(in, i);
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) acc = fma2(y[j], y[j], acc);
    }
    float sum[1] = {acc.x + acc.y};
    row_sum<THREADS>(sum, tpr, &buf[0]);
    const float2 r1 = both(a.scale * rsqrtf(sum[0] * inv_d + a.eps));
    acc = both(0.f);
    float2 h[ITER][VEC / 2];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int c = (t + i * tpr) * VEC;
      const Raw<TY, VEC> y = R::y(in, i);
      const Raw<T, VEC> r = R::x(in, kResidual, i), g = R::x(in, GATE == kNoGate ? kResidual : kGate, i);
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) {
        float2 act, slope;
        activation<GATE>(g[j], act, slope);
        h[i][j] = fma2(mul2(mul2(y[j], r1), w1[i][j]), act, r[j]);
        acc = fma2(h[i][j], h[i][j], acc);
      }
      if (live && c < a.d) store_vec<T, VEC>(static_cast<T*>(a.h) + base + c, h[i]);
    }
    R::fetch(ring, stage, a, row + R::kStages * step, t, tpr);
    stage = stage + 1 == R::kStages ? 0 : stage + 1;
    if (a.w_pre) {
      sum[0] = acc.x + acc.y;
      row_sum<THREADS>(sum, tpr, &buf[1]);
      const float2 r2 = both(rsqrtf(sum[0] * inv_d + a.eps));
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int c = (t + i * tpr) * VEC;
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) h[i][j] = mul2(mul2(h[i][j], r2), w2[i][j]);
        if (live && c < a.d) store_vec<T, VEC>(static_cast<T*>(a.x) + base + c, h[i]);
      }
    } else {
      __syncthreads();  // buf[0] is written again in the next round
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename TY, typename T, int VEC, int ITER, int THREADS, int GATE>
__global__ void __launch_bounds__(THREADS, Ring<TY, T, VEC, ITER, THREADS, true>::kBlocks)
    block_norm_backward_kernel(const rsm_block_norm_backward_args a, int tpr) {
  using R = Ring<TY, T, VEC, ITER, THREADS, true>;
  __shared__ __align__(16) float buf[2][2][32];
  extern __shared__ __align__(16) unsigned char ring[];
  const int rpb = blockDim.x / tpr;
  const int sub = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int64_t step = (int64_t)gridDim.x * rpb;
  const float inv_d = 1.f / (float)a.d;
  int64_t row = (int64_t)blockIdx.x * rpb + sub;
#pragma unroll
  for (int k = 0; k < R::kStages; ++k) R::fetch(ring, k, a, row + k * step, t, tpr);
  Raw<float, VEC> w1[ITER], w2[ITER];
  float2 s1[ITER][VEC / 2], s2[ITER][VEC / 2];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int c = (t + i * tpr) * VEC;
    w1[i].zero(); w2[i].zero();
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) s1[i][j] = s2[i][j] = both(0.f);
    if (c < a.d) {
      w1[i].load(a.w_post + c);
      if (a.w_pre) w2[i].load(a.w_pre + c);
    }
  }
  int stage = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * rpb; row0 < a.rows; row0 += step, row += step) {
    R::wait();
    const unsigned char* in = ring + stage * R::kStage;
    const bool live = row < a.rows;
    const int64_t base = row * a.d;
    float2 acc = both(0.f);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const Raw<TY, VEC> y = R::y(in, i);
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) acc = fma2(y[j], y[j], acc);
    }
    float one[1] = {acc.x + acc.y};
    row_sum<THREADS>(one, tpr, &buf[0][0]);
    const float rs1 = rsqrtf(one[0] * inv_d + a.eps);
    const float2 r1 = both(rs1), r1s = both(a.scale * rs1);
    float2 acc2 = acc = both(0.f);
    float2 h[ITER][VEC / 2];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const Raw<TY, VEC> y = R::y(in, i);
      const Raw<T, VEC> r = R::x(in, kResidual, i), dx = R::x(in, kDx, i), g = R::x(in, GATE == kNoGate ? kResidual : kGate, i);
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) {
        float2 act, slope;
        activation<GATE>(g[j], act, slope);
        h[i][j] = fma2(mul2(mul2(y[j], r1s), w1[i][j]), act, r[j]);
        acc = fma2(h[i][j], h[i][j], acc);
        acc2 = fma2(mul2(dx[j], w2[i][j]), h[i][j], acc2);
      }
    }
    float two[2] = {acc.x + acc.y, acc2.x + acc2.y};
    row_sum<THREADS>(two, tpr, &buf[1][0]);
    const float rs2 = rsqrtf(two[0] * inv_d + a.eps);
    const float2 r2 = both(rs2), k2 = both(-rs2 * (rs2 * (two[1] * inv_d))), al = both(a.scale);
    acc = both(0.f);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int c = (t + i * tpr) * VEC;
      const Raw<TY, VEC> yy = R::y(in, i);
      const Raw<T, VEC> dxx = R::x(in, kDx, i), dh = R::x(in, kDh, i), g = R::x(in, GATE == kNoGate ? kResidual : kGate, i);
      float2 dg[VEC / 2], dH[VEC / 2];
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) {
        float2 act, slope;
        activation<GATE>(g[j], act, slope);
        const float2 dx = dxx[j], y = yy[j], hn = mul2(h[i][j], r2);
        s2[i][j] = fma2(dx, hn, s2[i][j]);
        dH[j] = fma2(hn, k2, fma2(mul2(dx, w2[i][j]), r2, dh[j]));
        const float2 du = mul2(dH[j], al), ya = mul2(y, r1), dn = mul2(du, act);
        if (GATE != kNoGate) dg[j] = mul2(mul2(du, slope), mul2(ya, w1[i][j]));
        s1[i][j] = fma2(dn, ya, s1[i][j]);
        h[i][j] = mul2(dn, w1[i][j]);  // f
        acc = fma2(h[i][j], y, acc);
      }
      if (live && c < a.d) {
        if (a.dresidual) store_vec<T, VEC>(static_cast<T*>(a.dresidual) + base + c, dH);
        if (GATE != kNoGate && a.dgate) store_vec<T, VEC>(static_cast<T*>(a.dgate) + base + c, dg);
      }
    }
    one[0] = acc.x + acc.y;
    row_sum<THREADS>(one, tpr, &buf[0][1]);
    const float2 k1 = both(-rs1 * (rs1 * (one[0] * inv_d)));
    if (a.dy) {
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int c = (t + i * tpr) * VEC;
        const Raw<TY, VEC> y = R::y(in, i);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) h[i][j] = fma2(mul2(y[j], r1), k1, mul2(h[i][j], r1));
        if (live && c < a.d) store_vec<TY, VEC>(static_cast<TY*>(a.dy) + base + c, h[i]);
      }
    }
    R::fetch(ring, stage, a, row + R::kStages * step, t, tpr);
    stage = stage + 1 == R::kStages ? 0 : stage + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  float* part = static_cast<float*>(a.workspace) + (int64_t)blockIdx.x * 2 * a.d;
  if (rpb == 1) {
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int c = (t + i * tpr) * VEC;
      if (c < a.d) {
        store_vec<float, VEC>(part + c, s1[i]);
        store_vec<float, VEC>(part + a.d + c, s2[i]);
      }
    }
    return;
  }
  // the block's rows join where the ring was ([rpb][2][d], which is smaller)
  float* sums = reinterpret_cast<float*>(ring);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int c = (t + i * tpr) * VEC;
    if (c < a.d) {
      store_vec<float, VEC>(sums + sub * 2 * a.d + c, s1[i]);
      store_vec<float, VEC>(sums + sub * 2 * a.d + a.d + c, s2[i]);
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * a.d; c += blockDim.x) {
    float s = 0.f;
    for (int k = 0; k < rpb; ++k) s += sums[k * 2 * a.d + c];
    part[c] = s;
  }
}

// dw[c] = sum over the blocks' partial sums, 8 strided sums per column joined in shared memory (the
// same order in every call).
__global__ void __launch_bounds__(256) weight_sum_kernel(const float* part, int nparts, int d, float* dw_post,
                                                         float* dw_pre) {
  __shared__ float s[8][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  float sum = 0.f;
  if (col < 2 * d)
    for (int i = k; i < nparts; i += 8) sum += part[(int64_t)i * 2 * d + col];
  s[k][threadIdx.x & 31] = sum;
  __syncthreads();
  if (k == 0 && col < 2 * d) {
    for (int i = 1; i < 8; ++i) sum += s[i][threadIdx.x & 31];
    float* out = col < d ? dw_post : dw_pre;
    if (out) out[col < d ? col : col - d] = sum;
  }
}

// Threads and values per thread for a row of d: pieces of `vec` values (16 bytes where the rows allow it), 8
// values per thread up to 256 threads, then 16 up to 512 threads. (4, where a row has
// 32 values or less and 8 lanes.) A row has a block of its own from 128 threads on: rows that share barriers wait for
// one another (32768 rows of 1024, gradients: blocks of 256 threads 163 us, of 128 139).
struct Shape {
  int vec, tpr, iter, threads;
};
Shape shape_for(int d, rsm_dtype dtype) {
  Shape s;
  s.vec = dtype == RSM_BF16 && d % 8 == 0 ? 8 : 4;
  const int pieces = (d + s.vec - 1) / s.vec;
  s.iter = pieces <= 8 ? 1 : (d <= 2048 ? 8 : 16) / s.vec;
  const int per = (pieces + s.iter - 1) / s.iter;
  s.tpr = per <= 8 ? 8 : per <= 16 ? 16 : per <= 32 ? 32 : per <= 64 ? 64 : (per + 127) / 128 * 128;
  s.threads = std::max(s.tpr, 128);
  return s;
}
// Block size that the kernels are compiled for.
int compiled_threads(const Shape& s) { return s.threads <= 128 ? 128 : s.threads <= 256 ? 256 : 512; }
// As many blocks as stay resident, and no more than there are rows for.
int blocks_for(int64_t rows, const Shape& s, int per_sm) {
  const int rpb = s.threads / s.tpr;
  return (int)std::min<int64_t>((rows + rpb - 1) / rpb, (int64_t)per_sm * device_sm_count());
}
int backward_blocks(int64_t rows, const Shape& s) {
  return blocks_for(rows, s, (s.vec * s.iter <= 8 ? 768 : 512) / compiled_threads(s));
}

template <class A> int gate_of(const A& a) { return !a.gate ? kNoGate : a.act == RSM_ACT_SILU ? kSilu : kSigmoid; }

// Calls f with the block size and the gate as compile-time constants.
template <int VALUES, class F> cudaError_t with_constants(int threads, int gate, F f) {
  auto gated = [&](auto t) {
    if (gate == kNoGate) return f(t, std::integral_constant<int, kNoGate>());
    if (gate == kSilu) return f(t, std::integral_constant<int, kSilu>());
    return f(t, std::integral_constant<int, kSigmoid>());
  };
  if constexpr (VALUES <= 8) {
    if (threads == 128) return gated(std::integral_constant<int, 128>());
  }
  if constexpr (VALUES >= 8) {
    if (threads == 256) return gated(std::integral_constant<int, 256>());
  }
  if constexpr (VALUES == 16) {
    if (threads == 512) return gated(std::integral_constant<int, 512>());
  }
  return cudaErrorInvalidConfiguration;
}

template <typename TY, typename T, int VEC, int ITER>
cudaError_t forward_as(const rsm_block_norm_args& a, const Shape& s, cudaStream_t stream) {
  return with_constants<VEC * ITER>(compiled_threads(s), gate_of(a), [&](auto threads, auto gate) {
    using R = Ring<TY, T, VEC, ITER, decltype(threads)::value, false>;
    constexpr auto* kernel = block_norm_kernel<TY, T, VEC, ITER, decltype(threads)::value, decltype(gate)::value>;
    cudaError_t e = set_smem_limit<kernel>(R::kBytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)blocks_for(a.rows, s, R::kBlocks), s.threads, R::kBytes, stream>>>(a, s.tpr);
    return cudaGetLastError();
  });
}

template <typename TY, typename T, int VEC, int ITER>
cudaError_t backward_as(const rsm_block_norm_backward_args& a, const Shape& s, cudaStream_t stream) {
  const int grid = backward_blocks(a.rows, s);
  cudaError_t e = with_constants<VEC * ITER>(compiled_threads(s), gate_of(a), [&](auto threads, auto gate) {
    using R = Ring<TY, T, VEC, ITER, decltype(threads)::value, true>;
    constexpr auto* kernel = block_norm_backward_kernel<TY, T, VEC, ITER, decltype(threads)::value, decltype(gate)::value>;
    cudaError_t e = set_smem_limit<kernel>(R::kBytes);
    if (e != cudaSuccess) return e;
    kernel<<<grid, s.threads, R::kBytes, stream>>>(a, s.tpr);
    return cudaGetLastError();
  });
  if (e != cudaSuccess || !(a.dw_post || a.dw_pre)) return e;
  weight_sum_kernel<<<(2 * a.d + 31) / 32, 256, 0, stream>>>(static_cast<const float*>(a.workspace), grid, a.d,
                                                             a.dw_post, a.dw_pre);
  return cudaGetLastError();
}

// Calls f with the types and the shape as compile-time constants.
template <class F> cudaError_t dispatch(rsm_dtype y_dtype, rsm_dtype dtype, const Shape& s, F f) {
  auto four = [&](auto ty, auto t) {
    if (s.iter == 1) return f(ty, t, std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
    if (s.iter == 2) return f(ty, t, std::integral_constant<int, 4>(), std::integral_constant<int, 2>());
    return f(ty, t, std::integral_constant<int, 4>(), std::integral_constant<int, 4>());
  };
  auto shaped = [&](auto ty, auto t) {
    if (s.vec == 4) return four(ty, t);
    if (s.iter == 1) return f(ty, t, std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
    return f(ty, t, std::integral_constant<int, 8>(), std::integral_constant<int, 2>());
  };
  if (dtype == RSM_F32) return four(float(), float());
  if (y_dtype == RSM_F32) return shaped(float(), __nv_bfloat16());
  return shaped(__nv_bfloat16(), __nv_bfloat16());
}

}  // namespace

cudaError_t launch_block_norm(const rsm_block_norm_args& a, cudaStream_t stream) {
  const Shape s = shape_for(a.d, a.dtype);
  return dispatch(a.y_dtype, a.dtype, s, [&](auto ty, auto t, auto vec, auto iter) {
    return forward_as<decltype(ty), decltype(t), decltype(vec)::value, decltype(iter)::value>(a, s, stream);
  });
}

size_t block_norm_backward_workspace_bytes(const rsm_block_norm_backward_args& a) {
  return (size_t)backward_blocks(a.rows, shape_for(a.d, a.dtype)) * 2 * a.d * sizeof(float);
}

cudaError_t launch_block_norm_backward(const rsm_block_norm_backward_args& a, cudaStream_t stream) {
  const Shape s = shape_for(a.d, a.dtype);
  return dispatch(a.y_dtype, a.dtype, s, [&](auto ty, auto t, auto vec, auto iter) {
    return backward_as<decltype(ty), decltype(t), decltype(vec)::value, decltype(iter)::value>(a, s, stream);
  });
}

}  // namespace rsm
