// block_norm.cu -- the norms around a block, fused with its output gate and residual scale, and
// their gradients (rsm_block_norm_forward, rsm_block_norm_backward).
//
//   r1 = rsqrt(mean(y^2) + eps),  n = y r1 w_post,  h = res + scale n act(g)
//   r2 = rsqrt(mean(h^2) + eps),  x = h r2 w_pre
// and, with e = dx w_pre,
//   dH = dh + r2 e - h r2^3 mean(e h),  dres = dH,  du = scale dH
//   dg = du n act'(g),  f = du act(g) w_post,  dy = r1 f - y r1^3 mean(f y)
//   dw_post = sum_rows du act(g) y r1,  dw_pre = sum_rows dx h r2
// Everything is fp32, two values per instruction, between the loads and the stores; h is normalised before it is rounded, and the
// backward forms it again from its inputs, so no rounded value enters a sum.
//
// A row stays in registers: TPR threads hold VEC * ITER values each, and the row crosses memory once
// (bound: HBM bandwidth). The row sums go over shuffles and, past one warp, one exchange in shared
// memory. In the backward each thread adds up its columns' weight gradients in registers over all of its
// rows; the blocks' sums are joined by a second kernel in a fixed order (no atomics: the result does not
// change from call to call).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace rsm {

namespace {

constexpr int kMaxThreads = 512;

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

// Sums of NV values over the TPR threads of a row (TPR a multiple of 32; every thread of the block
// calls it). `buf` holds one value per warp and NV; successive calls alternate between two buffers,
// so one barrier per call is enough. The second stage reads the warps' sums four at a time.
template <int NV> RSM_DEV void row_sum(float (&v)[NV], int tpr, float (*buf)[32]) {
#pragma unroll
  for (int k = 0; k < NV; ++k) v[k] = warp_sum_f(v[k]);
  if (tpr == 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) buf[k][warp] = v[k];
  }
  __syncthreads();
  const int nw = tpr >> 5, w0 = warp & ~(nw - 1);  // (nw is a power of two, 2 to 16)
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

// What a thread holds of a row. Rows behind the last one, and columns behind d, are zero.
template <typename TY, typename T, int VEC, int ITER, bool GATED> struct Row {
  Raw<TY, VEC> y[ITER];
  Raw<T, VEC> g[ITER], r[ITER];
  template <class A> RSM_DEV void load(const A& a, int64_t row, int t, int tpr) {
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int c = (t + i * tpr) * VEC;
      y[i].zero(); g[i].zero(); r[i].zero();
      if (row < a.rows && c < a.d) {
        const int64_t at = row * a.d + c;
        y[i].load(static_cast<const TY*>(a.y) + at);
        if (GATED) g[i].load(static_cast<const T*>(a.gate) + at);
        r[i].load(static_cast<const T*>(a.residual) + at);
      }
    }
  }
};
template <typename T, int VEC, int ITER> struct Grads {
  Raw<T, VEC> dx[ITER], dh[ITER];
  template <class A> RSM_DEV void load(const A& a, int64_t row, int t, int tpr) {
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int c = (t + i * tpr) * VEC;
      dx[i].zero(); dh[i].zero();
      if (row < a.rows && c < a.d) {
        const int64_t at = row * a.d + c;
        if (a.dx) dx[i].load(static_cast<const T*>(a.dx) + at);
        if (a.dh) dh[i].load(static_cast<const T*>(a.dh) + at);
      }
    }
  }
};

// The blocks stay and take row after row. Where a row is one piece per thread (ITER = 1) the next row is on
// its way while this one is summed up and written: without that, the memory idles during the two row sums
// (32768 rows of 2048, fp32 y: 236 us against 123 at the copy's rate).
template <typename TY, typename T, int VEC, int ITER, int THREADS, int GATE>
__global__ void __launch_bounds__(THREADS, ITER == 1 ? 768 / THREADS : 1) block_norm_kernel(const rsm_block_norm_args a, int tpr) {
  __shared__ __align__(16) float buf[2][32];
  const int rpb = blockDim.x / tpr;
  const int t = threadIdx.x % tpr;
  const int64_t step = (int64_t)gridDim.x * rpb;
  const float inv_d = 1.f / (float)a.d;
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
  Row<TY, T, VEC, ITER, GATE != kNoGate> next;
  int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr;
  if (ITER == 1) next.load(a, row, t, tpr);
  // (every thread of the block makes the same number of rounds: the sums hold barriers)
  for (int64_t row0 = (int64_t)blockIdx.x * rpb; row0 < a.rows; row0 += step, row += step) {
    Row<TY, T, VEC, ITER, GATE != kNoGate> in;
    if (ITER == 1) {
      in = next;
      next.load(a, row + step, t, tpr);
    } else {
      in.load(a, row, t, tpr);
    }
    const bool live = row < a.rows;
    const int64_t base = row * a.d;
    float2 acc = both(0.f);
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) acc = fma2(in.y[i][j], in.y[i][j], acc);
    float sum[1] = {acc.x + acc.y};
    row_sum(sum, tpr, &buf[0]);
    const float2 r1 = both(a.scale * rsqrtf(sum[0] * inv_d + a.eps));
    acc = both(0.f);
    float2 h[ITER][VEC / 2];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int c = (t + i * tpr) * VEC;
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) {
        float2 act, slope;
        activation<GATE>(in.g[i][j], act, slope);
        h[i][j] = fma2(mul2(mul2(in.y[i][j], r1), w1[i][j]), act, in.r[i][j]);
        acc = fma2(h[i][j], h[i][j], acc);
      }
      if (live && c < a.d) store_vec<T, VEC>(static_cast<T*>(a.h) + base + c, h[i]);
    }
    if (a.w_pre) {
      sum[0] = acc.x + acc.y;
      row_sum(sum, tpr, &buf[1]);
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
}

template <typename TY, typename T, int VEC, int ITER, int THREADS, int GATE>
__global__ void __launch_bounds__(THREADS, 512 / THREADS)
    block_norm_backward_kernel(const rsm_block_norm_backward_args a, int tpr) {
  __shared__ __align__(16) float buf[2][2][32];
  extern __shared__ float sums[];  // [rpb][2][d]: joins the rows of a block, rpb > 1 only
  const int rpb = blockDim.x / tpr;
  const int sub = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int64_t step = (int64_t)gridDim.x * rpb;
  const float inv_d = 1.f / (float)a.d;
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
  Row<TY, T, VEC, ITER, GATE != kNoGate> next;
  Grads<T, VEC, ITER> next_d;
  int64_t row = (int64_t)blockIdx.x * rpb + sub;
  if (ITER == 1) {
    next.load(a, row, t, tpr);
    next_d.load(a, row, t, tpr);
  }
  for (int64_t row0 = (int64_t)blockIdx.x * rpb; row0 < a.rows; row0 += step, row += step) {
    Row<TY, T, VEC, ITER, GATE != kNoGate> in;
    Grads<T, VEC, ITER> d;
    if (ITER == 1) {
      in = next;
      d = next_d;
      next.load(a, row + step, t, tpr);
      next_d.load(a, row + step, t, tpr);
    } else {
      in.load(a, row, t, tpr);
      d.load(a, row, t, tpr);
    }
    const bool live = row < a.rows;
    const int64_t base = row * a.d;
    float2 acc = both(0.f);
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) acc = fma2(in.y[i][j], in.y[i][j], acc);
    float one[1] = {acc.x + acc.y};
    row_sum(one, tpr, &buf[0][0]);
    const float rs1 = rsqrtf(one[0] * inv_d + a.eps);
    const float2 r1 = both(rs1), r1s = both(a.scale * rs1);
    float2 acc2 = acc = both(0.f);
    float2 h[ITER][VEC / 2];
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) {
        float2 act, slope;
        activation<GATE>(in.g[i][j], act, slope);
        h[i][j] = fma2(mul2(mul2(in.y[i][j], r1s), w1[i][j]), act, in.r[i][j]);
        acc = fma2(h[i][j], h[i][j], acc);
        acc2 = fma2(mul2(d.dx[i][j], w2[i][j]), h[i][j], acc2);
      }
    float two[2] = {acc.x + acc.y, acc2.x + acc2.y};
    row_sum(two, tpr, &buf[1][0]);
    const float rs2 = rsqrtf(two[0] * inv_d + a.eps);
    const float2 r2 = both(rs2), k2 = both(-rs2 * rs2 * rs2 * (two[1] * inv_d)), al = both(a.scale);
    acc = both(0.f);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int c = (t + i * tpr) * VEC;
      float2 dg[VEC / 2], dH[VEC / 2];
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) {
        float2 act, slope;
        activation<GATE>(in.g[i][j], act, slope);
        const float2 dx = d.dx[i][j], y = in.y[i][j];
        s2[i][j] = fma2(mul2(dx, h[i][j]), r2, s2[i][j]);
        dH[j] = fma2(h[i][j], k2, fma2(mul2(dx, w2[i][j]), r2, d.dh[i][j]));
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
    row_sum(one, tpr, &buf[0][1]);
    const float2 k1 = both(-rs1 * rs1 * rs1 * (one[0] * inv_d));
    if (a.dy) {
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int c = (t + i * tpr) * VEC;
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) h[i][j] = fma2(in.y[i][j], k1, mul2(h[i][j], r1));
        if (live && c < a.d) store_vec<TY, VEC>(static_cast<TY*>(a.dy) + base + c, h[i]);
      }
    }
  }
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

// Threads and values per thread for a row of d: pieces of `vec` values, the fewest threads (a power of two,
// at least a warp) that hold the row in one piece each, at most 512.
struct Shape {
  int vec, tpr, iter, threads;
};
Shape shape_of(int d, int vec) {
  Shape s;
  s.vec = vec;
  const int pieces = d / s.vec;
  s.tpr = 32;
  while (s.tpr < pieces && s.tpr < kMaxThreads) s.tpr *= 2;
  s.iter = (pieces + s.tpr - 1) / s.tpr;
  s.iter = s.iter <= 2 ? s.iter : 4;
  s.threads = std::max(s.tpr, 256);
  return s;
}
// 16-byte pieces where the rows allow it
Shape shape_for(int d, rsm_dtype dtype) { return shape_of(d, dtype == RSM_BF16 && d % 8 == 0 ? 8 : 4); }
int backward_blocks(int64_t rows, const Shape& s) {
  const int rpb = s.threads / s.tpr;
  const int64_t need = (rows + rpb - 1) / rpb;
  return (int)std::min<int64_t>(need, (int64_t)(512 / s.threads) * device_sm_count());
}

template <class A> int gate_of(const A& a) { return !a.gate ? kNoGate : a.act == RSM_ACT_SILU ? kSilu : kSigmoid; }

// Calls f with the block size and the gate as compile-time constants. (Rows of more than one piece per
// thread always take the larger block.)
template <int ITER, class F> void with_constants(int threads, int gate, F f) {
  auto gated = [&](auto t) {
    if (gate == kNoGate) f(t, std::integral_constant<int, kNoGate>());
    else if (gate == kSilu) f(t, std::integral_constant<int, kSilu>());
    else f(t, std::integral_constant<int, kSigmoid>());
  };
  if constexpr (ITER == 1) {
    if (threads == 256) return gated(std::integral_constant<int, 256>());
  }
  gated(std::integral_constant<int, 512>());
}

template <typename TY, typename T, int VEC, int ITER>
cudaError_t forward_as(const rsm_block_norm_args& a, const Shape& s, cudaStream_t stream) {
  const int rpb = s.threads / s.tpr;
  const int64_t need = (a.rows + rpb - 1) / rpb;
  const int64_t grid = std::min<int64_t>(need, (int64_t)(768 / s.threads) * device_sm_count());
  with_constants<ITER>(s.threads, gate_of(a), [&](auto threads, auto gate) {
    block_norm_kernel<TY, T, VEC, ITER, decltype(threads)::value, decltype(gate)::value>
        <<<(unsigned)grid, s.threads, 0, stream>>>(a, s.tpr);
  });
  return cudaGetLastError();
}

template <typename TY, typename T, int VEC, int ITER>
cudaError_t backward_as(const rsm_block_norm_backward_args& a, const Shape& s, cudaStream_t stream) {
  const int rpb = s.threads / s.tpr;
  const int bytes = rpb > 1 ? rpb * 2 * a.d * 4 : 0;  // at most 8 * 2 * 256 * 4
  const int grid = backward_blocks(a.rows, s);
  with_constants<ITER>(s.threads, gate_of(a), [&](auto threads, auto gate) {
    block_norm_backward_kernel<TY, T, VEC, ITER, decltype(threads)::value, decltype(gate)::value>
        <<<grid, s.threads, bytes, stream>>>(a, s.tpr);
  });
  cudaError_t e = cudaGetLastError();
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
