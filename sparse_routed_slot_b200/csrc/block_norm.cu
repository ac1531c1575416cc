// block_norm.cu -- the norms around a block, fused with its output gate and residual scale, and
// their gradients (rsm_block_norm_forward, rsm_block_norm_backward).
//
//   r1 = rsqrt(mean(y^2) + eps),  n = y r1 w_post,  h = res + scale n act(g)
//   r2 = rsqrt(mean(h^2) + eps),  x = h r2 w_pre
// and, with e = dx w_pre,
//   dH = dh + r2 e - h r2^3 mean(e h),  dres = dH,  du = scale dH
//   dg = du n act'(g),  f = du act(g) w_post,  dy = r1 f - y r1^3 mean(f y)
//   dw_post = sum_rows du act(g) y r1,  dw_pre = sum_rows dx h r2
// Everything is fp32 between the loads and the stores; h is normalised before it is rounded, and the
// backward forms it again from its inputs, so no rounded value enters a sum.
//
// A row stays in registers: TPR threads hold VEC * ITER values each, and the row crosses memory once
// (bound: HBM bandwidth). The row sums go over shuffles and, past one warp, one exchange in shared
// memory. The forward runs one row per TPR threads; the backward is persistent, so that each thread
// adds up its columns' weight gradients in registers over all of its rows; the blocks' sums are joined
// by a second kernel in a fixed order (no atomics: the result does not change from call to call).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace rsm {

namespace {

constexpr int kMaxThreads = 512;

template <typename T, int VEC> RSM_DEV void load_vec(const T* p, float (&x)[VEC]) {
  if constexpr (sizeof(T) == 2 && VEC == 8) {
    const uint4 t = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      float t[4];
      In<T>::ld4(p + i, t);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i + j] = t[j];
    }
  }
}

template <typename T, int VEC> RSM_DEV void store_vec(T* p, const float (&x)[VEC]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    if constexpr (VEC == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  }
}

// Sums of NV values over the TPR threads of a row (TPR a multiple of 32; every thread of the block
// calls it). `buf` holds one value per warp and NV; successive calls alternate between two buffers,
// so one barrier per call is enough.
template <int NV> RSM_DEV void row_sum(float (&v)[NV], int tpr, float* buf) {
#pragma unroll
  for (int k = 0; k < NV; ++k) v[k] = warp_sum_f(v[k]);
  if (tpr == 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) buf[k * 32 + warp] = v[k];
  }
  __syncthreads();
  const int nw = tpr >> 5, w0 = warp / nw * nw;
#pragma unroll
  for (int k = 0; k < NV; ++k) v[k] = warp_sum_f(lane < nw ? buf[k * 32 + w0 + lane] : 0.f);
}

RSM_DEV void activation(rsm_act act, float g, float& a, float& slope) {
  const float s = sigmoid_f32(g);
  if (act == RSM_ACT_SILU) {
    a = g * s;
    slope = s * (1.f + g * (1.f - s));
  } else {
    a = s;
    slope = s * (1.f - s);
  }
}

template <typename TY, typename T, int VEC, int ITER>
__global__ void __launch_bounds__(kMaxThreads) block_norm_kernel(const rsm_block_norm_args a, int tpr) {
  __shared__ float buf[2][32];
  const int rpb = blockDim.x / tpr;
  const int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr;
  const int t = threadIdx.x % tpr;
  const bool live = row < a.rows;
  const int64_t base = row * a.d;
  float y[ITER][VEC], g[ITER][VEC], r[ITER][VEC], w1[ITER][VEC], w2[ITER][VEC];
  float sum[1] = {0.f};
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int c = (t + i * tpr) * VEC;
    const bool in = live && c < a.d;
#pragma unroll
    for (int j = 0; j < VEC; ++j) y[i][j] = g[i][j] = r[i][j] = w1[i][j] = w2[i][j] = 0.f;
    if (in) {
      load_vec<TY, VEC>(static_cast<const TY*>(a.y) + base + c, y[i]);
      if (a.gate) load_vec<T, VEC>(static_cast<const T*>(a.gate) + base + c, g[i]);
      load_vec<T, VEC>(static_cast<const T*>(a.residual) + base + c, r[i]);
      load_vec<float, VEC>(a.w_post + c, w1[i]);
      if (a.w_pre) load_vec<float, VEC>(a.w_pre + c, w2[i]);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum[0] = fmaf(y[i][j], y[i][j], sum[0]);
  }
  const float inv_d = 1.f / (float)a.d;
  row_sum(sum, tpr, buf[0]);
  const float r1 = rsqrtf(sum[0] * inv_d + a.eps);
  sum[0] = 0.f;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int c = (t + i * tpr) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      float act = 1.f, slope;
      if (a.gate) activation(a.act, g[i][j], act, slope);
      r[i][j] = fmaf(a.scale * (y[i][j] * r1 * w1[i][j]), act, r[i][j]);
      sum[0] = fmaf(r[i][j], r[i][j], sum[0]);
    }
    if (live && c < a.d) store_vec<T, VEC>(static_cast<T*>(a.h) + base + c, r[i]);
  }
  if (!a.w_pre) return;
  row_sum(sum, tpr, buf[1]);
  const float r2 = rsqrtf(sum[0] * inv_d + a.eps);
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int c = (t + i * tpr) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) r[i][j] = r[i][j] * r2 * w2[i][j];
    if (live && c < a.d) store_vec<T, VEC>(static_cast<T*>(a.x) + base + c, r[i]);
  }
}

template <typename TY, typename T, int VEC, int ITER>
__global__ void __launch_bounds__(kMaxThreads) block_norm_backward_kernel(const rsm_block_norm_backward_args a, int tpr) {
  __shared__ float buf[2][2][32];
  extern __shared__ float sums[];  // [rpb][2][d]: joins the rows of a block, rpb > 1 only
  const int rpb = blockDim.x / tpr;
  const int sub = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const float inv_d = 1.f / (float)a.d;
  float w1[ITER][VEC], w2[ITER][VEC], s1[ITER][VEC], s2[ITER][VEC];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int c = (t + i * tpr) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) w1[i][j] = w2[i][j] = s1[i][j] = s2[i][j] = 0.f;
    if (c < a.d) {
      load_vec<float, VEC>(a.w_post + c, w1[i]);
      if (a.w_pre) load_vec<float, VEC>(a.w_pre + c, w2[i]);
    }
  }
  for (int64_t row0 = (int64_t)blockIdx.x * rpb; row0 < a.rows; row0 += (int64_t)gridDim.x * rpb) {
    const int64_t row = row0 + sub;
    const bool live = row < a.rows;
    const int64_t base = row * a.d;
    float y[ITER][VEC], g[ITER][VEC], h[ITER][VEC], dx[ITER][VEC], dh[ITER][VEC];
    float one[1] = {0.f};
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int c = (t + i * tpr) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) y[i][j] = g[i][j] = h[i][j] = dx[i][j] = dh[i][j] = 0.f;
      if (live && c < a.d) {
        load_vec<TY, VEC>(static_cast<const TY*>(a.y) + base + c, y[i]);
        if (a.gate) load_vec<T, VEC>(static_cast<const T*>(a.gate) + base + c, g[i]);
        load_vec<T, VEC>(static_cast<const T*>(a.residual) + base + c, h[i]);
        if (a.dx) load_vec<T, VEC>(static_cast<const T*>(a.dx) + base + c, dx[i]);
        if (a.dh) load_vec<T, VEC>(static_cast<const T*>(a.dh) + base + c, dh[i]);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) one[0] = fmaf(y[i][j], y[i][j], one[0]);
    }
    row_sum(one, tpr, buf[0][0]);
    const float r1 = rsqrtf(one[0] * inv_d + a.eps);
    float two[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float act = 1.f, slope;
        if (a.gate) activation(a.act, g[i][j], act, slope);
        h[i][j] = fmaf(a.scale * (y[i][j] * r1 * w1[i][j]), act, h[i][j]);
        two[0] = fmaf(h[i][j], h[i][j], two[0]);
        two[1] = fmaf(dx[i][j] * w2[i][j], h[i][j], two[1]);
      }
    row_sum(two, tpr, buf[1][0]);
    const float r2 = rsqrtf(two[0] * inv_d + a.eps);
    const float k2 = r2 * r2 * r2 * (two[1] * inv_d);
    one[0] = 0.f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int c = (t + i * tpr) * VEC;
      float dg[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float act = 1.f, slope = 0.f;
        if (a.gate) activation(a.act, g[i][j], act, slope);
        s2[i][j] = fmaf(dx[i][j] * h[i][j], r2, s2[i][j]);
        const float dH = dh[i][j] + (r2 * (dx[i][j] * w2[i][j]) - h[i][j] * k2);
        dh[i][j] = dH;
        const float du = a.scale * dH;
        const float yr = y[i][j] * r1;
        dg[j] = du * (yr * w1[i][j]) * slope;
        s1[i][j] = fmaf(du * act, yr, s1[i][j]);
        h[i][j] = du * act * w1[i][j];  // f
        one[0] = fmaf(h[i][j], y[i][j], one[0]);
      }
      if (live && c < a.d) {
        if (a.dresidual) store_vec<T, VEC>(static_cast<T*>(a.dresidual) + base + c, dh[i]);
        if (a.dgate) store_vec<T, VEC>(static_cast<T*>(a.dgate) + base + c, dg);
      }
    }
    row_sum(one, tpr, buf[0][1]);
    const float k1 = r1 * r1 * r1 * (one[0] * inv_d);
    if (a.dy) {
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        const int c = (t + i * tpr) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[i][j] = r1 * h[i][j] - y[i][j] * k1;
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

// Threads and values per thread for a row of d: 16-byte bf16 pieces where the rows allow it, the
// fewest threads (a power of two, at least a warp) that hold the row in one piece each, at most 512.
struct Shape {
  int vec, tpr, iter, threads;
};
Shape shape_for(int d) {
  Shape s;
  s.vec = d % 8 == 0 ? 8 : 4;
  const int pieces = d / s.vec;
  s.tpr = 32;
  while (s.tpr < pieces && s.tpr < kMaxThreads) s.tpr *= 2;
  s.iter = (pieces + s.tpr - 1) / s.tpr;
  s.iter = s.iter <= 2 ? s.iter : 4;
  s.threads = std::max(s.tpr, 256);
  return s;
}

int backward_blocks(int64_t rows, const Shape& s) {
  const int rpb = s.threads / s.tpr;
  const int64_t need = (rows + rpb - 1) / rpb;
  const int per_sm = std::max(1, 1024 / s.threads);
  return (int)std::min<int64_t>(need, (int64_t)per_sm * device_sm_count());
}

template <typename TY, typename T, int VEC, int ITER>
cudaError_t forward_as(const rsm_block_norm_args& a, const Shape& s, cudaStream_t stream) {
  const int rpb = s.threads / s.tpr;
  const int64_t grid = (a.rows + rpb - 1) / rpb;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  block_norm_kernel<TY, T, VEC, ITER><<<(unsigned)grid, s.threads, 0, stream>>>(a, s.tpr);
  return cudaGetLastError();
}

template <typename TY, typename T, int VEC, int ITER>
cudaError_t backward_as(const rsm_block_norm_backward_args& a, const Shape& s, cudaStream_t stream) {
  const int rpb = s.threads / s.tpr;
  const int bytes = rpb > 1 ? rpb * 2 * a.d * 4 : 0;  // at most 8 * 2 * 256 * 4
  const int grid = backward_blocks(a.rows, s);
  block_norm_backward_kernel<TY, T, VEC, ITER><<<grid, s.threads, bytes, stream>>>(a, s.tpr);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !(a.dw_post || a.dw_pre)) return e;
  weight_sum_kernel<<<(2 * a.d + 31) / 32, 256, 0, stream>>>(static_cast<const float*>(a.workspace), grid, a.d,
                                                             a.dw_post, a.dw_pre);
  return cudaGetLastError();
}

// Calls f with the types and the shape as compile-time constants.
template <class F> cudaError_t dispatch(rsm_dtype y_dtype, rsm_dtype dtype, const Shape& s, F f) {
  auto shaped = [&](auto ty, auto t) {
    if (s.vec == 8) {
      if (s.iter == 1) return f(ty, t, std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
      return f(ty, t, std::integral_constant<int, 8>(), std::integral_constant<int, 2>());
    }
    if (s.iter == 1) return f(ty, t, std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
    if (s.iter == 2) return f(ty, t, std::integral_constant<int, 4>(), std::integral_constant<int, 2>());
    return f(ty, t, std::integral_constant<int, 4>(), std::integral_constant<int, 4>());
  };
  if (dtype == RSM_F32) return shaped(float(), float());
  if (y_dtype == RSM_F32) return shaped(float(), __nv_bfloat16());
  return shaped(__nv_bfloat16(), __nv_bfloat16());
}

}  // namespace

cudaError_t launch_block_norm(const rsm_block_norm_args& a, cudaStream_t stream) {
  const Shape s = shape_for(a.d);
  return dispatch(a.y_dtype, a.dtype, s, [&](auto ty, auto t, auto vec, auto iter) {
    return forward_as<decltype(ty), decltype(t), decltype(vec)::value, decltype(iter)::value>(a, s, stream);
  });
}

size_t block_norm_backward_workspace_bytes(const rsm_block_norm_backward_args& a) {
  return (size_t)backward_blocks(a.rows, shape_for(a.d)) * 2 * a.d * sizeof(float);
}

cudaError_t launch_block_norm_backward(const rsm_block_norm_backward_args& a, cudaStream_t stream) {
  const Shape s = shape_for(a.d);
  return dispatch(a.y_dtype, a.dtype, s, [&](auto ty, auto t, auto vec, auto iter) {
    return backward_as<decltype(ty), decltype(t), decltype(vec)::value, decltype(iter)::value>(a, s, stream);
  });
}

}  // namespace rsm
