// attn_simt.cu -- window and paged attention on CUDA cores, in fp32 (any head dimension, page size
// and dtype), with its gradients; and the small kernels every attention path shares (delta, the
// join of split rows, the cache write, the input check).
//
// Forward, one block per 64 packed query rows (token, head of the group): the keys pass by in tiles
// of BB; a running maximum m and sum l per row keep the softmax in one pass,
//   m' = max(m, max_j s_j),  l' = l e^{m-m'} + sum_j e^{s_j-m'},  acc' = acc e^{m-m'} + sum_j e^{s_j-m'} v_j
// Backward without atomics, so that its sums have one order: one kernel owns 64 keys and walks the
// query rows that see them (dk, dv), another owns 64 query rows and walks their keys (dq); both form
// p = e^{s - lse} and ds = p (dO.v - delta) again, 7 tile products against the 5 of a shared walk.
//
// All products have the same two shapes, 64 stationary rows (16 x 16 threads, 4 rows each) against
// BB streamed ones: W = A B^T over the head dimension and acc += W B. Both read 16-byte pieces of
// shared memory, the rows padded by 16 bytes so that 8 neighbouring rows use different banks. What bounds
// them is shared memory, which hands out 32 words a cycle: a thread's 4 x 4 (4 x 2) products use a word
// twice (1.3 times) and the FMA pipe could take 4. A score is four interleaved sums, two per packed FMA: as one
// sum of D terms it is off by twice as much, and o, dq and dk with it (2 x 777 tokens: 5.8e-7 of the gradients'
// norm, now 3.9e-7; the same time). Neither 8 rows per thread and half the threads nor warp-level
// tf32 products of split operands were faster at the sizes fp32 runs at, where blocks are few and latency
// counts (forward and gradients of 2 x 777 tokens, 4 heads of 64: 234 and 201 us a call against 175).
#include <algorithm>

#include "attention.cuh"

namespace rsm {

namespace {

using namespace attn;

constexpr int kBA = 64;        // stationary rows
constexpr int kThreads = 256;  // 16 x 16

template <int DP> struct Tile {
  // streamed rows per step: 64 where two blocks per SM still fit their tiles, 32 otherwise
  static constexpr int kBB = DP <= 64 ? 64 : 32;
};

template <typename T> struct Out;
template <> struct Out<float> {
  static RSM_DEV void st4(float* p, float a, float b, float c, float d) {
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
  }
};
template <> struct Out<__nv_bfloat16> {
  static RSM_DEV void st4(__nv_bfloat16* p, float a, float b, float c, float d) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
  }
};

// Row r of a tile of N rows comes from base + offset(r) (fp32 in shared memory), or is zero where
// offset(r) < 0. 16 threads share a row, so a row's offset (divisions by the group or page size) is found
// once per 16 bytes x D / 64 and thread. Columns past D are left alone: no product reads them into a
// column that is stored. With `used`, it gets whether each row is there.
RSM_DEV float4 read4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
RSM_DEV float4 read4(const __nv_bfloat16* p) {
  const uint2 t = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(t.x << 16), __uint_as_float(t.x & 0xffff0000u), __uint_as_float(t.y << 16),
                     __uint_as_float(t.y & 0xffff0000u));
}
template <typename T, int DP, int N, class Off>
RSM_DEV void load_rows(float* dst, const void* base, int D, int tx, int ty, Off offset, int* used = nullptr) {
  float4 x[N / 16][DP / 64];  // (all loads before the first store: one trip to memory, not one per row)
#pragma unroll
  for (int k = 0; k < N / 16; ++k) {
    const int r = ty + 16 * k;
    const int64_t off = offset(r);
    if (used && tx == 0) used[r] = off >= 0;
#pragma unroll
    for (int jj = 0; jj < DP / 64; ++jj) {
      const int c = 4 * tx + 64 * jj;
      x[k][jj] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (off >= 0 && c < D) x[k][jj] = read4(static_cast<const T*>(base) + off + c);
    }
  }
#pragma unroll
  for (int k = 0; k < N / 16; ++k)
#pragma unroll
    for (int jj = 0; jj < DP / 64; ++jj)
      if (4 * tx + 64 * jj < D)
        *reinterpret_cast<float4*>(dst + (ty + 16 * k) * (DP + 4) + 4 * tx + 64 * jj) = x[k][jj];
}

// c[i][j] = sum_d A[ty + 16 i][d] B[tx + 16 j][d]
template <int DP, int BB>
RSM_DEV void product_nt(const float* A, const float* B, int D, int tx, int ty, float (&c)[4][BB / 16]) {
  float2 s[4][BB / 16][2];  // four sums per score, joined at the end: one sum of D terms is off by twice as much
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < BB / 16; ++j) s[i][j][0] = s[i][j][1] = both(0.f);
#pragma unroll 2
  for (int d = 0; d < D; d += 4) {
    float4 a[4], b[BB / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * (DP + 4) + d);
#pragma unroll
    for (int j = 0; j < BB / 16; ++j) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * (DP + 4) + d);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < BB / 16; ++j) {
        s[i][j][0] = fma2(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), s[i][j][0]);
        s[i][j][1] = fma2(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), s[i][j][1]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < BB / 16; ++j) c[i][j] = (s[i][j][0].x + s[i][j][0].y) + (s[i][j][1].x + s[i][j][1].y);
}

// acc[i][jj] += sum_k W[ty + 16 i][k] B[k][4 tx + 64 jj ..]
template <int DP, int BB>
RSM_DEV void product_nn(const float* W, const float* B, int tx, int ty, float4 (&acc)[4][DP / 64]) {
#pragma unroll 2
  for (int k = 0; k < BB; k += 4) {
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(W + (ty + 16 * i) * (BB + 4) + k);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
      for (int jj = 0; jj < DP / 64; ++jj) {
        const float4 b = *reinterpret_cast<const float4*>(B + (k + u) * (DP + 4) + 4 * tx + 64 * jj);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = u == 0 ? w[i].x : u == 1 ? w[i].y : u == 2 ? w[i].z : w[i].w;
          const float2 lo = fma2(both(x), make_float2(b.x, b.y), make_float2(acc[i][jj].x, acc[i][jj].y));
          const float2 hi = fma2(both(x), make_float2(b.z, b.w), make_float2(acc[i][jj].z, acc[i][jj].w));
          acc[i][jj] = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
      }
    }
  }
}

RSM_DEV float half_warp_max(float v) {
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
  return v;
}
RSM_DEV float half_warp_sum(float v) {
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

constexpr float kNegInf = -__builtin_inff();

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) attn_simt_kernel(const AttnParams p, int ntiles) {
  constexpr int BB = Tile<DP>::kBB;
  extern __shared__ float sm[];
  __shared__ int used[BB];  // keys of the tile that are there
  float* sQ = sm;
  float* sK = sQ + kBA * (DP + 4);
  float* sV = sK + BB * (DP + 4);
  float* sP = sV + BB * (DP + 4);
  const int split = blockIdx.x % p.splits;
  const int item = blockIdx.x / p.splits;
  const int tile = item % ntiles, pair = item / ntiles;
  const int hk = pair % p.Hkv, b = pair / p.Hkv;
  const Seq s = sequence(p, b);
  if (s.kv != s.pos0 + s.nq && threadIdx.x == 0 && p.table) raise_status(RSM_ERR_BAD_PAGE);
  const int nq = p.table ? min(s.nq, p.max_q) : s.nq;
  const int r0 = tile * kBA;
  const int rows = (int)min((int64_t)nq * p.G - r0, (int64_t)kBA);
  if (rows <= 0) return;
  const int G = p.G, D = p.D;
  auto q_index = [&](int r) { return (s.row0 + (r0 + r) / G) * p.H + hk * G + (r0 + r) % G; };
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  load_rows<T, DP, kBA>(sQ, p.q, D, tx, ty, [&](int r) { return r < rows ? q_index(r) * D : (int64_t)-1; });
  int pos[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) pos[i] = s.pos0 + (r0 + ty + 16 * i) / G;
  const Walk walk = key_walk(s.pos0 + r0 / G, s.pos0 + (r0 + rows - 1) / G, s.kv, p.window, p.sinks, BB);
  const int w0 = (int)((int64_t)walk.n * split / p.splits), w1 = (int)((int64_t)walk.n * (split + 1) / p.splits);

  const Seen seen = keys_seen(s.pos0, s.pos0 + nq - 1, s.kv, p.window, p.sinks);
  const float scale2 = p.scale * kLog2e;
  float m[4], l[4];
  float4 acc[4][DP / 64];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = kNegInf;
    l[i] = 0.f;
#pragma unroll
    for (int jj = 0; jj < DP / 64; ++jj) acc[i][jj] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int w = w0; w < w1; ++w) {
    const int k0 = walk.tile(w) * BB;
    __syncthreads();
    // rows that nothing sees are zero, so that a weight of zero meets no stale NaN
    auto off = [&](int r) { return seen.has(k0 + r) ? kv_offset(p, b, hk, k0 + r) : (int64_t)-1; };
    load_rows<T, DP, BB>(sK, p.k, D, tx, ty, off, used);
    load_rows<T, DP, BB>(sV, p.v, D, tx, ty, off);
    __syncthreads();
    float c[4][BB / 16];
    product_nt<DP, BB>(sQ, sK, D, tx, ty, c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = kNegInf;
#pragma unroll
      for (int j = 0; j < BB / 16; ++j) {
        const int key = k0 + tx + 16 * j;
        if (!used[tx + 16 * j] || !sees(pos[i], key, p.window, p.sinks)) c[i][j] = kNegInf;
        top = fmaxf(top, c[i][j]);
      }
      const float mn = fmaxf(m[i], half_warp_max(top));
      const float ref = mn == kNegInf ? 0.f : mn;  // nothing seen yet: every weight below is e^-inf = 0
      const float corr = exp2f((m[i] - ref) * scale2);  // (m is in the products' units: a difference rounds less)
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < BB / 16; ++j) {
        const float x = exp2f((c[i][j] - ref) * scale2);
        sum += x;
        sP[(ty + 16 * i) * (BB + 4) + tx + 16 * j] = x;
      }
      l[i] = l[i] * corr + half_warp_sum(sum);
#pragma unroll
      for (int jj = 0; jj < DP / 64; ++jj) {
        acc[i][jj].x *= corr; acc[i][jj].y *= corr; acc[i][jj].z *= corr; acc[i][jj].w *= corr;
      }
    }
    __syncwarp();  // a row of P is written and read by the same half warp
    product_nn<DP, BB>(sP, sV, tx, ty, acc);
  }
  const int64_t total = (int64_t)p.T * (p.table ? 1 : p.B) * p.H;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 16 * i;
    if (r >= rows) continue;
    const int64_t at = q_index(r);
    const float inv = l[i] > 0.f ? 1.f / l[i] : l[i] == 0.f ? 0.f : l[i];  // (a NaN stays one)
    const float lse = l[i] == 0.f ? kNegInf : fmaf(m[i], p.scale, logf(l[i]));
#pragma unroll
    for (int jj = 0; jj < DP / 64; ++jj) {
      const int d = 4 * tx + 64 * jj;
      if (d >= D) continue;
      const float4 a = acc[i][jj];
      if (p.splits > 1)
        Out<float>::st4(p.part_o + (split * total + at) * D + d, a.x * inv, a.y * inv, a.z * inv, a.w * inv);
      else
        Out<T>::st4(static_cast<T*>(p.o) + at * D + d, a.x * inv, a.y * inv, a.z * inv, a.w * inv);
      if (sizeof(T) == 2 && p.o_low) {
        auto low = [&](float x) { return x - __bfloat162float(__float2bfloat16_rn(x)); };
        Out<T>::st4(static_cast<T*>(p.o_low) + at * D + d, low(a.x * inv), low(a.y * inv), low(a.z * inv), low(a.w * inv));
      }
    }
    if (tx == 0) {
      if (p.splits > 1) p.part_lse[split * total + at] = lse;
      else if (p.lse) p.lse[at] = lse;
    }
  }
}

// How the walks of the first key tiles, whose keys every later row sees, are cut: `parts` blocks per tile,
// each with its share of the query rows, leave fp32 sums that a small kernel adds in order. Uncut, the
// longest walk is what the kernel ends with (777 tokens, window 128, groups of 2: 413 us of 495).
struct Cut {
  int tiles;    // key tiles that are cut
  int parts;
  float* part;  // [pairs][tiles][parts][64][2][D]
};

// Gradients. DQ: the stationary rows are query rows (A1 = q, A2 = dO), the streamed ones keys
// (B1 = k, B2 = v) and acc2 = dq. Otherwise the stationary rows are keys (k, v), the streamed ones
// query rows (q, dO), acc1 = dv and acc2 = dk.
template <typename T, int DP, bool DQ>
__global__ void __launch_bounds__(kThreads) attn_simt_backward_kernel(const AttnParams p, int ntiles, Cut cut) {
  constexpr int BB = 32;
  extern __shared__ float sm[];
  float* sA1 = sm;
  float* sA2 = sA1 + kBA * (DP + 4);
  float* sB1 = sA2 + kBA * (DP + 4);
  float* sB2 = sB1 + BB * (DP + 4);
  float* sW2 = sB2 + BB * (DP + 4);
  float* sW1 = sW2 + kBA * (BB + 4);              // DQ: not used
  float* sStat = DQ ? sW1 : sW1 + kBA * (BB + 4);  // lse and delta of the query rows
  int tile, pair, part = 0;
  if (DQ) {
    tile = blockIdx.x % ntiles;
    pair = blockIdx.x / ntiles;
  } else {
    // the cut tiles' parts come first
    const int items = ntiles + cut.tiles * (cut.parts - 1);
    const int item = blockIdx.x % items;
    pair = blockIdx.x / items;
    const bool is_cut = item < cut.tiles * cut.parts;
    tile = is_cut ? item / cut.parts : item - cut.tiles * (cut.parts - 1);
    part = is_cut ? item % cut.parts : 0;
  }
  const bool to_part = !DQ && tile < cut.tiles;
  const int hk = pair % p.Hkv, b = pair / p.Hkv;
  const int G = p.G, D = p.D, T_ = p.T;
  const int nrows = T_ * G;  // packed query rows of this pair
  const int a0 = tile * kBA;
  auto q_index = [&](int r) { return ((int64_t)b * T_ + r / G) * p.H + hk * G + r % G; };
  auto q_off = [&](int r) { return r < nrows ? q_index(r) * D : (int64_t)-1; };
  auto k_off = [&](int key) { return key < T_ ? kv_offset(p, b, hk, key) : (int64_t)-1; };
  auto load_stats = [&](int r0, int n) {
    for (int r = threadIdx.x; r < n; r += kThreads) {
      const bool in = r0 + r < nrows;
      sStat[2 * r] = in ? p.lse[q_index(r0 + r)] : 0.f;
      sStat[2 * r + 1] = in ? p.delta[q_index(r0 + r)] : 0.f;
    }
  };
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  Walk walk{0, 0, 0};
  int w0 = 0, w1;
  if (DQ) {
    load_rows<T, DP, kBA>(sA1, p.q, D, tx, ty, [&](int r) { return q_off(a0 + r); });
    load_rows<T, DP, kBA>(sA2, p.dO, D, tx, ty, [&](int r) { return q_off(a0 + r); });
    load_stats(a0, kBA);
    walk = key_walk(a0 / G, (min(nrows, a0 + kBA) - 1) / G, T_, p.window, p.sinks, BB);
    w1 = walk.n;
  } else {
    load_rows<T, DP, kBA>(sA1, p.k, D, tx, ty, [&](int r) { return k_off(a0 + r); });
    load_rows<T, DP, kBA>(sA2, p.v, D, tx, ty, [&](int r) { return k_off(a0 + r); });
    int t0, t1;
    query_range(a0, min(a0 + kBA, T_) - 1, T_, p.window, p.sinks, t0, t1);
    walk.first = t0 * G / BB;
    walk.n = (t1 * G - 1) / BB + 1 - walk.first;
    w1 = walk.n;
    if (to_part) {
      w0 = (int)((int64_t)walk.n * part / cut.parts);
      w1 = (int)((int64_t)walk.n * (part + 1) / cut.parts);
    }
  }
  int pos[4];  // DQ: the rows' places
#pragma unroll
  for (int i = 0; i < 4; ++i) pos[i] = (a0 + ty + 16 * i) / G;
  float4 acc1[DQ ? 1 : 4][DP / 64], acc2[4][DP / 64];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int jj = 0; jj < DP / 64; ++jj) {
      if (!DQ) acc1[DQ ? 0 : i][jj] = make_float4(0.f, 0.f, 0.f, 0.f);
      acc2[i][jj] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  for (int w = w0; w < w1; ++w) {
    const int b0 = walk.tile(w) * BB;
    __syncthreads();
    if (DQ) {
      load_rows<T, DP, BB>(sB1, p.k, D, tx, ty, [&](int r) { return k_off(b0 + r); });
      load_rows<T, DP, BB>(sB2, p.v, D, tx, ty, [&](int r) { return k_off(b0 + r); });
    } else {
      load_rows<T, DP, BB>(sB1, p.q, D, tx, ty, [&](int r) { return q_off(b0 + r); });
      load_rows<T, DP, BB>(sB2, p.dO, D, tx, ty, [&](int r) { return q_off(b0 + r); });
      load_stats(b0, BB);
    }
    __syncthreads();
    float c1[4][BB / 16], c2[4][BB / 16];
    product_nt<DP, BB>(sA1, sB1, D, tx, ty, c1);
    product_nt<DP, BB>(sA2, sB2, D, tx, ty, c2);
#pragma unroll
    for (int j = 0; j < BB / 16; ++j) {
      const int rb = tx + 16 * j;
      const int there = DQ ? b0 + rb < T_ : b0 + rb < nrows;
      const int pos_b = DQ ? 0 : (b0 + rb) / G;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ra = ty + 16 * i;
        const bool in_a = DQ ? a0 + ra < nrows : a0 + ra < T_;
        const float* st = sStat + 2 * (DQ ? ra : rb);
        const bool seen = there && in_a && (DQ ? sees(pos[i], b0 + rb, p.window, p.sinks) : sees(pos_b, a0 + ra, p.window, p.sinks));
        const float pr = seen ? exp2f(fmaf(c1[i][j], p.scale, -st[0]) * kLog2e) : 0.f;
        const float ds = seen ? pr * (c2[i][j] - st[1]) : 0.f;
        sW2[ra * (BB + 4) + rb] = ds;
        if (!DQ) sW1[ra * (BB + 4) + rb] = pr;
      }
    }
    __syncwarp();  // a row of the weights is written and read by the same half warp
    product_nn<DP, BB>(sW2, sB1, tx, ty, acc2);
    if constexpr (!DQ) product_nn<DP, BB>(sW1, sB2, tx, ty, acc1);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = a0 + ty + 16 * i;
    const int64_t off = DQ ? q_off(r) : k_off(r);
    if (off < 0) continue;
    float* sums = to_part ? cut.part + ((((int64_t)pair * cut.tiles + tile) * cut.parts + part) * kBA + ty + 16 * i) * 2 * D : nullptr;
#pragma unroll
    for (int jj = 0; jj < DP / 64; ++jj) {
      const int d = 4 * tx + 64 * jj;
      if (d >= D) continue;
      const float4 a = acc2[i][jj];
      const float4 k4 = make_float4(a.x * p.scale, a.y * p.scale, a.z * p.scale, a.w * p.scale);
      const float4 v4 = DQ ? a : acc1[DQ ? 0 : i][jj];
      if (to_part) {
        *reinterpret_cast<float4*>(sums + d) = v4;
        *reinterpret_cast<float4*>(sums + D + d) = k4;
        continue;
      }
      T* g = static_cast<T*>(DQ ? p.dq : p.dk);
      if (g) Out<T>::st4(g + off + d, k4.x, k4.y, k4.z, k4.w);
      if (!DQ && p.dv) Out<T>::st4(static_cast<T*>(p.dv) + off + d, v4.x, v4.y, v4.z, v4.w);
    }
  }
}

// Adds the parts of the cut tiles up, in order, 16 bytes of dv or dk per thread.
template <typename T> __global__ void __launch_bounds__(256) cut_sum_kernel(const AttnParams p, Cut cut) {
  const int per = p.D / 2;  // pieces of 4 of a row's dv and dk
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int d = (int)(e % per) * 4;
  const int64_t row = e / per;
  const int r = (int)(row % kBA), tile = (int)(row / kBA % cut.tiles);
  const int64_t pair = row / kBA / cut.tiles;
  const int key = tile * kBA + r;
  if (pair >= (int64_t)p.B * p.Hkv || key >= p.T) return;
  const float* part = cut.part + ((pair * cut.tiles + tile) * cut.parts * kBA + r) * 2 * p.D + d;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = 0; c < cut.parts; ++c) {
    const float4 x = *reinterpret_cast<const float4*>(part + (int64_t)c * kBA * 2 * p.D);
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  }
  T* out = static_cast<T*>(d < p.D ? p.dv : p.dk);
  const int64_t at = (pair / p.Hkv * p.T + key) * p.Hkv + pair % p.Hkv;
  if (out) Out<T>::st4(out + at * p.D + (d < p.D ? d : d - p.D), s.x, s.y, s.z, s.w);
}

// delta = dO . o, a warp per row.
template <typename T>
__global__ void __launch_bounds__(256) delta_kernel(const T* dO, const T* o, const T* o_low, float* delta, int64_t rows, int D) {
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int lane = threadIdx.x & 31;
  float sum = 0.f;
  for (int d = lane * 4; d < D; d += 128) {
    float a[4], x[4];
    In<T>::ld4(dO + row * D + d, a);
    In<T>::ld4(o + row * D + d, x);
    if (o_low) {
      float low[4];
      In<T>::ld4(o_low + row * D + d, low);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] += low[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = fmaf(a[i], x[i], sum);
  }
  sum = warp_sum_f(sum);
  if (lane == 0) delta[row] = sum;
}

// o = sum_s e^{lse_s - lse} o_s over the splits, a warp per row. Rows that no block computed (behind
// the last sequence, or past max_q) are left alone.
template <typename T>
__global__ void __launch_bounds__(256) combine_kernel(const AttnParams p) {
  const int64_t total = (int64_t)p.T * p.H;
  const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (at >= total) return;
  const int lane = threadIdx.x & 31;
  const int tok = (int)(at / p.H);
  // the token's sequence: the last b with cu_q[b] <= tok
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu_q[mid] <= tok) lo = mid; else hi = mid;
  }
  const Seq s = sequence(p, lo);
  if (tok < s.row0 || tok >= s.row0 + min(s.nq, p.max_q)) return;
  float top = kNegInf;
  for (int i = lane; i < p.splits; i += 32) top = fmaxf(top, p.part_lse[i * total + at]);
  top = warp_max_f(top);
  const float ref = top == kNegInf ? 0.f : top;
  float sum = 0.f;
  for (int i = lane; i < p.splits; i += 32) sum += expf(p.part_lse[i * total + at] - ref);
  sum = warp_sum_f(sum);
  const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
  for (int d = lane * 4; d < p.D; d += 128) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < p.splits; ++i) {
      const float w = expf(p.part_lse[i * total + at] - ref) * inv;
      if (w == 0.f) continue;
      const float4 x = *reinterpret_cast<const float4*>(p.part_o + (i * total + at) * p.D + d);
      a.x = fmaf(w, x.x, a.x); a.y = fmaf(w, x.y, a.y); a.z = fmaf(w, x.z, a.z); a.w = fmaf(w, x.w, a.w);
    }
    Out<T>::st4(static_cast<T*>(p.o) + at * p.D + d, a.x, a.y, a.z, a.w);
  }
  if (lane == 0 && p.lse) p.lse[at] = sum == 0.f ? kNegInf : ref + logf(sum);
}

// Writes the new tokens' rows of Hkv*D elements to their places, 16 bytes per thread and step; a row
// is contiguous on both sides. Bound by the copy itself (2 reads and 2 writes of the rows).
__global__ void __launch_bounds__(256) append_kernel(const rsm_paged_append_args a, int chunks) {
  const int64_t n = (int64_t)a.N * chunks;
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (int64_t)gridDim.x * blockDim.x) {
    const int tok = (int)(e / chunks);
    const int c = (int)(e - (int64_t)tok * chunks);
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu_q[mid] <= tok) lo = mid; else hi = mid;
    }
    const int c0 = max(a.cu_q[lo], 0), c1 = min(a.cu_q[lo + 1], a.N);
    if (tok < c0 || tok >= c1) continue;
    const int64_t pos = (int64_t)max(a.kv_len[lo], 0) - (c1 - tok);
    if (pos < 0) continue;
    const int64_t slot = pos / a.page_size;
    const int pg = slot < a.table_width ? a.page_table[(int64_t)lo * a.table_width + slot] : -1;
    if ((unsigned)pg >= (unsigned)a.num_pages) {
      raise_status(RSM_ERR_BAD_PAGE);
      continue;
    }
    const int64_t to = ((int64_t)pg * a.page_size + pos % a.page_size) * chunks + c;
    static_cast<uint4*>(a.k_cache)[to] = static_cast<const uint4*>(a.k)[e];
    static_cast<uint4*>(a.v_cache)[to] = static_cast<const uint4*>(a.v)[e];
  }
}

template <typename T>
__global__ void __launch_bounds__(256) check_finite_kernel(const T* x, int64_t n) {
  bool bad = false;
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (int64_t)gridDim.x * blockDim.x)
    bad |= !finite_f32(In<T>::ld(x + e));
  if (bad) raise_status(RSM_ERR_NONFINITE);
}

int64_t all_rows(const AttnParams& p) { return (int64_t)p.T * (p.table ? 1 : p.B) * p.H; }

int64_t row_tiles(const AttnParams& p) {
  const int64_t nq = p.table ? p.max_q : p.T;
  return (nq * p.G + kBA - 1) / kBA;
}

template <typename T, int DP>
cudaError_t forward_dp(const AttnParams& p, cudaStream_t stream) {
  constexpr int BB = Tile<DP>::kBB;
  constexpr int bytes = ((kBA + 2 * BB) * (DP + 4) + kBA * (BB + 4)) * 4;
  cudaError_t e = set_smem_limit<attn_simt_kernel<T, DP>>(bytes);
  if (e != cudaSuccess) return e;
  const int64_t nt = row_tiles(p);
  const int64_t grid = nt * p.Hkv * p.B * p.splits;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  attn_simt_kernel<T, DP><<<(unsigned)grid, kThreads, bytes, stream>>>(p, (int)nt);
  return cudaGetLastError();
}

// The tiles that hold sinks are cut where the walk past the window is longer than the window (unless there
// are so many that the walks are all alike). All tiles are, where whole ones would leave SMs idle.
Cut cut_for(const AttnParams& p) {
  Cut c{0, 1, nullptr};
  const int ntiles = (p.T + kBA - 1) / kBA;
  const int tiles = (std::min(p.sinks, p.T) + kBA - 1) / kBA;
  const int64_t near = std::min<int64_t>(p.T, (int64_t)kBA + p.window);
  if (tiles > 0 && tiles <= 4 && p.T >= 2 * near) {
    c.tiles = std::min(tiles, ntiles);
    c.parts = (int)std::min<int64_t>(64, p.T / near);
  }
  const int64_t blocks = std::max<int64_t>(1, (int64_t)ntiles * p.Hkv * p.B);
  const int64_t steps = near * p.G / 32;  // of a whole tile
  const int parts = (int)std::min<int64_t>({device_sm_count() / blocks, steps / 2, 8});
  if (parts > 1) {
    c.tiles = ntiles;
    c.parts = std::max(std::min(c.parts, 8), parts);
  }
  return c;
}

size_t cut_bytes(const AttnParams& p, const Cut& c) {
  return c.tiles ? (size_t)p.B * p.Hkv * c.tiles * c.parts * kBA * 2 * p.D * sizeof(float) : 0;
}

template <typename T, int DP>
cudaError_t backward_dp(const AttnParams& p, float* part, cudaStream_t stream) {
  constexpr int BB = 32;
  constexpr int bytes = ((2 * kBA + 2 * BB) * (DP + 4) + 2 * kBA * (BB + 4) + 2 * kBA) * 4;
  static_assert(bytes <= 232448, "shared memory budget");
  Cut cut = cut_for(p);
  cut.part = part;
  if (p.dk || p.dv) {
    cudaError_t e = set_smem_limit<attn_simt_backward_kernel<T, DP, false>>(bytes);
    if (e != cudaSuccess) return e;
    const int nt = (p.T + kBA - 1) / kBA;
    const int64_t pairs = (int64_t)p.Hkv * p.B;
    const int64_t grid = (nt + (int64_t)cut.tiles * (cut.parts - 1)) * pairs;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    attn_simt_backward_kernel<T, DP, false><<<(unsigned)grid, kThreads, bytes, stream>>>(p, nt, cut);
    e = cudaGetLastError();
    if (e == cudaSuccess && cut.tiles) {
      const int64_t n = pairs * cut.tiles * kBA * (p.D / 2);
      cut_sum_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(p, cut);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
  }
  if (p.dq) {
    cudaError_t e = set_smem_limit<attn_simt_backward_kernel<T, DP, true>>(bytes);
    if (e != cudaSuccess) return e;
    const int64_t nt = row_tiles(p);
    const int64_t grid = nt * p.Hkv * p.B;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    attn_simt_backward_kernel<T, DP, true><<<(unsigned)grid, kThreads, bytes, stream>>>(p, (int)nt, cut);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_attn_simt(const AttnParams& p, rsm_dtype dtype, cudaStream_t stream) {
  if (dtype == RSM_F32)
    return p.D <= 64 ? forward_dp<float, 64>(p, stream)
                     : p.D <= 128 ? forward_dp<float, 128>(p, stream) : forward_dp<float, 256>(p, stream);
  return p.D <= 64 ? forward_dp<__nv_bfloat16, 64>(p, stream)
                   : p.D <= 128 ? forward_dp<__nv_bfloat16, 128>(p, stream) : forward_dp<__nv_bfloat16, 256>(p, stream);
}

size_t attn_simt_backward_bytes(const AttnParams& p) { return cut_bytes(p, cut_for(p)); }

cudaError_t launch_attn_simt_backward(const AttnParams& p, rsm_dtype dtype, float* part, cudaStream_t stream) {
  if (dtype == RSM_F32)
    return p.D <= 64 ? backward_dp<float, 64>(p, part, stream)
                     : p.D <= 128 ? backward_dp<float, 128>(p, part, stream) : backward_dp<float, 256>(p, part, stream);
  return p.D <= 64 ? backward_dp<__nv_bfloat16, 64>(p, part, stream)
                   : p.D <= 128 ? backward_dp<__nv_bfloat16, 128>(p, part, stream)
                                : backward_dp<__nv_bfloat16, 256>(p, part, stream);
}

cudaError_t launch_attn_delta(const AttnParams& p, rsm_dtype dtype, cudaStream_t stream) {
  const int64_t rows = all_rows(p);
  const unsigned grid = (unsigned)((rows + 7) / 8);
  if (dtype == RSM_F32)
    delta_kernel<float><<<grid, 256, 0, stream>>>(static_cast<const float*>(p.dO), static_cast<const float*>(p.o), nullptr,
                                                  p.delta, rows, p.D);
  else
    delta_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(static_cast<const __nv_bfloat16*>(p.dO),
                                                          static_cast<const __nv_bfloat16*>(p.o),
                                                          static_cast<const __nv_bfloat16*>(p.o_low), p.delta, rows, p.D);
  return cudaGetLastError();
}

cudaError_t launch_attn_combine(const AttnParams& p, rsm_dtype dtype, cudaStream_t stream) {
  const unsigned grid = (unsigned)((all_rows(p) + 7) / 8);
  if (dtype == RSM_F32) combine_kernel<float><<<grid, 256, 0, stream>>>(p);
  else combine_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

// Blocks that share the keys of a row: enough for two blocks per SM where there are few rows, and
// never under 4 key tiles each. The cache's length is known on the device alone; the table's width
// bounds it, and each block takes its share of the real length.
int attn_simt_splits(const AttnParams& p) {
  if (!p.table) return 1;
  const int64_t blocks = std::max<int64_t>(1, row_tiles(p) * p.Hkv * p.B);
  int64_t keys = (int64_t)p.table_width * p.page;
  if (p.window > 0) keys = std::min<int64_t>(keys, (int64_t)p.window + p.sinks + p.max_q);
  const int64_t tiles = (keys + 31) / 32;
  const int64_t want = (2 * device_sm_count() + blocks - 1) / blocks;
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, tiles / 4, 64}));
}

cudaError_t launch_paged_append(const rsm_paged_append_args& a, cudaStream_t stream) {
  const int chunks = (int)((int64_t)a.Hkv * a.D * (a.dtype == RSM_F32 ? 4 : 2) / 16);
  const int64_t n = (int64_t)a.N * chunks;
  const int64_t grid = std::min<int64_t>((n + 255) / 256, 8 * (int64_t)device_sm_count());
  append_kernel<<<(unsigned)grid, 256, 0, stream>>>(a, chunks);
  return cudaGetLastError();
}

cudaError_t launch_check_finite(const void* x, int64_t n, rsm_dtype dtype, cudaStream_t stream) {
  const unsigned grid = (unsigned)std::min<int64_t>((n + 255) / 256, 8 * (int64_t)device_sm_count());
  if (dtype == RSM_F32) check_finite_kernel<float><<<grid, 256, 0, stream>>>(static_cast<const float*>(x), n);
  else check_finite_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(static_cast<const __nv_bfloat16*>(x), n);
  return cudaGetLastError();
}

}  // namespace rsm
