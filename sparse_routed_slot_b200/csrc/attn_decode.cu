// attn_decode.cu -- paged attention of single tokens (and other calls with at most 16 query rows per
// key/value head and sequence), bf16.
//
// Such a call reads every key and value once and computes little: it is bound by that read. K and V go
// straight from memory to registers, 16 bytes per lane, in the layout that the warp-level tensor products
// (m16n8k16) want, so there is no shared memory, no barrier and nothing to wait for but the data. With Q's
// rows as the narrow side of the products no row of them is wasted on up to 8 query rows:
//   S^T = K Q^T   16 keys x 8 rows. A product sums over columns in any order, so lane 4 g + t takes the
//                 contiguous columns 8 t .. 8 t + 7 of a block of 32 for keys g and g + 8
//   O^T += V^T P^T  16 columns x 8 rows over 16 keys. The lane has columns 8 g .. 8 g + 7 of keys 2 t, 2 t + 1,
//                 2 t + 8, 2 t + 9; byte permutes make the pairs of keys that the product takes, and column
//                 8 g + 2 j (+ 1) stands in row g (g + 8) of product j
//   P^T from S^T's accumulators by an 8 x 8 transpose across the lanes.
// The weights are rounded to bf16 for the product; scores, statistics and sums are fp32. As in the tile
// kernel, the reference of a row's exponentials moves only past 2^32.
//
// Each warp walks its own tiles of 16 keys (every eighth of the block's) and the block's warps join at the
// end in shared memory, blocks that share a sequence's keys in a second kernel. 16 warps per SM keep
// 16 x 8 KB on their way (head dimension 128); the copy's rate needs about 45 KB.
#include <algorithm>

#include "attention.cuh"

namespace rsm {

namespace {

using namespace attn;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kKeys = 16;
constexpr float kNegInf = -__builtin_inff();
constexpr float kSlack = 32.f;

RSM_DEV void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
RSM_DEV uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
RSM_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
RSM_DEV uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}
// Over the eight lanes with the same t.
RSM_DEV float over_keys_max(float v) {
#pragma unroll
  for (int d = 4; d <= 16; d <<= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
  return v;
}
RSM_DEV float over_keys_sum(float v) {
#pragma unroll
  for (int d = 4; d <= 16; d <<= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

// NQ: groups of 8 query rows. A row is (token, head of the group), as everywhere.
template <int DP, int NQ>
__global__ void __launch_bounds__(kThreads, DP <= 128 && NQ == 1 ? 2 : 1) attn_decode_kernel(const AttnParams p) {
  constexpr int kR = 8 * NQ;
  constexpr int kC = DP / 32, kB = DP / 64;  // blocks of columns of the two products
  extern __shared__ float sm[];              // [warps][kR][DP]
  __shared__ float s_m[kWarps][kR], s_l[kWarps][kR];
  const int split = blockIdx.x % p.splits;
  const int pair = blockIdx.x / p.splits;
  const int hk = pair % p.Hkv, b = pair / p.Hkv;
  const Seq s = sequence(p, b);
  if (s.kv != s.pos0 + s.nq && threadIdx.x == 0) raise_status(RSM_ERR_BAD_PAGE);
  const int G = p.G, D = p.D;
  const int nq = min(s.nq, p.max_q);
  const int rows = nq * G;
  if (rows <= 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  auto q_index = [&](int r) { return (s.row0 + r / G) * p.H + hk * G + r % G; };

  // Q as the products take it: row g of each group, columns 32 c + 8 t .. + 7
  uint4 q[NQ][kC];
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int r = 8 * n + g, d = 32 * c + 8 * t;
      q[n][c] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows && d < D)
        q[n][c] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + q_index(r) * D + d));
    }

  const Walk walk = key_walk(s.pos0, s.pos0 + nq - 1, s.kv, p.window, p.sinks, kKeys);
  const int w0 = (int)((int64_t)walk.n * split / p.splits), w1 = (int)((int64_t)walk.n * (split + 1) / p.splits);
  const float scale2 = p.scale * kLog2e;
  const int64_t row_step = (int64_t)p.Hkv * D;
  const bool one_page = p.page % kKeys == 0;  // a tile of keys stands in one page
  float m[NQ][2], l[NQ][2], o[NQ][kB * 4][4];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n][0] = m[n][1] = kNegInf;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int j = 0; j < kB * 4; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
  }
  // Offset of key k0 + i of a tile; -1 where there is no such key. `base` is that of k0 where one page has all.
  auto offset = [&](int k0, int i, int64_t base) -> int64_t {
    if (k0 + i >= s.kv) return -1;
    return one_page ? (base < 0 ? -1 : base + i * row_step) : kv_offset(p, b, hk, k0 + i);
  };
  auto tile_base = [&](int w) -> int64_t {
    return one_page && w < w1 ? kv_offset(p, b, hk, walk.tile(w) * kKeys) : -1;
  };
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  int64_t base = tile_base(w0 + warp);
#pragma unroll 1
  for (int w = w0 + warp; w < w1; w += kWarps) {
    const int k0 = walk.tile(w) * kKeys;
    uint4 k[2][kC], v[4][kB];
    int64_t ko[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ko[i] = offset(k0, g + 8 * i, base);
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int d = 32 * c + 8 * t;
        k[i][c] = zero;
        if (ko[i] >= 0 && d < D) k[i][c] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.k) + ko[i] + d));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t vo = offset(k0, 2 * t + (i & 1) + 8 * (i >> 1), base);
#pragma unroll
      for (int c = 0; c < kB; ++c) {
        const int d = 64 * c + 8 * g;
        v[i][c] = zero;
        if (vo >= 0 && d < D) v[i][c] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.v) + vo + d));
      }
    }
    base = tile_base(w + kWarps);  // the table's answer for the next tile comes meanwhile
    uint32_t pt[NQ][2];            // the weights as the second product takes them
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float c4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        mma(c4, k[0][c].x, k[1][c].x, k[0][c].y, k[1][c].y, q[n][c].x, q[n][c].y);
        mma(c4, k[0][c].z, k[1][c].z, k[0][c].w, k[1][c].w, q[n][c].z, q[n][c].w);
      }
      // c4[e]: key g + 8 (e / 2), row 2 t + e % 2
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = k0 + g + 8 * (e >> 1), r = 8 * n + 2 * t + (e & 1);
        const bool seen = ko[e >> 1] >= 0 && r < rows && sees(s.pos0 + r / G, key, p.window, p.sinks);
        c4[e] = seen ? c4[e] * scale2 : kNegInf;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float top = over_keys_max(fmaxf(c4[e], c4[2 + e]));
        const bool move = top > m[n][e] + kSlack;
        if (__any_sync(kFull, move)) {
          const float f = move ? ex2(m[n][e] - top) : 1.f;
          l[n][e] *= f;
#pragma unroll
          for (int j = 0; j < kB * 4; ++j) {
            o[n][j][e] *= f;
            o[n][j][2 + e] *= f;
          }
          if (move) m[n][e] = top;
        }
        const float ref = m[n][e] == kNegInf ? 0.f : m[n][e];
        c4[e] = ex2(c4[e] - ref);
        c4[2 + e] = ex2(c4[2 + e] - ref);
        l[n][e] += c4[e] + c4[2 + e];
      }
      pt[n][0] = transpose8(pack(c4[0], c4[1]));
      pt[n][1] = transpose8(pack(c4[2], c4[3]));
    }
#pragma unroll
    for (int c = 0; c < kB; ++c) {
      const uint32_t x[4][4] = {{v[0][c].x, v[0][c].y, v[0][c].z, v[0][c].w},
                                {v[1][c].x, v[1][c].y, v[1][c].z, v[1][c].w},
                                {v[2][c].x, v[2][c].y, v[2][c].z, v[2][c].w},
                                {v[3][c].x, v[3][c].y, v[3][c].z, v[3][c].w}};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a0 = __byte_perm(x[0][j], x[1][j], 0x5410), a1 = __byte_perm(x[0][j], x[1][j], 0x7632);
        const uint32_t a2 = __byte_perm(x[2][j], x[3][j], 0x5410), a3 = __byte_perm(x[2][j], x[3][j], 0x7632);
#pragma unroll
        for (int n = 0; n < NQ; ++n) mma(o[n][4 * c + j], a0, a1, a2, a3, pt[n][0], pt[n][1]);
      }
    }
  }
  // ---- the warps' results. o[n][4 c + j][e]: column 64 c + 8 g + 2 j + e / 2, row 8 n + 2 t + e % 2
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * n + 2 * t + e;
      const float sum = over_keys_sum(l[n][e]);
      if (g == 0) {
        s_m[warp][r] = m[n][e];
        s_l[warp][r] = sum;
      }
#pragma unroll
      for (int c = 0; c < kB; ++c) {
        float* to = sm + (warp * kR + r) * DP + 64 * c + 8 * g;
        *reinterpret_cast<float4*>(to) = make_float4(o[n][4 * c][e], o[n][4 * c][2 + e], o[n][4 * c + 1][e], o[n][4 * c + 1][2 + e]);
        *reinterpret_cast<float4*>(to + 4) = make_float4(o[n][4 * c + 2][e], o[n][4 * c + 2][2 + e], o[n][4 * c + 3][e], o[n][4 * c + 3][2 + e]);
      }
    }
  __syncthreads();
  const int64_t total = (int64_t)p.T * p.H;
  for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
    const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
    float top = kNegInf;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
    const float ref = top == kNegInf ? 0.f : top;
    float sum = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(s_m[w][r] - ref);  // (a warp that saw nothing: 0)
      const float4 x = *reinterpret_cast<const float4*>(sm + (w * kR + r) * DP + d);
      sum = fmaf(f, s_l[w][r], sum);
      a.x = fmaf(f, x.x, a.x); a.y = fmaf(f, x.y, a.y); a.z = fmaf(f, x.z, a.z); a.w = fmaf(f, x.w, a.w);
    }
    const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;  // (a NaN stays one)
    const int64_t at = q_index(r);
    if (p.splits > 1)
      *reinterpret_cast<float4*>(p.part_o + (split * total + at) * D + d) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at * D + d) =
          make_uint2(pack(a.x * inv, a.y * inv), pack(a.z * inv, a.w * inv));
    if (d == 0) {
      const float lse = sum == 0.f ? kNegInf : (ref + log2f(sum)) * kLn2;
      if (p.splits > 1) p.part_lse[split * total + at] = lse;
      else if (p.lse) p.lse[at] = lse;
    }
  }
}

template <int DP, int NQ> cudaError_t launch_as(const AttnParams& p, cudaStream_t stream) {
  constexpr int bytes = kWarps * 8 * NQ * DP * 4;
  cudaError_t e = set_smem_limit<attn_decode_kernel<DP, NQ>>(bytes);
  if (e != cudaSuccess) return e;
  const int64_t grid = (int64_t)p.B * p.Hkv * p.splits;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  attn_decode_kernel<DP, NQ><<<(unsigned)grid, kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

bool attn_decode_supported(const AttnParams& p, rsm_dtype dtype) {
  return dtype == RSM_BF16 && p.table && (int64_t)p.max_q * p.G <= 16;
}

// Blocks that share a sequence's keys: where sequences and heads alone are fewer than four blocks per SM,
// enough for that, of at least 128 keys each (one tile per warp) by the table's width.
int attn_decode_splits(const AttnParams& p) {
  int64_t keys = (int64_t)p.table_width * p.page;
  if (p.window > 0) keys = std::min<int64_t>(keys, (int64_t)p.window + p.sinks + p.max_q);
  const int64_t want = 4 * device_sm_count() / std::max<int64_t>(1, (int64_t)p.B * p.Hkv);
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, keys / (kKeys * kWarps), 64}));
}

cudaError_t launch_attn_decode(const AttnParams& p, cudaStream_t stream) {
  const bool two = p.max_q * p.G > 8;
  if (p.D <= 64) return two ? launch_as<64, 2>(p, stream) : launch_as<64, 1>(p, stream);
  if (p.D <= 128) return two ? launch_as<128, 2>(p, stream) : launch_as<128, 1>(p, stream);
  return two ? launch_as<256, 2>(p, stream) : launch_as<256, 1>(p, stream);
}

}  // namespace rsm
