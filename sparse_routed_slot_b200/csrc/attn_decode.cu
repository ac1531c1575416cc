// attn_decode.cu -- paged attention of single tokens (and other calls with at most 16 query rows per
// key/value head and sequence), bf16.
//
// Such a call reads every key and value once and computes little: it is bound by that read. Each warp walks
// its own tiles of 16 keys (every fourth of the block's) through a ring in shared memory that it fills by
// asynchronous copies, 16 bytes per lane, two tiles ahead: the 8 warps of an SM keep 128 KB in flight (head
// dimension 128), and no warp waits for another until the end. An SM has two blocks, so that one's start and
// join hide behind the other's reads (one block of 8 warps: 128 sequences of 2048 keys, 16/4 heads of 128, 116 us
// against 106, of 100 keys, heads of 64, 32 against 19). (Straight to registers, 16 warps with a tile each got 4.0 TB/s,
// 8 warps with two tiles 3.7.) The rest are warp-level tensor products (m16n8k16) with Q's rows as the narrow
// side, so that none of it is wasted on up to 8 query rows:
//   S^T = K Q^T   16 keys x 8 rows. A product sums over columns in any order, so lane 4 g + t takes the
//                 contiguous columns 8 t .. 8 t + 7 of a block of 32 for keys g and g + 8
//   O^T += V^T P^T  16 columns x 8 rows over 16 keys. The lane has columns 8 g .. 8 g + 7 of keys 2 t, 2 t + 1,
//                 2 t + 8, 2 t + 9; byte permutes make the pairs of keys that the product takes, and column
//                 8 g + 2 j (+ 1) stands in row g (g + 8) of product j
//   P^T from S^T's accumulators by an 8 x 8 transpose across the lanes.
// With 9 to 16 rows of head dimension 256 the registers do not suffice (450 to 640 bytes spilled per thread): 64
// sequences of 4096 keys, 4 key/value heads, take 282 us there (3.8 TB/s), with up to 8 rows 170 to 174 (6.2 to 6.3).
// The weights are rounded to bf16 for the product; scores, statistics and sums are fp32. As in the tile
// kernel, the reference of a row's exponentials moves only past 2^32. The block's warps join at the end in
// shared memory. Up to 8 blocks that share a sequence's keys are a cluster and join through each other's
// shared memory (one launch and no workspace: the step of one short sequence 31 -> 24 us a call); more leave
// their results to a second kernel.
#include <cooperative_groups.h>

#include <algorithm>

#include "attention.cuh"

namespace rsm {

namespace {

using namespace attn;

constexpr int kKeys = 16;
constexpr float kNegInf = -__builtin_inff();
constexpr float kSlack = 32.f;
constexpr int kCluster = 8;  // blocks that may join through shared memory

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

template <int DP> struct Layout {
  static constexpr int kWarps = DP <= 128 ? 4 : 2, kThreads = 32 * kWarps;
  static constexpr int kTile = kKeys * DP * 2;            // bytes of a tile of keys (or values)
  static constexpr int kStages = DP <= 64 ? 6 : 3;        // 192 KB in all
  static constexpr int kBytes = kWarps * kStages * 2 * kTile;
};

// 16 bytes to shared memory, or zeros.
RSM_DEV void copy16(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
RSM_DEV uint4 lds16(uint32_t at) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at));
  return x;
}

// NQ: groups of 8 query rows. A row is (token, head of the group), as everywhere. ONE: a tile of keys stands in
// one page (pages of multiples of 16); else each half does (multiples of 8), or rows are looked up one by one.
// (40 sequences of 5000 keys, pages of 24: row by row 110 us, by halves 57; two starts per tile where one does
// cost 2 to 3 %.)
template <int DP, int NQ, bool ONE>
__global__ void __launch_bounds__(Layout<DP>::kThreads, 2) attn_decode_kernel(const AttnParams p) {
  using L = Layout<DP>;
  constexpr int kWarps = L::kWarps, kThreads = L::kThreads, kStages = L::kStages;
  constexpr int kR = 8 * NQ;
  constexpr int kC = DP / 32, kB = DP / 64;  // blocks of columns of the two products
  constexpr int kPieces = DP / 8;            // 16-byte pieces of a row
  extern __shared__ float sm[];              // the warps' rings, and at the end [warps][kR][DP]
  static_assert((kWarps + 1) * kR * DP * 4 <= L::kBytes, "the results fit the rings");
  __shared__ float s_m[kWarps][kR], s_l[kWarps][kR], s_top[kR], s_sum[kR];
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
  const Seen seen = keys_seen(s.pos0, s.pos0 + nq - 1, s.kv, p.window, p.sinks);
  const float scale2 = p.scale * kLog2e;
  const int64_t row_step = (int64_t)p.Hkv * D;
  const bool known = ONE || p.page % 8 == 0;  // where a tile's halves start is looked up ahead
  float m[NQ][2], l[NQ][2], o[NQ][kB * 4][4];
  int pos[NQ][2];  // places of rows 8 n + 2 t and + 1
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n][0] = m[n][1] = kNegInf;
    pos[n][0] = s.pos0 + (8 * n + 2 * t) / G;
    pos[n][1] = s.pos0 + (8 * n + 2 * t + 1) / G;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int j = 0; j < kB * 4; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
  }
  // Where a tile of keys, or each half of it, starts; -1 where it has no key that is seen, or no page.
  struct Base {
    int64_t part[ONE ? 1 : 2];
  };
  // Offset of key k0 + i of a tile; -1 where nothing sees it or it has no page.
  auto offset = [&](int k0, int i, const Base& base) -> int64_t {
    if (!seen.has(k0 + i)) return -1;
    if (!known) return kv_offset(p, b, hk, k0 + i);
    const int64_t from = base.part[ONE || i < 8 ? 0 : 1];
    return from < 0 ? -1 : from + (ONE ? i : i & 7) * row_step;
  };
  auto tile_base = [&](int w) {
    Base base;
    const int k0 = w < w1 ? walk.tile(w) * kKeys : 0;
#pragma unroll
    for (int h = 0; h < (ONE ? 1 : 2); ++h)
      base.part[h] = known && w < w1 && seen.any(k0 + 8 * h, ONE ? kKeys : 8) ? kv_offset(p, b, hk, k0 + 8 * h) : -1;
    return base;
  };
  auto held = [&](const Base& base) { return base.part[0] >= 0 && (ONE || base.part[ONE ? 0 : 1] >= 0); };
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sm) + warp * (kStages * 2 * L::kTile);
  // Pieces stand in an order of their own per row, so that the 8 lanes of a quarter warp read different banks:
  // lanes g = 2 i, 2 i + 1 and all t of the keys, lanes g = 2 i, 2 i + 1 and rows 2 t of the values.
  auto k_at = [](int row, int piece) { return (uint32_t)(row * DP * 2 + ((piece ^ ((row & 1) << 2)) << 4)); };
  auto v_at = [](int row, int piece) { return (uint32_t)(row * DP * 2 + ((piece ^ (row & 6)) << 4)); };
  // Nearly every tile is a whole one of known pages: its addresses are a lane's place plus multiples of a row, its
  // scores are all seen. (With the general arithmetic for every tile, 780 instructions per tile and warp, the
  // arithmetic and not the memory set the pace: 434 us for 256 sequences of 2048 to 4096 keys, 16/4 heads of 128,
  // which take 268 to 282 now.)
  const bool full_rows = known && D == DP;
  const __nv_bfloat16* lane_k = static_cast<const __nv_bfloat16*>(p.k) + (lane / kPieces) * row_step + 8 * (lane % kPieces);
  const __nv_bfloat16* lane_v = static_cast<const __nv_bfloat16*>(p.v) + (lane / kPieces) * row_step + 8 * (lane % kPieces);
  const int64_t hop = (32 / kPieces) * row_step;  // from one copy of the lane to its next
  auto fetch = [&](int w, const Base& base, int stage) {
    const uint32_t to = ring + stage * 2 * L::kTile;
    const int k0 = walk.tile(w) * kKeys;
    if (full_rows && w < w1 && held(base) && seen.all(k0, kKeys)) {
      const __nv_bfloat16 *fk = lane_k + base.part[0], *fv = lane_v + base.part[0];
#pragma unroll
      for (int i = 0; i < kKeys * kPieces / 32; ++i) {
        if (!ONE && i == kKeys * kPieces / 64) {
          fk = lane_k + base.part[ONE ? 0 : 1];
          fv = lane_v + base.part[ONE ? 0 : 1];
        }
        const int row = 32 / kPieces * i + lane / kPieces;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + k_at(row, lane % kPieces)), "l"(fk) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + L::kTile + v_at(row, lane % kPieces)), "l"(fv)
                     : "memory");
        fk += hop;
        fv += hop;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      return;
    }
#pragma unroll
    for (int i = 0; i < kKeys * kPieces / 32; ++i) {
      const int row = (32 * i + lane) / kPieces, piece = lane % kPieces;
      const int64_t off = w < w1 ? offset(k0, row, base) : -1;
      const bool there = off >= 0 && 8 * piece < D;
      const int64_t at = there ? off + 8 * piece : 0;
      copy16(to + k_at(row, piece), static_cast<const __nv_bfloat16*>(p.k) + at, there);
      copy16(to + L::kTile + v_at(row, piece), static_cast<const __nv_bfloat16*>(p.v) + at, there);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto attend = [&](int w, const Base& base, int stage) {
    const int k0 = walk.tile(w) * kKeys;
    const uint32_t from = ring + stage * 2 * L::kTile;
    const bool whole = known && held(base) && k0 + kKeys <= s.kv && k0 + kKeys - 1 <= s.pos0 &&
                       (p.window <= 0 || s.pos0 + nq - 1 - k0 < p.window || k0 + kKeys <= p.sinks);
    uint4 k[2][kC];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < kC; ++c) k[i][c] = lds16(from + k_at(g + 8 * i, 4 * c + t));
    uint32_t pt[NQ][2];            // the weights as the second product takes them
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float c4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        mma(c4, k[0][c].x, k[1][c].x, k[0][c].y, k[1][c].y, q[n][c].x, q[n][c].y);
        mma(c4, k[0][c].z, k[1][c].z, k[0][c].w, k[1][c].w, q[n][c].z, q[n][c].w);
      }
      // c4[e]: key g + 8 (e / 2), row 2 t + e % 2 (rows past the last are zeros, and stay finite)
#pragma unroll
      for (int e = 0; e < 4; ++e) c4[e] *= scale2;
      if (!whole) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = g + 8 * (e >> 1);
          if (offset(k0, i, base) < 0 || !sees(pos[n][e & 1], k0 + i, p.window, p.sinks)) c4[e] = kNegInf;
        }
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
      uint32_t v[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = lds16(from + L::kTile + v_at(2 * t + (i & 1) + 8 * (i >> 1), 8 * c + g));
        v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a0 = __byte_perm(v[0][j], v[1][j], 0x5410), a1 = __byte_perm(v[0][j], v[1][j], 0x7632);
        const uint32_t a2 = __byte_perm(v[2][j], v[3][j], 0x5410), a3 = __byte_perm(v[2][j], v[3][j], 0x7632);
#pragma unroll
        for (int n = 0; n < NQ; ++n) mma(o[n][4 * c + j], a0, a1, a2, a3, pt[n][0], pt[n][1]);
      }
    }
  };
  {
    // `base` of the tiles in the ring and of the one after them: the table's answer comes a step ahead of its use
    Base bases[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i) bases[i] = tile_base(w0 + warp + i * kWarps);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(w0 + warp + i * kWarps, bases[i], i);
    int stage = 0;
#pragma unroll 1
    for (int w = w0 + warp; w < w1; w += kWarps) {
      fetch(w + (kStages - 1) * kWarps, bases[kStages - 1], stage == 0 ? kStages - 1 : stage - 1);
      const Base coming = tile_base(w + kStages * kWarps);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();  // every lane's part of the tile
      attend(w, bases[0], stage);
      __syncwarp();  // the stage may be filled again
#pragma unroll
      for (int i = 0; i + 1 < kStages; ++i) bases[i] = bases[i + 1];
      bases[kStages - 1] = coming;
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
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
  const bool joined = p.splits > 1 && p.splits <= kCluster;
  float* mine = sm + kWarps * kR * DP;  // the block's own sums, where the cluster reads them: [kR][DP]
  auto finish = [&](int r, int d, float4 a, float sum, float ref) {
    const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;  // (a NaN stays one)
    const int64_t at = q_index(r);
    const float lse = sum == 0.f ? kNegInf : (ref + log2f(sum)) * kLn2;
    a = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    if (p.splits > kCluster) {
      *reinterpret_cast<float4*>(p.part_o + (split * total + at) * D + d) = a;
      if (d == 0) p.part_lse[split * total + at] = lse;
    } else {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at * D + d) = make_uint2(pack(a.x, a.y), pack(a.z, a.w));
      if (d == 0 && p.lse) p.lse[at] = lse;
    }
  };
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
    if (!joined) {
      finish(r, d, a, sum, ref);
    } else {
      *reinterpret_cast<float4*>(mine + r * DP + d) = a;
      if (d == 0) {
        s_top[r] = top;
        s_sum[r] = sum;
      }
    }
  }
  if (!joined) return;
  // every block of the cluster has its sums ready; each finishes its share of the outputs
  cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  cluster.sync();
  for (int e = split * kThreads + threadIdx.x; e < rows * (D / 4); e += p.splits * kThreads) {
    const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
    float top = kNegInf;
    for (int i = 0; i < p.splits; ++i) top = fmaxf(top, *cluster.map_shared_rank(&s_top[r], i));
    const float ref = top == kNegInf ? 0.f : top;
    float sum = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < p.splits; ++i) {
      const float f = ex2(*cluster.map_shared_rank(&s_top[r], i) - ref);
      const float4 x = *reinterpret_cast<const float4*>(cluster.map_shared_rank(mine + r * DP + d, i));
      sum = fmaf(f, *cluster.map_shared_rank(&s_sum[r], i), sum);
      a.x = fmaf(f, x.x, a.x); a.y = fmaf(f, x.y, a.y); a.z = fmaf(f, x.z, a.z); a.w = fmaf(f, x.w, a.w);
    }
    finish(r, d, a, sum, ref);
  }
  cluster.sync();  // no block leaves while another reads its memory
}

template <int DP, int NQ, bool ONE> cudaError_t launch_as(const AttnParams& p, cudaStream_t stream) {
  constexpr int bytes = Layout<DP>::kBytes;
  static_assert(bytes <= 232448 - 4096, "shared memory budget");
  cudaError_t e = set_smem_limit<attn_decode_kernel<DP, NQ, ONE>>(bytes);
  if (e != cudaSuccess) return e;
  const int64_t grid = (int64_t)p.B * p.Hkv * p.splits;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (p.splits == 1 || p.splits > kCluster) {
    attn_decode_kernel<DP, NQ, ONE><<<(unsigned)grid, Layout<DP>::kThreads, bytes, stream>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3((unsigned)grid);
  config.blockDim = dim3(Layout<DP>::kThreads);
  config.dynamicSmemBytes = bytes;
  config.stream = stream;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = (unsigned)p.splits;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  config.attrs = &cluster;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, attn_decode_kernel<DP, NQ, ONE>, p);
}

}  // namespace

bool attn_decode_supported(const AttnParams& p, rsm_dtype dtype) {
  // (a cache of no pages has no address to copy from)
  return dtype == RSM_BF16 && p.table && p.num_pages > 0 && p.table_width > 0 && (int64_t)p.max_q * p.G <= 16;
}

// Blocks that share a sequence's keys: where sequences and heads alone are fewer blocks than stay resident (two
// per SM), enough for that, of at least 128 keys each by the table's width. (Twice as many: 40 sequences of
// 5000 keys, 8/2 heads of 80, 79 us against 54; 32 of 2048, 16/4 heads of 128, 49 against 42.)
int attn_decode_splits(const AttnParams& p) {
  int64_t keys = (int64_t)p.table_width * p.page;
  if (p.window > 0) keys = std::min<int64_t>(keys, (int64_t)p.window + p.sinks + p.max_q);
  const int64_t want = 2 * device_sm_count() / std::max<int64_t>(1, (int64_t)p.B * p.Hkv);
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, keys / (kKeys * 8), 64}));
}

bool attn_decode_joins(const AttnParams& p) { return p.splits <= kCluster; }

template <int DP> cudaError_t launch_rows(const AttnParams& p, cudaStream_t stream) {
  const bool two = p.max_q * p.G > 8, one = p.page % kKeys == 0;
  if (two) return one ? launch_as<DP, 2, true>(p, stream) : launch_as<DP, 2, false>(p, stream);
  return one ? launch_as<DP, 1, true>(p, stream) : launch_as<DP, 1, false>(p, stream);
}

cudaError_t launch_attn_decode(const AttnParams& p, cudaStream_t stream) {
  return p.D <= 64 ? launch_rows<64>(p, stream) : p.D <= 128 ? launch_rows<128>(p, stream) : launch_rows<256>(p, stream);
}

}  // namespace rsm
