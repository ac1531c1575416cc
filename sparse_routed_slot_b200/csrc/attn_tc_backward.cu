// attn_tc_backward.cu -- gradients of window attention for bf16 inputs on the 5th-generation tensor cores.
//
// Two kernels, so that no sum depends on the order in which blocks finish (7 tile products per pair of
// tiles against the 5 of one kernel that would add dq up with atomics):
//   dk, dv: a block owns 128 keys and walks the packed query rows (token, head of the group) that see them
//     S^T = K Q^T, dP^T = V dO^T            (fp32 in TMEM, a thread per key)
//     P^T = 2^(S'^T - lse), dS^T = P^T (dP^T - delta)   -> bf16 in TMEM
//     dV += P^T dO, dK += dS^T Q            (Q and dO as TMA wrote them, contracted over their rows)
//   dq: a block owns 128 query rows and walks their keys
//     S = Q K^T, dP = dO V^T, dS = P (dP - delta) -> bf16 in TMEM, dQ += dS K
// P and dS are rounded to bf16 for their products (2^-9 each); delta comes from the stored o.
//
// The order of the products keeps the tensor core busy through the exponentials. dk, dv (512 TMEM columns
// in all: S^T, dP^T, dV, dK): dV_i, S_{i+1}, dK_i, dP_{i+1}: P_{i+1} is formed while dK_i and dP_{i+1} run,
// dS_{i+1} while dV_{i+1} and S_{i+2} do. dq: dP_{i+1}, dQ_i, S_{i+2} with two S buffers: dS_i over S_i,
// P_{i+1} formed during dP_{i+1}.
//
// Warps: 0-7 rows (warps 0-3 columns 0..63 of a tile, 4-7 columns 64..127), 8 copies, 9 MMA issuer.
//
// Keys below `sinks` are seen by every later row. Where that makes the first key tiles' walks much longer
// than a window, the part behind the window is cut into chunks for further blocks; these leave fp32 sums of
// the sink rows in the workspace, and a small kernel adds them in order.
#include <algorithm>

#include "attn_tc.cuh"

namespace rsm {

namespace {

using namespace attn;

constexpr int kBM = 128, kBN = 128;
constexpr int kThreads = 320, kRowThreads = 256;
constexpr int kCopyWarp = 8, kMmaWarp = 9;
constexpr int kChunkTiles = 16;  // query tiles per chunk behind the window
constexpr int kMaxSinkTiles = 4;

struct Maps {
  CUtensorMap q, k, v, dO;
};

template <int DP> struct Layout {
  static constexpr int kTile = kBM * DP * 2;
  static constexpr int kBytesKv = 6 * kTile + 1024;  // K, V, Q x 2, dO x 2
  static constexpr int kBytesQ = 7 * kTile + 1024;   // Q, dO, K x 3, V x 2
};

// K step j (16 columns) of a K-major tile: 32 bytes inside a 64-column block, then the next block.
RSM_DEV uint64_t kstep(int j) { return (uint64_t)(((j >> 2) * (kBM * 128) + (j & 3) * 32) >> 4); }
// K step j (16 rows) of an MN-major tile.
RSM_DEV uint64_t rstep(int j) { return (uint64_t)(j * 2048 >> 4); }
// TMEM column of K step j of a bf16 operand written over an fp32 tile by two groups of warps: columns
// 0..63 of the tile stand in its columns 0..31, columns 64..127 in its columns 64..95, so that no group
// writes where the other still reads.
RSM_DEV uint32_t acol(int j) { return (uint32_t)((j >> 2) * 64 + (j & 3) * 8); }

template <int DP>
RSM_DEV void product_ss(uint32_t d, uint64_t a, uint64_t b) {
  constexpr uint32_t id = tc::idesc_bf16(kBM, kBN, 0, 0);
#pragma unroll
  for (int j = 0; j < DP / 16; ++j) tc::mma_bf16_ss(d, a + kstep(j), b + kstep(j), id, j > 0);
}

template <int DP>
RSM_DEV void product_ts(uint32_t d, uint32_t a, uint64_t b, bool add) {
  constexpr uint32_t id = tc::idesc_bf16(kBM, DP, 0, 1);
#pragma unroll
  for (int j = 0; j < kBN / 16; ++j) tc::mma_bf16_ts(d, a + acol(j), b + rstep(j), id, add || j > 0);
}

struct Setup {
  unsigned char* sm;
  uint32_t tb;
};

RSM_DEV unsigned char* aligned_smem(unsigned char* raw) {
  return reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
}

// Rows [used, 128) of a tile, which no copy writes, as zeros (they are contracted over).
template <int DP> RSM_DEV void clear_rows(unsigned char* tile, int used) {
  for (int e = threadIdx.x; e < (kBM - used) * (DP / 8); e += kThreads) {
    const int row = used + e / (DP / 8), c = e % (DP / 8);
    *reinterpret_cast<uint4*>(tile + (c >> 3) * (kBM * 128) + row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
  }
}

template <int NC> RSM_DEV void store_row(__nv_bfloat16* to, uint32_t tmem, float scale, int cols, bool live) {
#pragma unroll
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

// How the walks of the key tiles are cut (host and device).
struct Chunks {
  int tiles;       // key tiles
  int sink_tiles;  // of them cut (0: none is)
  int far;         // chunks behind the window, per cut tile
  float* part;     // [pairs][sink_tiles][far + 1][128][2][D]
};

// Last query tile that a key tile's window reaches.
RSM_DEV int window_last(int k1, int T, int window, int tok_tile) {
  return (int)((min((int64_t)T, (int64_t)k1 + window) - 1) / tok_tile);
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_dkv_kernel(const __grid_constant__ Maps maps, const AttnParams p,
                                                                  int tok_tile, Chunks ch) {
  using L = Layout<DP>;
  constexpr int kBlocks = DP / 64;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t kv_full, q_full[2], q_empty[2], do_full[2], do_empty[2], st_full[2], s_full, dp_full, p_full,
      ds_full, fin;
  __shared__ __align__(16) float stat[2][2][kBM];  // per stage: lse (base 2) and delta of the rows
  __shared__ uint32_t s_tbase;

  // Blocks of the first key tiles, whose walks are longest, start first; behind them the far chunks.
  const int pairs = p.Hkv * p.B;
  const int pair = blockIdx.x % pairs, item = blockIdx.x / pairs;
  const bool is_far = item >= ch.tiles;
  const int kt = is_far ? (item - ch.tiles) % ch.sink_tiles : item;
  const int chunk = is_far ? 1 + (item - ch.tiles) / ch.sink_tiles : 0;
  const int hk = pair % p.Hkv, b = pair / p.Hkv;
  const int G = p.G, D = p.D, T = p.T;
  const int k0 = kt * kBN;
  const int k1 = min(k0 + kBN, T) - 1;
  const bool cut = kt < ch.sink_tiles;
  int j0 = k0 / tok_tile, j1;  // query tiles [j0, j1)
  {
    int t0, t1;
    query_range(k0, k1, T, p.window, p.sinks, t0, t1);
    j1 = (t1 - 1) / tok_tile + 1;
    if (cut) {
      const int w = window_last(k1, T, p.window, tok_tile) + 1;
      if (is_far) {
        j0 = min(w + (chunk - 1) * kChunkTiles, j1);
        j1 = min(j0 + kChunkTiles, j1);
      } else {
        j1 = w;
      }
    }
  }
  const int n = j1 - j0;
  const int rows_tile = tok_tile * G;

  unsigned char* sm = aligned_smem(smem_raw);
  unsigned char *sK = sm, *sV = sm + L::kTile, *sQ = sm + 2 * L::kTile, *sO = sm + 4 * L::kTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kMmaWarp) tc::tmem_alloc(&s_tbase, 512);
  if (threadIdx.x == 0) {
    tc::mbar_init(&kv_full, 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&q_full[i], 1);
      tc::mbar_init(&q_empty[i], 1);
      tc::mbar_init(&do_full[i], 1);
      tc::mbar_init(&do_empty[i], 1);
      tc::mbar_init(&st_full[i], 32);
    }
    tc::mbar_init(&s_full, 1);
    tc::mbar_init(&dp_full, 1);
    tc::mbar_init(&p_full, kRowThreads);
    tc::mbar_init(&ds_full, kRowThreads);
    tc::mbar_init(&fin, 1);
    tc::fence_mbar_init();
  }
  if (rows_tile < kBM) {
    for (int i = 0; i < 2; ++i) {
      clear_rows<DP>(sQ + i * L::kTile, rows_tile);
      clear_rows<DP>(sO + i * L::kTile, rows_tile);
    }
    tc::fence_async_smem();
  }
  tc::tmem_fence_before();
  __syncthreads();
  tc::tmem_fence_after();
  const uint32_t tb = s_tbase;
  const uint32_t cS = tb, cP = tb + 128, cV = tb + 256, cK = tb + 256 + DP;

  if (warp == kCopyWarp) {
    // =========================================================================== copies
    if (lane == 0) {
      tc::mbar_arrive_expect_tx(&kv_full, 2 * L::kTile);
      for (int c = 0; c < kBlocks; ++c) {
        tc::tma_load_4d(sK + c * (kBN * 128), &maps.k, &kv_full, 64 * c, hk, k0, b);
        tc::tma_load_4d(sV + c * (kBN * 128), &maps.v, &kv_full, 64 * c, hk, k0, b);
      }
    }
    __syncwarp();
    int nq = 0, ndo = 0;
    for (int i = 0; i < n; ++i) {
      const int st = i & 1, round = i >> 1;
      const int tok = (j0 + i) * tok_tile;
      auto copy = [&](uint64_t* full, const CUtensorMap* map, unsigned char* dst) {
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(full, (uint32_t)(rows_tile * 128 * kBlocks));
          for (int c = 0; c < kBlocks; ++c) tc::tma_load_4d(dst + c * (kBM * 128), map, full, 64 * c, hk * G, tok, b);
        }
        __syncwarp();
      };
      if (round > 0 && !wait_warp(&q_empty[st], (round - 1) & 1)) break;
      copy(&q_full[st], &maps.q, sQ + st * L::kTile);
      nq = i + 1;
      // the stage's statistics were last read for a dS that the emptied Q tile's product used
      const int rows = min(rows_tile, (T - tok) * G);
      float a[4], d[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = lane + 32 * e;
        const int64_t at = ((int64_t)b * T + tok + r / G) * p.H + hk * G + r % G;
        a[e] = r < rows ? p.lse[at] * kLog2e : 0.f;
        d[e] = r < rows ? p.delta[at] : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        stat[st][0][lane + 32 * e] = a[e];
        stat[st][1][lane + 32 * e] = d[e];
      }
      mbar_arrive(&st_full[st]);
      __syncwarp();
      if (round > 0 && !wait_warp(&do_empty[st], (round - 1) & 1)) break;
      copy(&do_full[st], &maps.dO, sO + st * L::kTile);
      ndo = i + 1;
    }
    // no copy may outlive the block, whatever became of its readers
    tc::mbar_wait(&kv_full, 0);
    for (int i = max(0, nq - 2); i < nq; ++i) tc::mbar_wait(&q_full[i & 1], (i >> 1) & 1);
    for (int i = max(0, ndo - 2); i < ndo; ++i) tc::mbar_wait(&do_full[i & 1], (i >> 1) & 1);
  } else if (warp == kMmaWarp) {
    // =========================================================================== MMA issuer
    const uint64_t dK = tc::smem_desc(tc::smem_u32(sK), 16, 1024), dV = tc::smem_desc(tc::smem_u32(sV), 16, 1024);
    const uint64_t dQ = tc::smem_desc(tc::smem_u32(sQ), 16, 1024), dO = tc::smem_desc(tc::smem_u32(sO), 16, 1024);
    const uint64_t rQ = tc::smem_desc(tc::smem_u32(sQ), kBM * 128, 1024), rO = tc::smem_desc(tc::smem_u32(sO), kBM * 128, 1024);
    auto stage = [](int i) -> uint64_t { return (uint64_t)(((i & 1) * L::kTile) >> 4); };
    if (tc::elect_one()) {
      auto scores = [&](int i) {
        product_ss<DP>(cS, dK, dQ + stage(i));
        tc::mma_commit(&s_full);
      };
      auto dprobs = [&](int i) {
        product_ss<DP>(cP, dV, dO + stage(i));
        tc::mma_commit(&dp_full);
      };
      bool ok = n > 0 && wait_one(&kv_full, 0) && wait_one(&q_full[0], 0);
      if (ok) {
        scores(0);
        ok = wait_one(&do_full[0], 0);
        if (ok) dprobs(0);
      }
#pragma unroll 1
      for (int i = 0; ok && i < n; ++i) {
        const int nx = i + 1;
        if (nx < n && !(ok = wait_one(&q_full[nx & 1], (nx >> 1) & 1))) break;
        if (!(ok = wait_one(&p_full, i & 1))) break;
        tc::tmem_fence_after();
        product_ts<DP>(cV, cS, rO + stage(i), i > 0);
        tc::mma_commit(&do_empty[i & 1]);
        if (nx < n) {
          scores(nx);
          if (!(ok = wait_one(&do_full[nx & 1], (nx >> 1) & 1))) break;
        }
        if (!(ok = wait_one(&ds_full, i & 1))) break;
        tc::tmem_fence_after();
        product_ts<DP>(cK, cP, rQ + stage(i), i > 0);
        tc::mma_commit(&q_empty[i & 1]);
        if (nx < n) dprobs(nx);
      }
      tc::mma_commit(&fin);
    }
    __syncwarp();
    tc::mbar_wait(&fin, 0);  // every MMA issued is done before the block gives up its memory
  } else {
    // =========================================================================== keys
    const int half = warp >> 2;
    const int r = threadIdx.x & 127;
    const int key = k0 + r;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32);
    const uint32_t tS = tc::tmem_addr(cS, lane_base, 64 * half), tP = tc::tmem_addr(cP, lane_base, 64 * half);
    const float scale2 = p.scale * kLog2e;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int tok = (j0 + i) * tok_tile;
      const int rows = min(rows_tile, (T - tok) * G);
      // rows [lo, hi) of the tile see the key
      const int lo = (key - tok) * G - 64 * half;
      const int64_t end = key < p.sinks ? rows : min((int64_t)rows, ((int64_t)key + p.window - tok) * G);
      const int hi = (int)max(end, (int64_t)0) - 64 * half;
      const bool whole = __all_sync(kFull, lo <= 0 && hi >= 64);
      const float4* sl = reinterpret_cast<const float4*>(&stat[i & 1][0][64 * half]);
      const float4* sd = reinterpret_cast<const float4*>(&stat[i & 1][1][64 * half]);
      if (!(ok = wait_warp(&st_full[i & 1], (i >> 1) & 1))) break;
      if (!(ok = wait_warp(&s_full, i & 1))) break;
      tc::tmem_fence_after();
      float x[64];
      tc::tmem_ld32(tS, *reinterpret_cast<float(*)[32]>(&x[0]));
      tc::tmem_ld32(tS + 32, *reinterpret_cast<float(*)[32]>(&x[32]));
      tc::tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 64; c += 4) {
        const float4 e = sl[c >> 2];
        x[c] = ex2(fmaf(x[c], scale2, -e.x));
        x[c + 1] = ex2(fmaf(x[c + 1], scale2, -e.y));
        x[c + 2] = ex2(fmaf(x[c + 2], scale2, -e.z));
        x[c + 3] = ex2(fmaf(x[c + 3], scale2, -e.w));
      }
      if (!whole) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c < lo || c >= hi) x[c] = 0.f;
      }
      {
        float w[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) w[c] = __uint_as_float(pack_bf16(x[2 * c], x[2 * c + 1]));
        tc::tmem_st32(tS, w);
      }
      tc::tmem_wait_st();
      tc::tmem_fence_before();
      mbar_arrive(&p_full);
      if (!(ok = wait_warp(&dp_full, i & 1))) break;
      tc::tmem_fence_after();
      float w[32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float y[32];
        tc::tmem_ld32(tP + 32 * h, y);
        tc::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 d = sd[(32 * h + c) >> 2];
          const float* q = &x[32 * h + c];
          // a row that does not see the key has a weight of zero and may have any dP: 0 * finite
          w[16 * h + c / 2] = __uint_as_float(pack_bf16(q[0] * (y[c] - d.x), q[1] * (y[c + 1] - d.y)));
          w[16 * h + c / 2 + 1] = __uint_as_float(pack_bf16(q[2] * (y[c + 2] - d.z), q[3] * (y[c + 3] - d.w)));
        }
      }
      tc::tmem_st32(tP, w);
      tc::tmem_wait_st();
      tc::tmem_fence_before();
      mbar_arrive(&ds_full);
    }
    if (ok) ok = wait_warp(&fin, 0);
    if (ok) {
      tc::tmem_fence_after();
      const uint32_t src = tc::tmem_addr(half ? cK : cV, lane_base, 0);
      const float f = half ? p.scale : 1.f;
      const bool to_part = cut && key < p.sinks;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(half ? p.dk : p.dv);
      const bool live = key < T && out && !is_far && !to_part && n > 0;
      store_row<DP>(out + (((int64_t)b * T + key) * p.Hkv + hk) * D, src, f, D, live);
      if (__any_sync(kFull, to_part && key < T)) {
        float* to = ch.part + ((((int64_t)pair * ch.sink_tiles + kt) * (ch.far + 1) + chunk) * kBN + r) * 2 * D + half * D;
#pragma unroll
        for (int c = 0; c < DP; c += 32) {
          float x[32];
          tc::tmem_ld32(src + c, x);
          tc::tmem_wait_ld();
          if (to_part && key < T) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              if (c + e < D)
                *reinterpret_cast<float4*>(to + c + e) =
                    n > 0 ? make_float4(x[e] * f, x[e + 1] * f, x[e + 2] * f, x[e + 3] * f) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
      }
    }
  }
  tc::tmem_fence_before();
  __syncthreads();
  tc::tmem_fence_after();
  if (warp == kMmaWarp) tc::tmem_dealloc(tb, 512);
}

// Adds the chunks of the sink rows up, in order, a warp per row.
__global__ void __launch_bounds__(256) sink_sum_kernel(const AttnParams p, Chunks ch) {
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int r = (int)(w % kBN);
  const int kt = (int)(w / kBN % ch.sink_tiles);
  const int64_t pair = w / kBN / ch.sink_tiles;
  const int key = kt * kBN + r;
  if (pair >= (int64_t)p.B * p.Hkv || key >= p.sinks || key >= p.T) return;
  const int hk = (int)(pair % p.Hkv);
  const int64_t b = pair / p.Hkv;
  const float* part = ch.part + ((pair * ch.sink_tiles + kt) * (ch.far + 1) * kBN + r) * 2 * p.D;
  const int64_t step = (int64_t)kBN * 2 * p.D;
  const int64_t at = ((b * p.T + key) * p.Hkv + hk) * p.D;
  for (int d = lane * 2; d < 2 * p.D; d += 64) {
    float2 s = make_float2(0.f, 0.f);
    for (int c = 0; c <= ch.far; ++c) {
      const float2 x = *reinterpret_cast<const float2*>(part + c * step + d);
      s.x += x.x;
      s.y += x.y;
    }
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(d < p.D ? p.dv : p.dk);
    if (out) *reinterpret_cast<uint32_t*>(out + at + (d < p.D ? d : d - p.D)) = pack_bf16(s.x, s.y);
  }
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_dq_kernel(const __grid_constant__ Maps maps, const AttnParams p,
                                                                 int tok_tile, int ntiles) {
  using L = Layout<DP>;
  constexpr int kBlocks = DP / 64;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t q_full, k_full[3], k_empty[3], v_full[2], v_empty[2], s_full[2], dp_full, ds_full, fin;
  __shared__ uint32_t s_tbase;

  const int tile = ntiles - 1 - blockIdx.x % ntiles;  // the last tiles see the most keys: they start first
  const int pair = blockIdx.x / ntiles;
  const int hk = pair % p.Hkv, b = pair / p.Hkv;
  const int G = p.G, D = p.D, T = p.T;
  const int tok0 = tile * tok_tile;
  const int ntok = min(tok_tile, T - tok0);
  const Walk walk = key_walk(tok0, tok0 + ntok - 1, T, p.window, p.sinks, kBN);
  const int n = walk.n;  // at least 1: every row sees itself

  unsigned char* sm = aligned_smem(smem_raw);
  unsigned char *sQ = sm, *sO = sm + L::kTile, *sK = sm + 2 * L::kTile, *sV = sm + 5 * L::kTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kMmaWarp) tc::tmem_alloc(&s_tbase, 512);
  if (threadIdx.x == 0) {
    tc::mbar_init(&q_full, 1);
    for (int i = 0; i < 3; ++i) {
      tc::mbar_init(&k_full[i], 1);
      tc::mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&v_full[i], 1);
      tc::mbar_init(&v_empty[i], 1);
      tc::mbar_init(&s_full[i], 1);
    }
    tc::mbar_init(&dp_full, 1);
    tc::mbar_init(&ds_full, kRowThreads);
    tc::mbar_init(&fin, 1);
    tc::fence_mbar_init();
  }
  tc::tmem_fence_before();
  __syncthreads();
  tc::tmem_fence_after();
  const uint32_t tb = s_tbase;
  const uint32_t cS = tb, cP = tb + 256, cQ = tb + 384;  // S at 0 and 128

  if (warp == kCopyWarp) {
    // =========================================================================== copies
    if (lane == 0) {
      tc::mbar_arrive_expect_tx(&q_full, (uint32_t)(2 * tok_tile * G * 128 * kBlocks));
      for (int c = 0; c < kBlocks; ++c) {
        tc::tma_load_4d(sQ + c * (kBM * 128), &maps.q, &q_full, 64 * c, hk * G, tok0, b);
        tc::tma_load_4d(sO + c * (kBM * 128), &maps.dO, &q_full, 64 * c, hk * G, tok0, b);
      }
    }
    __syncwarp();
    int nk = 0, nv = 0;
    for (int i = 0; i < n; ++i) {
      const int k0 = walk.tile(i) * kBN;
      auto copy = [&](uint64_t* full, const CUtensorMap* map, unsigned char* dst) {
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(full, L::kTile);
          for (int c = 0; c < kBlocks; ++c) tc::tma_load_4d(dst + c * (kBN * 128), map, full, 64 * c, hk, k0, b);
        }
        __syncwarp();
      };
      if (i >= 3 && !wait_warp(&k_empty[i % 3], (i / 3 - 1) & 1)) break;
      copy(&k_full[i % 3], &maps.k, sK + (i % 3) * L::kTile);
      nk = i + 1;
      if (i >= 2 && !wait_warp(&v_empty[i & 1], ((i >> 1) - 1) & 1)) break;
      copy(&v_full[i & 1], &maps.v, sV + (i & 1) * L::kTile);
      nv = i + 1;
    }
    // no copy may outlive the block, whatever became of its readers
    tc::mbar_wait(&q_full, 0);
    for (int i = max(0, nk - 3); i < nk; ++i) tc::mbar_wait(&k_full[i % 3], (i / 3) & 1);
    for (int i = max(0, nv - 2); i < nv; ++i) tc::mbar_wait(&v_full[i & 1], (i >> 1) & 1);
  } else if (warp == kMmaWarp) {
    // =========================================================================== MMA issuer
    const uint64_t dQ = tc::smem_desc(tc::smem_u32(sQ), 16, 1024), dO = tc::smem_desc(tc::smem_u32(sO), 16, 1024);
    const uint64_t dK = tc::smem_desc(tc::smem_u32(sK), 16, 1024), dV = tc::smem_desc(tc::smem_u32(sV), 16, 1024);
    const uint64_t rK = tc::smem_desc(tc::smem_u32(sK), kBN * 128, 1024);
    auto at = [](int i) -> uint64_t { return (uint64_t)((i * L::kTile) >> 4); };
    if (tc::elect_one()) {
      bool ok = wait_one(&q_full, 0);
      auto scores = [&](int i) {
        ok = ok && wait_one(&k_full[i % 3], (i / 3) & 1);
        if (!ok) return;
        product_ss<DP>(cS + (i & 1) * 128, dQ, dK + at(i % 3));
        tc::mma_commit(&s_full[i & 1]);
      };
      auto dprobs = [&](int i) {
        product_ss<DP>(cP, dO, dV + at(i & 1));
        tc::mma_commit(&dp_full);
        tc::mma_commit(&v_empty[i & 1]);
      };
      scores(0);
      ok = ok && wait_one(&v_full[0], 0);
      if (ok) dprobs(0);
      if (n > 1) scores(1);
#pragma unroll 1
      for (int i = 0; ok && i < n; ++i) {
        if (i + 1 < n && !(ok = wait_one(&v_full[(i + 1) & 1], ((i + 1) >> 1) & 1))) break;
        if (!(ok = wait_one(&ds_full, i & 1))) break;
        tc::tmem_fence_after();
        if (i + 1 < n) dprobs(i + 1);
        product_ts<DP>(cQ, cS + (i & 1) * 128, rK + at(i % 3), i > 0);
        tc::mma_commit(&k_empty[i % 3]);
        if (i + 2 < n) scores(i + 2);
      }
      tc::mma_commit(&fin);
    }
    __syncwarp();
    tc::mbar_wait(&fin, 0);  // every MMA issued is done before the block gives up its memory
  } else {
    // =========================================================================== rows
    const int half = warp >> 2;
    const int r = threadIdx.x & 127;
    const int pos = tok0 + r / G;
    const bool live = r < ntok * G;
    const int64_t row = ((int64_t)b * T + pos) * p.H + hk * G + r % G;
    const float lse = live ? p.lse[row] * kLog2e : 0.f, delta = live ? p.delta[row] : 0.f;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32);
    const uint32_t tS = tc::tmem_addr(cS, lane_base, 64 * half), tP = tc::tmem_addr(cP, lane_base, 64 * half);
    const float scale2 = p.scale * kLog2e;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int k0 = walk.tile(i) * kBN + 64 * half;
      if (!(ok = wait_warp(&s_full[i & 1], (i >> 1) & 1))) break;
      tc::tmem_fence_after();
      const uint32_t tSi = tS + (i & 1) * 128;
      float x[64];
      tc::tmem_ld32(tSi, *reinterpret_cast<float(*)[32]>(&x[0]));
      tc::tmem_ld32(tSi + 32, *reinterpret_cast<float(*)[32]>(&x[32]));
      tc::tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 64; ++c) x[c] = ex2(fmaf(x[c], scale2, -lse));
      const bool whole = k0 + 63 <= tok0 && (tok0 + ntok - 1 - k0 < p.window || k0 + 63 < p.sinks);
      if (!whole) {
        const int hi = pos - k0, lo = pos - p.window + 1 - k0, sk = p.sinks - k0;
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c > hi || (c < lo && c >= sk)) x[c] = 0.f;
      }
      if (!(ok = wait_warp(&dp_full, i & 1))) break;
      tc::tmem_fence_after();
      float w[32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float y[32];
        tc::tmem_ld32(tP + 32 * h, y);
        tc::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 32; c += 2)
          w[16 * h + c / 2] = __uint_as_float(
              pack_bf16(x[32 * h + c] * (y[c] - delta), x[32 * h + c + 1] * (y[c + 1] - delta)));
      }
      tc::tmem_st32(tSi, w);
      tc::tmem_wait_st();
      tc::tmem_fence_before();
      mbar_arrive(&ds_full);
    }
    if (ok) ok = wait_warp(&fin, 0);
    if (ok) {
      tc::tmem_fence_after();
      constexpr int kHalf = DP / 2;
      store_row<kHalf>(static_cast<__nv_bfloat16*>(p.dq) + row * D + half * kHalf, tc::tmem_addr(cQ, lane_base, half * kHalf),
                       p.scale, D - half * kHalf, live);
    }
  }
  tc::tmem_fence_before();
  __syncthreads();
  tc::tmem_fence_after();
  if (warp == kMmaWarp) tc::tmem_dealloc(tb, 512);
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

Chunks chunks_for(const AttnParams& p) {
  Chunks ch{};
  const int tok = kBM / p.G;
  ch.tiles = (p.T + kBN - 1) / kBN;
  const int ns = std::min((std::min(p.sinks, p.T) + kBN - 1) / kBN, ch.tiles);
  const int nq = (p.T + tok - 1) / tok;
  const int near = (int)((std::min<int64_t>(p.T, (int64_t)kBN - 1 + p.window) - 1) / tok) + 1;
  // worth it where the part behind the window is longer than two chunks: a cut costs each chunk's block
  // its own K and V tile and the sum of the parts
  if (ns > 0 && ns <= kMaxSinkTiles && nq - near > 2 * kChunkTiles) {
    ch.sink_tiles = ns;
    ch.far = (nq - near + kChunkTiles - 1) / kChunkTiles;
  }
  return ch;
}

size_t part_bytes(const AttnParams& p, const Chunks& ch) {
  return up256((size_t)p.B * p.Hkv * ch.sink_tiles * (ch.sink_tiles ? ch.far + 1 : 0) * kBN * 2 * p.D * sizeof(float));
}

template <int DP> cudaError_t launch_dp(const Maps& maps, const AttnParams& p, const Chunks& ch, cudaStream_t stream) {
  const int tok = kBM / p.G;
  const int64_t pairs = (int64_t)p.B * p.Hkv;
  if (p.dk || p.dv) {
    cudaError_t e = set_smem_limit<attn_tc_dkv_kernel<DP>>(Layout<DP>::kBytesKv);
    if (e != cudaSuccess) return e;
    const int64_t grid = pairs * (ch.tiles + (int64_t)ch.sink_tiles * ch.far);
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    attn_tc_dkv_kernel<DP><<<(unsigned)grid, kThreads, Layout<DP>::kBytesKv, stream>>>(maps, p, tok, ch);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (ch.sink_tiles) {
      sink_sum_kernel<<<(unsigned)((pairs * ch.sink_tiles * kBN + 7) / 8), 256, 0, stream>>>(p, ch);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
  }
  if (p.dq) {
    cudaError_t e = set_smem_limit<attn_tc_dq_kernel<DP>>(Layout<DP>::kBytesQ);
    if (e != cudaSuccess) return e;
    const int64_t ntiles = (p.T + tok - 1) / tok;
    if (ntiles * pairs > 0x7fffffff) return cudaErrorInvalidConfiguration;
    attn_tc_dq_kernel<DP><<<(unsigned)(ntiles * pairs), kThreads, Layout<DP>::kBytesQ, stream>>>(maps, p, tok, (int)ntiles);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t attn_tc_backward_bytes(const AttnParams& p) { return part_bytes(p, chunks_for(p)); }

cudaError_t launch_attn_tc_backward(const AttnParams& p, float* part, cudaStream_t stream) {
  Maps maps;
  const uint64_t D = p.D, H = p.H, Hkv = p.Hkv, T = p.T, B = p.B;
  const uint32_t tok = (uint32_t)(kBM / p.G);
  const std::array<uint64_t, 4> qd{D, H, T, B}, kd{D, Hkv, T, B};
  const std::array<uint64_t, 3> qs{D, H * D, T * H * D}, ks{D, Hkv * D, T * Hkv * D};
  const std::array<uint32_t, 4> qb{64, (uint32_t)p.G, tok, 1}, kb{64, 1, (uint32_t)kBN, 1};
  if (!make_map_bf16(&maps.q, p.q, qd, qs, qb) || !make_map_bf16(&maps.dO, p.dO, qd, qs, qb) ||
      !make_map_bf16(&maps.k, p.k, kd, ks, kb) || !make_map_bf16(&maps.v, p.v, kd, ks, kb))
    return cudaErrorInvalidValue;
  Chunks ch = chunks_for(p);
  ch.part = part;
  return p.D <= 64 ? launch_dp<64>(maps, p, ch, stream) : launch_dp<128>(maps, p, ch, stream);
}

}  // namespace rsm
