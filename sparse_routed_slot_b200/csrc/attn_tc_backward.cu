// attn_tc_backward.cu -- gradients of window attention for bf16 inputs on the 5th-generation tensor cores.
//
// Two runs of one kernel, so that no sum depends on the order in which blocks finish (7 tile products per
// pair of tiles against the 5 of one kernel that would add dq up with atomics). A block owns 128 rows
// (A1, A2) and walks those they meet in tiles of 64 (B1, B2):
//   dk, dv: A = keys (k, v), B = packed query rows (token, head of the group) that see them (q, dO)
//   dq:     A = packed query rows (q, dO), B = the keys they see (k, v)
//   S = A1 B1^T, E = A2 B2^T             fp32 in TMEM, a thread per row of A
//   P = 2^(S' - lse), Z = P (E - delta)  -> bf16 over S and E (rounded here: the next products take bf16)
//   G2 += Z B1  (dk or dq),  G1 += P B2  (dv; not in the dq run)
// delta = dO . o is formed with what rounding left of o where the forward kept it.
// S and E have two buffers each and two groups of 128 threads take the steps in turn, so S and E of the
// next step are there when a group comes back, and one group's exponentials run beside the other's loads.
// The tiles of 64 leave room for four stages of B: with 128 and two, each step waited for its copies
// (5500 cycles per 128 query rows for dk and dv, of which the tensor core needs 2560: S and E of 64 columns
// run at 3/4 rate, bound by their operands from shared memory).
//
// S, E and G are issued by threads of two warps: a satisfied wait costs an issuer 200 cycles in which it
// queues nothing, and one that had both (two waits per step) left the tensor core idle 2 of 5 cycles.
//
// Warps: 0-3 even steps, 4-7 odd steps, 8 copies (TMA), 9 issuer of S and E, 10 issuer of G1 and G2.
// TMEM columns: S buffers at 0 and 64, E buffers at 128 and 192, G2 at 256, G1 at 256 + DP.
//
// Keys below `sinks` are seen by every later row. Where that makes the first key tiles' walks much longer
// than a window, the part behind the window is cut into chunks for further blocks; these leave fp32 sums of
// the sink rows in the workspace, and a small kernel adds them in order.
#include <algorithm>

#include "attn_tc.cuh"

namespace rsm {

namespace {

using namespace attn;

constexpr int kBM = 128, kBN = 64;
constexpr int kThreads = 352;
constexpr int kCopyWarp = 8, kScoreWarp = 9, kGradWarp = 10;
constexpr int kStages = 4;
constexpr int kMinChunk = 16;  // query tiles per chunk behind the window, at least
constexpr int kMaxSinkTiles = 4;
constexpr int kStatRows = 32;   // rows per block of the statistics

// A: the block's rows, B: the rows that pass by (of 1 = q or k, 2 = dO or v); g1, g2: the results
struct Maps {
  CUtensorMap a1, a2, b1, b2, g1, g2;
};

template <int DP> struct Layout {
  static constexpr int kA = kBM * DP * 2, kB = kBN * DP * 2;
  static constexpr int kOffB = 2 * kA;
  static constexpr int kOffStat = kOffB + kStages * 2 * kB;
  static constexpr int kBytes = kOffStat + kStages * 512 + 1024;
  static_assert(kBytes <= 232448 - 1024, "shared memory budget");
};

// How the walks of the key tiles are cut.
struct Chunks {
  int tiles;       // key tiles
  int sink_tiles;  // of them cut (0: none is)
  int far;         // chunks behind the window, per cut tile
  int size;        // query tiles per chunk
  float* part;     // [pairs][sink_tiles][far + 1][128][2][D]
};

// The packed rows' statistics, in tiles of 64 rows: -lse (base 2) of the rows, then -delta.
RSM_DEV float* stat_of(float* stat, int64_t pair, int ntiles, int tok, int g, int tok_tile, int G) {
  const int tile = tok / tok_tile;
  return stat + (pair * ntiles + tile) * 2 * kBN + (tok - tile * tok_tile) * G + g;
}

// Last query tile that a key tile's window reaches.
RSM_DEV int window_last(int k1, int T, int window, int tok_tile) {
  return (int)((min((int64_t)T, (int64_t)k1 + window) - 1) / tok_tile);
}

// ntiles: dq: query tiles of 128 rows per pair; otherwise query tiles of 64 rows (the statistics').
template <int DP, bool DQ>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_backward_kernel(const __grid_constant__ Maps maps, const AttnParams p,
                                                                       int ntiles, int stat_tiles, Chunks ch) {
  using L = Layout<DP>;
  constexpr int kBlocks = DP / 64;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t a_full, full[kStages], empty[kStages], s_full[2], w_full[2], fin;
  __shared__ uint32_t s_tbase;

  const int G = p.G, D = p.D, T = p.T;
  const int tok64 = kBN / G;              // tokens of a tile of 64 packed rows
  const int tok_a = DQ ? kBM / G : 0;     // tokens of the block's query tile (dq)
  const int rows_b = DQ ? kBN : tok64 * G;  // rows that a copy brings

  // ---- what this block owns and walks
  int pair, tile, chunk = 0;
  bool is_far = false;
  if (DQ) {
    tile = ntiles - 1 - blockIdx.x % ntiles;  // the last tiles see the most keys: they start first
    pair = blockIdx.x / ntiles;
  } else {
    // blocks of the first key tiles, whose walks are longest, start first; behind them the far chunks
    const int pairs = p.Hkv * p.B;
    const int item = blockIdx.x / pairs;
    pair = blockIdx.x % pairs;
    is_far = item >= ch.tiles;
    tile = is_far ? (item - ch.tiles) % ch.sink_tiles : item;
    chunk = is_far ? 1 + (item - ch.tiles) / ch.sink_tiles : 0;
  }
  const int hk = pair % p.Hkv, b = pair / p.Hkv;
  const int tok0 = DQ ? tile * tok_a : 0;            // dq: the block's tokens [tok0, tok0 + ntok)
  const int ntok = DQ ? min(tok_a, T - tok0) : 0;
  const int key0 = DQ ? 0 : tile * kBM;              // dk, dv: the block's keys from key0 on
  const bool cut = !DQ && tile < ch.sink_tiles;
  Walk walk{0, 0, 0};
  if (DQ) {
    walk = key_walk(tok0, tok0 + ntok - 1, T, p.window, p.sinks, kBN);
  } else {
    const int k1 = min(key0 + kBM, T) - 1;
    int t0, t1;
    query_range(key0, k1, T, p.window, p.sinks, t0, t1);
    int j0 = t0 / tok64, j1 = (t1 - 1) / tok64 + 1;
    if (cut) {
      const int w = window_last(k1, T, p.window, tok64) + 1;
      if (is_far) {
        j0 = min(w + (chunk - 1) * ch.size, j1);
        j1 = min(j0 + ch.size, j1);
      } else {
        j1 = w;
      }
    }
    walk.first = j0;
    walk.n = j1 - j0;
  }
  const int n = walk.n;

  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kScoreWarp) tc::tmem_alloc(&s_tbase, 512);
  if (threadIdx.x == 0) {
    tc::mbar_init(&a_full, 1);
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s_full[i], 1);
      tc::mbar_init(&w_full[i], 4);
    }
    tc::mbar_init(&fin, 2);
    tc::fence_mbar_init();
  }
  if constexpr (!DQ) {
    // rows of a tile that no copy writes are contracted over all the same: zero
    const int gap = kBN - rows_b;
    for (int e = threadIdx.x; e < kStages * 2 * gap * (DP / 8); e += kThreads) {
      const int c = e % (DP / 8), row = rows_b + e / (DP / 8) % gap, which = e / (DP / 8) / gap;
      *reinterpret_cast<uint4*>(sm + L::kOffB + which * L::kB + (c >> 3) * (kBN * 128) + row * 128 + (c & 7) * 16) =
          make_uint4(0, 0, 0, 0);
    }
    tc::fence_async_smem();
  }
  tc::tmem_fence_before();
  __syncthreads();
  tc::tmem_fence_after();
  const uint32_t tb = s_tbase;
  const uint32_t c2 = tb + 256, c1 = tb + 256 + DP;

  if (warp == kCopyWarp) {
    // =========================================================================== copies
    if (tc::elect_one()) {
      const int head_a = DQ ? hk * G : hk, row_a = DQ ? tok0 : key0;
      const int head_b = DQ ? hk : hk * G;
      tc::mbar_arrive_expect_tx(&a_full, (uint32_t)(2 * (DQ ? tok_a * G : kBM) * 128 * kBlocks));
      for (int c = 0; c < kBlocks; ++c) {
        tc::tma_load_4d(sm + c * (kBM * 128), &maps.a1, &a_full, 64 * c, head_a, row_a, b);
        tc::tma_load_4d(sm + L::kA + c * (kBM * 128), &maps.a2, &a_full, 64 * c, head_a, row_a, b);
      }
      int issued = 0;
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const int st = i % kStages;
        if (i >= kStages && !wait_one(&empty[st], (i / kStages - 1) & 1)) break;
        const int j = walk.tile(i);
        const int row = DQ ? j * kBN : j * tok64;
        unsigned char* dst = sm + L::kOffB + st * 2 * L::kB;
        tc::mbar_arrive_expect_tx(&full[st], (uint32_t)(2 * rows_b * 128 * kBlocks + (DQ ? 0 : 512)));
        if (!DQ)
          tc::bulk_load(sm + L::kOffStat + st * 512, p.delta + ((int64_t)pair * stat_tiles + j) * 2 * kBN, 512, &full[st]);
        for (int c = 0; c < kBlocks; ++c) {
          tc::tma_load_4d(dst + c * (kBN * 128), &maps.b1, &full[st], 64 * c, head_b, row, b);
          tc::tma_load_4d(dst + L::kB + c * (kBN * 128), &maps.b2, &full[st], 64 * c, head_b, row, b);
        }
        issued = i + 1;
      }
      // no copy may outlive the block, whatever became of its readers
      tc::mbar_wait(&a_full, 0);
      for (int i = max(0, issued - kStages); i < issued; ++i) tc::mbar_wait(&full[i % kStages], (i / kStages) & 1);
    }
    __syncwarp();
  } else if (warp == kScoreWarp) {
    // =========================================================================== issuer of S and E
    constexpr uint32_t kId = tc::idesc_bf16(kBM, kBN, 0, 0);
    const uint64_t a1 = tc::smem_desc(tc::smem_u32(sm), 16, 1024), a2 = a1 + (uint64_t)(L::kA >> 4);
    const uint64_t dB = tc::smem_desc(tc::smem_u32(sm + L::kOffB), 16, 1024);
    auto kstep = [](int R, int j) -> uint64_t { return (uint64_t)(((j >> 2) * (R * 128) + (j & 3) * 32) >> 4); };
    if (tc::elect_one()) {
      bool ok = wait_one(&a_full, 0);
#pragma unroll 1
      for (int c = 0; ok && c < n; ++c) {
        // buffer c & 1 is free once the products of step c - 2 are done, which lets go of its stage, too
        ok = wait_one(&full[c % kStages], (c / kStages) & 1) &&
             (c < 2 || wait_one(&empty[(c - 2) % kStages], ((c - 2) / kStages) & 1));
        if (!ok) break;
        tc::tmem_fence_after();
        const uint64_t b1 = dB + (uint64_t)((c % kStages * 2 * L::kB) >> 4), b2 = b1 + (uint64_t)(L::kB >> 4);
#pragma unroll
        for (int j = 0; j < DP / 16; ++j)
          tc::mma_bf16_ss(tb + (c & 1) * kBN, a1 + kstep(kBM, j), b1 + kstep(kBN, j), kId, j > 0);
#pragma unroll
        for (int j = 0; j < DP / 16; ++j)
          tc::mma_bf16_ss(tb + 128 + (c & 1) * kBN, a2 + kstep(kBM, j), b2 + kstep(kBN, j), kId, j > 0);
        tc::mma_commit(&s_full[c & 1]);
      }
      tc::mma_commit(&fin);
    }
    __syncwarp();
    tc::mbar_wait(&fin, 0);  // every MMA issued is done before the block gives up its memory
  } else if (warp == kGradWarp) {
    // =========================================================================== issuer of G1 and G2
    constexpr uint32_t kId = tc::idesc_bf16(kBM, DP, 0, 1);
    // the tiles of B contracted over their rows: 64-column blocks 8 KB apart, 16 rows 2 KB
    const uint64_t rB = tc::smem_desc(tc::smem_u32(sm + L::kOffB), kBN * 128, 1024);
    if (tc::elect_one()) {
      bool ok = true;
#pragma unroll 1
      for (int i = 0; ok && i < n; ++i) {
        const int st = i % kStages;
        ok = wait_one(&full[st], (i / kStages) & 1) && wait_one(&w_full[i & 1], (i >> 1) & 1);
        if (!ok) break;
        tc::tmem_fence_after();
        const uint64_t r1 = rB + (uint64_t)((st * 2 * L::kB) >> 4), r2 = r1 + (uint64_t)(L::kB >> 4);
        const uint32_t aP = tb + (i & 1) * kBN, aZ = tb + 128 + (i & 1) * kBN;
        if (!DQ) {
#pragma unroll
          for (int j = 0; j < kBN / 16; ++j)
            tc::mma_bf16_ts(c1, aP + 8 * j, r2 + (uint64_t)(j * 2048 >> 4), kId, i > 0 || j > 0);
        }
#pragma unroll
        for (int j = 0; j < kBN / 16; ++j)
          tc::mma_bf16_ts(c2, aZ + 8 * j, r1 + (uint64_t)(j * 2048 >> 4), kId, i > 0 || j > 0);
        tc::mma_commit(&empty[st]);
      }
      tc::mma_commit(&fin);
    }
    __syncwarp();
    tc::mbar_wait(&fin, 0);
  } else {
    // =========================================================================== rows of A
    const int u = warp >> 2;
    const int r = threadIdx.x & 127;
    const int key = key0 + r;                                       // dk, dv
    const int pos = tok0 + r / G;                                   // dq
    const bool live = DQ ? r < ntok * G : key < T;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32);
    const uint32_t tS = tc::tmem_addr(tb, lane_base, u * kBN), tE = tc::tmem_addr(tb, lane_base, 128 + u * kBN);
    const float2 s2 = make_float2(p.scale * kLog2e, p.scale * kLog2e);
    float2 nl = make_float2(0.f, 0.f), nd = nl;  // dq: the row's statistics
    if (DQ && live) {
      const float* st = stat_of(p.delta, pair, stat_tiles, pos, r % G, tok64, G);
      nl = make_float2(st[0], st[0]);
      nd = make_float2(st[kBN], st[kBN]);
    }
    bool ok = true;
#pragma unroll 1
    for (int i = u; i < n; i += 2) {
      // columns [lo, hi) of the step, and [0, sk), meet this row
      const int j = walk.tile(i);
      int lo, hi, sk = 0;
      bool whole;
      if (DQ) {
        const int k0 = j * kBN;
        hi = pos - k0 + 1;
        lo = pos - p.window + 1 - k0;
        sk = min(p.sinks - k0, hi);
        whole = k0 + kBN - 1 <= tok0 && (tok0 + ntok - 1 - k0 < p.window || k0 + kBN - 1 < p.sinks);
      } else {
        const int tok = j * tok64;
        const int rows = min(rows_b, (T - tok) * G);
        lo = (key - tok) * G;
        hi = key < p.sinks ? rows : (int)min((int64_t)rows, max((int64_t)0, ((int64_t)key + p.window - tok) * G));
        whole = __all_sync(kFull, lo <= 0 && hi >= kBN);
      }
      const uint32_t m0 = whole ? ~0u : (below(hi) & ~below(lo)) | below(sk);
      const uint32_t m1 = whole ? ~0u : (below(hi - 32) & ~below(lo - 32)) | below(sk - 32);
      const float2* stl = reinterpret_cast<const float2*>(sm + L::kOffStat + (i % kStages) * 512);
      if (!DQ && !(ok = wait_warp(&full[i % kStages], (i / kStages) & 1))) break;
      if (!(ok = wait_warp(&s_full[u], (i >> 1) & 1))) break;
      tc::tmem_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x[32], e[32];
        tc::tmem_ld32(tS + 32 * h, x);
        tc::tmem_ld32(tE + 32 * h, e);
        tc::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 l2 = DQ ? nl : stl[16 * h + c / 2], d2 = DQ ? nd : stl[kBN / 2 + 16 * h + c / 2];
          float2 w = fma2(make_float2(x[c], x[c + 1]), s2, l2);
          w.x = ex2(w.x);
          w.y = ex2(w.y);
          const float2 z = mul2(w, add2(make_float2(e[c], e[c + 1]), d2));
          x[c] = w.x; x[c + 1] = w.y;
          e[c] = z.x; e[c + 1] = z.y;
        }
        if (!whole) {
          const uint32_t m = h ? m1 : m0;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!(m & (1u << c))) x[c] = e[c] = 0.f;
        }
        float w[16];
        if (!DQ) {
#pragma unroll
          for (int c = 0; c < 16; ++c) w[c] = __uint_as_float(pack_bf16(x[2 * c], x[2 * c + 1]));
          tc::tmem_st16(tS + 16 * h, w);
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) w[c] = __uint_as_float(pack_bf16(e[2 * c], e[2 * c + 1]));
        tc::tmem_st16(tE + 16 * h, w);
      }
      tc::tmem_wait_st();
      tc::tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&w_full[u]);
    }
    if (ok) ok = wait_warp(&fin, 0);
    tc::tmem_fence_after();
    // The tiles of A are done with: the results go through their memory to tensor stores, which leave out
    // what lies behind the last row and column. (Stored by the row's threads, 16 bytes each at the rows'
    // distance, they took 6000 cycles.)
    if (DQ) {
      constexpr int kHalf = DP / 2;  // each group has half of the columns
      if (ok) stage_row<kHalf>(sm, r, u * kHalf, tc::tmem_addr(c2, lane_base, u * kHalf), p.scale);
      tc::fence_async_smem();
      group_sync(1, 256);
      if (ok && threadIdx.x == 0) {
        for (int c = 0; c < kBlocks; ++c) tc::tma_store_4d(&maps.g2, sm + c * (kBM * 128), 64 * c, hk * G, tok0, b);
        tc::bulk_commit_group();
        tc::bulk_wait_read_all();
      }
    } else {
      const uint32_t src = tc::tmem_addr(u ? c2 : c1, lane_base, 0);  // group 0 has dv, group 1 dk
      const float f = u ? p.scale : 1.f;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(u ? p.dk : p.dv);
      if (!cut) {
        unsigned char* to = sm + u * L::kA;
        if (ok) stage_row<DP>(to, r, 0, src, f);
        tc::fence_async_smem();
        group_sync(1 + u, 128);
        if (ok && out && r == 0) {
          for (int c = 0; c < kBlocks; ++c)
            tc::tma_store_4d(u ? &maps.g2 : &maps.g1, to + c * (kBM * 128), 64 * c, hk, key0, b);
          tc::bulk_commit_group();
          tc::bulk_wait_read_all();
        }
      } else if (ok) {
        // the sink rows' sums go to the workspace; the first block of a cut tile has all of its other rows
        const bool to_part = key < p.sinks;
        store_row<DP>(out + (((int64_t)b * T + key) * p.Hkv + hk) * D, src, f, D, live && out && !is_far && !to_part);
        if (__any_sync(kFull, to_part && live)) {
          float* to = ch.part + ((((int64_t)pair * ch.sink_tiles + tile) * (ch.far + 1) + chunk) * kBM + r) * 2 * D + u * D;
#pragma unroll 1
          for (int c = 0; c < DP; c += 32) {
            float x[32];
            tc::tmem_ld32(src + c, x);
            tc::tmem_wait_ld();
            if (to_part && live) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                if (c + e < D)
                  *reinterpret_cast<float4*>(to + c + e) = n > 0 ? make_float4(x[e] * f, x[e + 1] * f, x[e + 2] * f, x[e + 3] * f)
                                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
            }
          }
        }
      }
    }
  }
  tc::tmem_fence_before();
  __syncthreads();
  tc::tmem_fence_after();
  if (warp == kScoreWarp) tc::tmem_dealloc(tb, 512);
}

// Statistics of every query row: -lse in base 2 and -delta, delta = dO . o; half a warp has two rows (131072
// rows of 128 columns: one row 28 us, two 22; its reads take 15 at the copy rate).
__global__ void __launch_bounds__(256) stat_kernel(const AttnParams p, int64_t rows, int tok_tile, int ntiles) {
  const int64_t first = (int64_t)blockIdx.x * kStatRows + (threadIdx.x >> 4);
  const int lane = threadIdx.x & 15;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  uint4 x[2], y[2], z[2];
  float lse[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t row = first + 16 * u, at = row * p.D + lane * 8;
    const bool there = row < rows && lane * 8 < p.D;
    x[u] = there ? *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.dO) + at) : none;
    y[u] = there ? *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.o) + at) : none;
    z[u] = there && p.o_low ? *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.o_low) + at) : none;
    lse[u] = row < rows ? p.lse[row] : 0.f;
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint32_t a[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, b[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
    const uint32_t c[4] = {z[u].x, z[u].y, z[u].z, z[u].w};
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16) + __uint_as_float(c[i] << 16), sum);
      sum = fmaf(__uint_as_float(a[i] & 0xffff0000u),
                 __uint_as_float(b[i] & 0xffff0000u) + __uint_as_float(c[i] & 0xffff0000u), sum);
    }
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    const int64_t row = first + 16 * u;
    if (lane == 0 && row < rows) {
      const int h = (int)(row % p.H);
      const int64_t t = row / p.H;
      float* to = stat_of(p.delta, t / p.T * p.Hkv + h / p.G, ntiles, (int)(t % p.T), h % p.G, tok_tile, p.G);
      to[0] = -lse[u] * kLog2e;
      to[kBN] = -sum;
    }
  }
}

// Adds the chunks of the sink rows up, in order, a warp per row.
__global__ void __launch_bounds__(256) sink_sum_kernel(const AttnParams p, Chunks ch, int sinks) {
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int key = (int)(w % sinks), kt = key / kBM, r = key % kBM;
  const int64_t pair = w / sinks;
  if (pair >= (int64_t)p.B * p.Hkv) return;
  const int hk = (int)(pair % p.Hkv);
  const int64_t b = pair / p.Hkv;
  const float* part = ch.part + ((pair * ch.sink_tiles + kt) * (ch.far + 1) * kBM + r) * 2 * p.D;
  const int64_t step = (int64_t)kBM * 2 * p.D;
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

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

int stat_tiles(const AttnParams& p) {
  const int tok = kBN / p.G;
  return (p.T + tok - 1) / tok;
}

size_t stat_bytes(const AttnParams& p) {
  return up256((size_t)p.B * p.Hkv * stat_tiles(p) * 2 * kBN * sizeof(float));
}

Chunks chunks_for(const AttnParams& p) {
  Chunks ch{};
  const int tok = kBN / p.G;
  ch.tiles = (p.T + kBM - 1) / kBM;
  const int ns = std::min((std::min(p.sinks, p.T) + kBM - 1) / kBM, ch.tiles);
  const int nq = stat_tiles(p);
  const int near = (int)((std::min<int64_t>(p.T, (int64_t)kBM - 1 + p.window) - 1) / tok) + 1;
  // Worth it where the part behind the window is longer than the part inside: a cut costs each chunk's block
  // its own K and V tile and the sum of the parts, and the longest walk is what the kernel ends with
  // (1537 tokens, window 200, groups of 3: 110 us uncut, 33 us cut).
  const int size = std::max(kMinChunk, near);
  if (ns > 0 && ns <= kMaxSinkTiles && nq - near > near) {
    ch.sink_tiles = ns;
    ch.size = size;
    ch.far = (nq - near + size - 1) / size;
  }
  return ch;
}

size_t part_bytes(const AttnParams& p, const Chunks& ch) {
  return up256((size_t)p.B * p.Hkv * ch.sink_tiles * (ch.sink_tiles ? ch.far + 1 : 0) * kBM * 2 * p.D * sizeof(float));
}

template <int DP, bool DQ>
cudaError_t launch_run(const Maps& maps, const AttnParams& p, const Chunks& ch, cudaStream_t stream) {
  cudaError_t e = set_smem_limit<attn_tc_backward_kernel<DP, DQ>>(Layout<DP>::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t pairs = (int64_t)p.B * p.Hkv;
  const int tok = kBM / p.G;
  const int ntiles = (p.T + tok - 1) / tok;
  const int64_t grid = DQ ? pairs * ntiles : pairs * (ch.tiles + (int64_t)ch.sink_tiles * ch.far);
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  attn_tc_backward_kernel<DP, DQ><<<(unsigned)grid, kThreads, Layout<DP>::kBytes, stream>>>(maps, p, ntiles, stat_tiles(p), ch);
  e = cudaGetLastError();
  if (e != cudaSuccess || DQ || !ch.sink_tiles) return e;
  const int sinks = std::min(p.sinks, p.T);
  sink_sum_kernel<<<(unsigned)((pairs * sinks + 7) / 8), 256, 0, stream>>>(p, ch, sinks);
  return cudaGetLastError();
}

}  // namespace

size_t attn_tc_backward_bytes(const AttnParams& p) { return stat_bytes(p) + part_bytes(p, chunks_for(p)); }

cudaError_t launch_attn_tc_backward(const AttnParams& params, void* workspace, cudaStream_t stream) {
  AttnParams p = params;
  p.delta = static_cast<float*>(workspace);
  Chunks ch = chunks_for(p);
  ch.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + stat_bytes(p));
  const int64_t rows = (int64_t)p.B * p.T * p.H;
  stat_kernel<<<(unsigned)((rows + kStatRows - 1) / kStatRows), 256, 0, stream>>>(p, rows, kBN / p.G, stat_tiles(p));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const uint64_t D = p.D, H = p.H, Hkv = p.Hkv, T = p.T, B = p.B;
  const std::array<uint64_t, 4> qd{D, H, T, B}, kd{D, Hkv, T, B};
  const std::array<uint64_t, 3> qs{D, H * D, T * H * D}, ks{D, Hkv * D, T * Hkv * D};
  auto q_map = [&](CUtensorMap* m, const void* x, int rows) {
    return make_map_bf16(m, x, qd, qs, {64, (uint32_t)p.G, (uint32_t)(rows / p.G), 1});
  };
  auto k_map = [&](CUtensorMap* m, const void* x, int rows) { return make_map_bf16(m, x, kd, ks, {64, 1, (uint32_t)rows, 1}); };
  Maps kv, dq;
  if (!k_map(&kv.a1, p.k, kBM) || !k_map(&kv.a2, p.v, kBM) || !q_map(&kv.b1, p.q, kBN) || !q_map(&kv.b2, p.dO, kBN) ||
      !q_map(&dq.a1, p.q, kBM) || !q_map(&dq.a2, p.dO, kBM) || !k_map(&dq.b1, p.k, kBN) || !k_map(&dq.b2, p.v, kBN))
    return cudaErrorInvalidValue;
  // (a result that is not wanted has a map that nothing is stored through)
  if (!k_map(&kv.g1, p.dv ? p.dv : p.v, kBM) || !k_map(&kv.g2, p.dk ? p.dk : p.k, kBM) ||
      !q_map(&dq.g2, p.dq ? p.dq : p.q, kBM))
    return cudaErrorInvalidValue;
  dq.g1 = dq.g2;
  if (p.dk || p.dv) e = p.D <= 64 ? launch_run<64, false>(kv, p, ch, stream) : launch_run<128, false>(kv, p, ch, stream);
  if (e == cudaSuccess && p.dq) e = p.D <= 64 ? launch_run<64, true>(dq, p, ch, stream) : launch_run<128, true>(dq, p, ch, stream);
  return e;
}

}  // namespace rsm
