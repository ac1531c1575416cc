// attn_tc.cu -- window and paged attention of bf16 inputs on the 5th-generation tensor cores.
//
// One block owns two tiles of 128 packed query rows (token, head of the group) of one key/value head
// and walks the keys they see in tiles of 64:
//   S = Q K^T            tcgen05.mma, both operands from shared memory, fp32 in TMEM
//   P = 2^(S' - m)       S' = scale log2(e) S; the row's thread reads S from TMEM and writes P back as
//                        bf16 over the same columns (the softmax weights are rounded here: the second
//                        product takes bf16, and half a step, 2^-9 of a weight, is what the bf16 outputs
//                        lose anyway)
//   O += P V             P from TMEM, V as the tile TMA wrote it (contracted over its rows), fp32 in TMEM
// The reference m of a row is its first tile's maximum and moves only when the running one has passed it by
// 2^32: fp32 sums and bf16 weights keep their relative precision at any scale, so O is next to never
// rescaled (at 2^8, a warp rescaled every fourth tile of 2048 random keys, at 1600 cycles).
// As the reference is not the row's maximum, the largest weight is rounded too. The dense form therefore
// divides by the sum of the rounded weights: what is left of their rounding in o is sum eta_j p_j (v_j - o),
// which vanishes with a single large weight. Divided by the unrounded sum, a peaked row kept eta v, and
// delta = dO . o carried it into ds, which is small there (window of 3 to 9 keys: dq off by 3.2e-3 of its norm
// instead of 2.6e-3). lse is the unrounded sum's. It costs 3 % (32768 tokens, 16 heads of 128: 609 -> 628 us). Nothing
// differentiates the paged form, which keeps the one sum.
//
// Each query tile has two S buffers, so that S of the next keys is there when the rows' threads finish
// with this one: the products, not the chain S -> P -> O -> S, set the pace (with one 128-key buffer per
// tile the chain took 6000 cycles per 128 keys and two query tiles, of which the tensor core was busy
// 2100). The two warps of a scheduler, one of each query tile, take turns at their exponentials: left
// alone they fall into step, and the special function units idle while both load and look for maxima.
// A step of 64 keys and two query tiles needs 1024 cycles of the special function units and 1280 of the
// tensor core (S of 64 keys runs at 3/4 rate, bound by its operands from shared memory) and takes 1950 (32768
// tokens, 16/4 heads of 128: from windows of 1024, 4096 and 8192 keys). A block takes 8000 to 10000 besides, to
// start, to drain and to write: one block per SM hides none of it.
// K and V tiles serve both query tiles.
//
// Warps: 0-3 and 4-7 the rows of tiles 0 and 1 (a thread per row), 8 copies (TMA), 9 and 10 the MMA issuers
// of tiles 0 and 1 (a wait in one does not hold the other's products back).
// TMEM columns: S (and P) buffers of tile t at 128 t and 128 t + 64, O at 256 + t DP.
// A paged cache is read page by page (page sizes that divide 64 or are multiples of it, from 8 on): a
// tile is 64 / page copies, of the pages that hold a key some row of the sequence sees. Rows of V that none sees
// are cleared before P multiplies them, so what the cache holds there does not matter.
#include <cuda.h>

#include <algorithm>

#include "attn_tc.cuh"

namespace rsm {

namespace {

using namespace attn;

constexpr int kBM = 128, kBN = 64;
constexpr int kThreads = 352;
constexpr int kCopyWarp = 8, kMmaWarp = 9;  // and kMmaWarp + 1
constexpr float kSlack = 32.f;  // how far (log2) the running maximum may pass the reference

struct Maps {
  CUtensorMap q, k, v, o, o_low;
};

template <int DP> struct Layout {
  static constexpr int kStages = 4;
  static constexpr int kQ = kBM * DP * 2, kTile = kBN * DP * 2;  // bytes of a query and of a key tile
  static constexpr int kOffK = 2 * kQ;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kBytes = kOffV + kStages * kTile + 1024;
  static_assert(kBytes <= 232448 - 1024, "shared memory budget");
};

// The steps of the block's walk [w0, w0 + n) in which one query tile sees the keys: [0, sinks) and [first, end).
struct Steps {
  int sinks, first, end;
  RSM_DEV bool operator()(int i) const { return i < end && (i >= first || i < sinks); }
  RSM_DEV int count() const {
    const int a = max(0, min(sinks, end));
    return a + max(0, end - max(a, first));
  }
};

RSM_DEV Steps steps_of(const Walk& all, int w0, int n, int p0, int p1, int kv, const AttnParams& p, bool any) {
  const Walk w = key_walk(p0, p1, kv, p.window, p.sinks, kBN);
  if (!any || w.n == 0) return {0, 0, 0};
  // step of the block's walk that has key tile x (the tiles of a query tile are tiles of the block)
  auto step = [&](int x) { return (x < all.ns ? x : all.ns + (x - all.first)) - w0; };
  Steps s;
  s.sinks = min(w.ns - w0, n);
  s.first = w.n > w.ns ? step(w.first) : n;
  s.end = min(n, w.n > w.ns ? step(w.first + (w.n - w.ns) - 1) + 1 : w.ns - w0);
  return s;
}

RSM_DEV void turn_wait(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
RSM_DEV void turn_pass(int id) { asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory"); }

template <int DP, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ Maps maps, const AttnParams p,
                                                              int tok_tile, int npairs) {
  using L = Layout<DP>;
  constexpr int NS = L::kStages;
  constexpr int kBlocks = DP / 64;  // 64-column blocks of a tile
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t q_full[2], full[NS], empty[NS], s_full[2][2], p_full[2][2], o_done[2], fin[2];
  __shared__ uint32_t bad_keys[NS];
  __shared__ uint32_t s_tbase;

  // the last query tiles see the most keys: they start first
  const int split = blockIdx.x % p.splits;
  const int item = blockIdx.x / p.splits;
  const int pair = npairs - 1 - item % npairs;
  const int hk = item / npairs % p.Hkv, b = item / npairs / p.Hkv;
  const Seq s = sequence(p, b);
  if (PAGED && s.kv != s.pos0 + s.nq && threadIdx.x == 0) raise_status(RSM_ERR_BAD_PAGE);
  const int nq = PAGED ? min(s.nq, p.max_q) : s.nq;
  const int tok0 = pair * 2 * tok_tile;
  if (tok0 >= nq) return;
  const int G = p.G, D = p.D;
  const int ntok0 = min(tok_tile, nq - tok0), ntok1 = max(0, min(tok_tile, nq - tok0 - tok_tile));
  const int pos0 = s.pos0 + tok0;
  const Walk walk = key_walk(pos0, pos0 + ntok0 + ntok1 - 1, s.kv, p.window, p.sinks, kBN);
  const int w0 = (int)((int64_t)walk.n * split / p.splits), w1 = (int)((int64_t)walk.n * (split + 1) / p.splits);
  const int n = w1 - w0;
  const Seen seen = keys_seen(s.pos0, s.pos0 + nq - 1, s.kv, p.window, p.sinks);
  const int ntiles = ntok1 > 0 ? 2 : 1;  // query tiles
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kMmaWarp) tc::tmem_alloc(&s_tbase, 512);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&q_full[i], 1);
      for (int u = 0; u < 2; ++u) {
        tc::mbar_init(&s_full[i][u], 1);
        tc::mbar_init(&p_full[i][u], 4);
      }
      tc::mbar_init(&o_done[i], 1);
      tc::mbar_init(&fin[i], 1);
    }
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], ntiles);
    }
    tc::fence_mbar_init();
  }
  tc::tmem_fence_before();
  __syncthreads();
  tc::tmem_fence_after();
  const uint32_t tb = s_tbase;

  if (warp == kCopyWarp) {
    // =========================================================================== copies
    if (lane == 0) {
      tc::tma_prefetch_desc(&maps.q);
      tc::tma_prefetch_desc(&maps.k);
      tc::tma_prefetch_desc(&maps.v);
      const uint32_t qbytes = (uint32_t)(tok_tile * G * 128 * kBlocks);
      for (int t = 0; t < ntiles; ++t) {
        tc::mbar_arrive_expect_tx(&q_full[t], qbytes);
        const int64_t tok = (PAGED ? s.row0 : 0) + tok0 + t * tok_tile;
        for (int c = 0; c < kBlocks; ++c)
          tc::tma_load_4d(sm + t * L::kQ + c * (kBM * 128), &maps.q, &q_full[t], 64 * c, hk * G, (int)tok,
                          PAGED ? 0 : b);
      }
    }
    __syncwarp();
    // Unit c of the ring: K of step c and V of step c - 2, which the issuers take up together.
    const int rows = PAGED ? min(p.page, kBN) : kBN;  // rows of one copy
    int page_id[3] = {0, 0, 0};                       // lane l: page l of the tiles of steps c, c - 1 and c - 2
    uint32_t wanted[3] = {0, 0, 0}, bad[3] = {0, 0, 0};
    int issued = 0;
#pragma unroll 1
    for (int c = 0; c < n + 2; ++c) {
      const int st = c % NS;
      page_id[2] = page_id[1]; page_id[1] = page_id[0];
      wanted[2] = wanted[1]; wanted[1] = wanted[0];
      bad[2] = bad[1]; bad[1] = bad[0];
      wanted[0] = c < n ? 1 : 0;
      if (PAGED && c < n) {
        const int key = walk.tile(w0 + c) * kBN + lane * rows;
        const bool in = lane * rows < kBN && seen.any(key, rows);
        if (in) page_id[0] = p.table[(int64_t)b * p.table_width + key / p.page];
        const bool usable = in && (unsigned)page_id[0] < (unsigned)p.num_pages;
        wanted[0] = __ballot_sync(kFull, usable);
        bad[0] = __ballot_sync(kFull, in && !usable);
        if (bad[0] && lane == 0) raise_status(RSM_ERR_BAD_PAGE);
      }
      if (c >= NS && !wait_warp(&empty[st], (c / NS - 1) & 1)) break;
      if (PAGED) {
        // bit g: the 8 keys from 8 g on stand in an unusable page
        const uint32_t bits = __ballot_sync(kFull, lane < kBN / 8 && ((bad[2] >> (8 * lane / rows)) & 1));
        if (lane == 0) bad_keys[st] = bits;
      }
      if (lane == 0)
        tc::mbar_arrive_expect_tx(&full[st], (uint32_t)(__popc(wanted[0]) + __popc(wanted[2])) * rows * 128 * kBlocks);
      __syncwarp();
      auto copy = [&](const CUtensorMap* map, unsigned char* dst, int step, uint32_t want, int id) {
        if ((want >> lane) & 1) {
          const int k0 = walk.tile(w0 + step) * kBN;
#pragma unroll
          for (int cb = 0; cb < kBlocks; ++cb) {
            if (PAGED)
              tc::tma_load_4d(dst + cb * (kBN * 128) + lane * rows * 128, map, &full[st], 64 * cb, hk,
                              p.page > kBN ? k0 % p.page : 0, id);
            else
              tc::tma_load_4d(dst + cb * (kBN * 128), map, &full[st], 64 * cb, hk, k0, b);
          }
        }
      };
      copy(&maps.v, sm + L::kOffV + st * L::kTile, c - 2, wanted[2], page_id[2]);
      copy(&maps.k, sm + L::kOffK + st * L::kTile, c, wanted[0], page_id[0]);
      __syncwarp();
      issued = c + 1;
    }
    // no copy may outlive the block, whatever became of its readers
    for (int c = max(0, issued - NS); c < issued; ++c) tc::mbar_wait(&full[c % NS], (c / NS) & 1);
    for (int t = 0; t < ntiles; ++t) tc::mbar_wait(&q_full[t], 0);
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    // =========================================================================== MMA issuers
    const int t = warp - kMmaWarp;
    constexpr uint32_t kIdS = tc::idesc_bf16(kBM, kBN, 0, 0), kIdO = tc::idesc_bf16(kBM, DP, 0, 1);
    const uint64_t dQ = tc::smem_desc(tc::smem_u32(sm + t * L::kQ), 16, 1024);
    const uint64_t dK = tc::smem_desc(tc::smem_u32(sm + L::kOffK), 16, 1024);
    // V: 64-column blocks 8 KB apart, groups of 8 keys 1 KB apart
    const uint64_t dV = tc::smem_desc(tc::smem_u32(sm + L::kOffV), kBN * 128, 1024);
    // K step j (16 columns) of a tile with R rows: 32 bytes inside a 64-column block, then the next block
    auto kstep = [](int R, int j) -> uint64_t { return (uint64_t)(((j >> 2) * (R * 128) + (j & 3) * 32) >> 4); };
    auto tile_at = [](int i) -> uint64_t { return (uint64_t)((i * L::kTile) >> 4); };
    const uint32_t cS = tb + t * 128, cO = tb + 256 + t * DP;
    const Steps act = steps_of(walk, w0, n, pos0 + t * tok_tile, pos0 + t * tok_tile + (t ? ntok1 : ntok0) - 1, s.kv, p,
                               t < ntiles);
    if (tc::elect_one()) {
      int ns = 0, np = 0;  // S and P V products issued
      bool ok = t < ntiles && n > 0 && wait_one(&q_full[t], 0);
#pragma unroll 1
      for (int c = 0; ok && c < n + 2; ++c) {
        const int st = c % NS;
        ok = wait_one(&full[st], (c / NS) & 1);
        if (!ok) break;
        if (c >= 2 && act(c - 2)) {
          ok = wait_one(&p_full[t][np & 1], (np >> 1) & 1);
          if (!ok) break;
          tc::tmem_fence_after();
          const uint64_t v = dV + tile_at(st);
#pragma unroll
          for (int j = 0; j < kBN / 16; ++j)
            tc::mma_bf16_ts(cO, cS + (np & 1) * kBN + 8 * j, v + (uint64_t)(j * 2048 >> 4), kIdO, np > 0 || j > 0);
          tc::mma_commit(&o_done[t]);
          ++np;
        }
        if (c < n && act(c)) {
          // into buffer ns & 1, over weights whose product was issued before: one thread's MMAs run in order
          const uint64_t k = dK + tile_at(st);
#pragma unroll
          for (int j = 0; j < DP / 16; ++j)
            tc::mma_bf16_ss(cS + (ns & 1) * kBN, dQ + kstep(kBM, j), k + kstep(kBN, j), kIdS, j > 0);
          tc::mma_commit(&s_full[t][ns & 1]);
          ++ns;
        }
        tc::mma_commit(&empty[st]);  // (at once where nothing was issued)
      }
      tc::mma_commit(&fin[t]);
    }
    __syncwarp();
    tc::mbar_wait(&fin[t], 0);  // every MMA issued is done before the block gives up its memory
  } else if (warp < kCopyWarp) {
    // =========================================================================== rows
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;
    const int ntok = t ? ntok1 : ntok0;
    const Steps act = steps_of(walk, w0, n, pos0 + t * tok_tile, pos0 + t * tok_tile + ntok - 1, s.kv, p, ntok > 0);
    const int tok = tok0 + t * tok_tile + r / G;
    const int pos = s.pos0 + tok;
    const int pmin = s.pos0 + tok0 + t * tok_tile, pmax = pmin + ntok - 1;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32);
    const uint32_t tS = tc::tmem_addr(tb, lane_base, t * 128), tO = tc::tmem_addr(tb, lane_base, 256 + t * DP);
    const float scale2 = p.scale * kLog2e;
    float m = kNegInf, l = 0.f, lr = 0.f;  // sums of the weights, and of the rounded ones
    int done = 0;
    bool ok = true;
    // The warps of both tiles that share a scheduler form their weights in turn: see above.
    const Steps other = steps_of(walk, w0, n, pos0 + (1 - t) * tok_tile, pos0 + (1 - t) * tok_tile + (t ? ntok0 : ntok1) - 1,
                                 s.kv, p, t || ntiles > 1);
    const int theirs = other.count();
    const int my_turn = 1 + 2 * (warp & 3) + t, their_turn = 1 + 2 * (warp & 3) + 1 - t;
    // Scores of step i into x (hidden ones -inf), and the row's reference moved where it has to. False: a wait expired.
    auto look = [&](int i, int k0, bool there, uint32_t tP, float (&x)[kBN]) {
      if (!there && !wait_warp(&s_full[t][done & 1], (done >> 1) & 1)) return false;
      tc::tmem_fence_after();
      tc::tmem_ld32(tP, *reinterpret_cast<float(*)[32]>(&x[0]));
      tc::tmem_ld32(tP + 32, *reinterpret_cast<float(*)[32]>(&x[32]));
      uint32_t bad = 0;
      if (PAGED) {
        // the list of unusable pages travels with the V tile
        if (!wait_warp(&full[(i + 2) % NS], ((i + 2) / NS) & 1)) return false;
        bad = *(volatile uint32_t*)&bad_keys[(i + 2) % NS];
      }
      tc::tmem_wait_ld();
      const bool whole = k0 + kBN - 1 <= min(pmin, s.kv - 1) &&
                         (p.window <= 0 || pmax - k0 < p.window || k0 + kBN - 1 < p.sinks) && !bad;
      if (!whole) {
        // columns [0, sk) and [lo, hi] are seen
        const int hi = min(pos, s.kv - 1) - k0;
        const int lo = p.window > 0 ? pos - p.window + 1 - k0 : 0;
        const int sk = min(p.sinks - k0, hi + 1);
#pragma unroll
        for (int c = 0; c < kBN; c += 32) {
          uint32_t w = (below(hi + 1 - c) & ~below(lo - c)) | below(sk - c);
          if (PAGED) {
            const uint32_t g = bad >> (c / 8);
            w &= ~((g & 1 ? 0xffu : 0u) | (g & 2 ? 0xff00u : 0u) | (g & 4 ? 0xff0000u : 0u) | (g & 8 ? 0xff000000u : 0u));
          }
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(w & (1u << e))) x[c + e] = kNegInf;
        }
        // (a tile with a key that no row of the sequence sees is whole for none)
        if (PAGED && (bad || !seen.all(k0, kBN))) {
          // key r of the tile: its V row is cleared where there is no such key, or nothing sees it
          if (r < kBN && (!seen.has(k0 + r) || ((bad >> (r / 8)) & 1))) {
            unsigned char* v = sm + L::kOffV + ((i + 2) % NS) * L::kTile + r * 128;
#pragma unroll
            for (int c = 0; c < kBlocks; ++c)
#pragma unroll
              for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4*>(v + c * (kBN * 128) + e * 16) = make_uint4(0, 0, 0, 0);
          }
          tc::fence_async_smem();
        }
      }
      float top4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int c = 4; c < kBN - 4; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) top4[e] = max3(top4[e], x[c + e], x[c + e + 4]);
#pragma unroll
      for (int e = 0; e < 4; ++e) top4[e] = fmaxf(top4[e], x[kBN - 4 + e]);
      const float top = fmaxf(max3(top4[0], top4[1], top4[2]), top4[3]) * scale2;
      const bool move = done == 0 || top > m + kSlack;
      // (a row that has seen nothing yet has nothing to rescale)
      if (__any_sync(kFull, move && m != kNegInf)) {
        // O is this warp's once the last product into it is done. (The next one takes this warp's weights, so
        // the parity names one phase.) Not once that product's unit is let go of, which takes the other tile's
        // issuer as well: with one query head per key/value head the other tile can be two steps ahead, and its
        // rows wait for the turn that this warp holds.
        if (!wait_warp(&o_done[t], (done - 1) & 1)) return false;
        tc::tmem_fence_after();
        const float f = move ? ex2(m - top) : 1.f;
        l *= f;
        lr *= f;
#pragma unroll 1
        for (int c = 0; c < DP; c += 16) {
          float o[16];
          tc::tmem_ld16(tO + c, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] *= f;
          tc::tmem_st16(tO + c, o);
        }
      }
      if (move) m = top;
      return true;
    };
    int i = 0;
    while (i < n && !act(i)) ++i;
    int k0 = walk.tile(w0 + i) * kBN;
    bool there = false;  // S of step i is known to be ready
#pragma unroll 1
    while (i < n) {
      const uint32_t tP = tS + (done & 1) * kBN;
      float x[kBN];
      ok = ok && look(i, k0, there, tP, x);
      int next = i + 1;
      while (next < n && !act(next)) ++next;
      const int k0_next = walk.tile(w0 + next) * kBN;
      // (a warp whose wait expired still takes and passes its turns: the other one is not left waiting)
      if (t ? done < theirs : done > 0 && done <= theirs) turn_wait(my_turn);
      // asked here, so that the answer comes while the exponentials run
      const bool ready = tc::mbar_test(&s_full[t][(done + 1) & 1], ((done + 1) >> 1) & 1);
      if (ok) {
        const float ref = m == kNegInf ? 0.f : m;
        const float2 s2 = make_float2(scale2, scale2), r2 = make_float2(-ref, -ref);
        float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0, low0 = sum0, low1 = sum0;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          float w[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float2 e = fma2(make_float2(x[16 * h + 2 * c], x[16 * h + 2 * c + 1]), s2, r2);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            if (c & 1) sum1 = add2(sum1, e);
            else sum0 = add2(sum0, e);
            const uint32_t u = pack_bf16(e.x, e.y);
            if (!PAGED) {
              const float2 rounded = make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
              if (c & 1) low1 = add2(low1, rounded);
              else low0 = add2(low0, rounded);
            }
            w[c] = __uint_as_float(u);
          }
          tc::tmem_st8(tP + 8 * h, w);
        }
        l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
        lr += (low0.x + low0.y) + (low1.x + low1.y);
      }
      if (t ? done + 1 < theirs : done < theirs) turn_pass(their_turn);
      if (ok) {
        tc::tmem_wait_st();
        tc::tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t][done & 1]);
      }
      there = __all_sync(kFull, ready);
      ++done;
      i = next;
      k0 = k0_next;
    }
    if (ok && done > 0) {
      ok = wait_warp(&fin[t], 0);
      tc::tmem_fence_after();
    }
    const bool live = r < ntok * G;
    const int64_t at = (s.row0 + tok) * p.H + hk * G + r % G;
    const int64_t total = (int64_t)p.T * (PAGED ? 1 : p.B) * p.H;
    const float by = PAGED ? l : lr;
    const float inv = by > 0.f ? 1.f / by : by == 0.f ? 0.f : by;  // (a NaN stays one)
    // Whole tiles go through the query tile's memory, which is done with, to a tensor store; so does the last
    // tile of a dense sequence, whose rows behind the end the store leaves out. Behind the end of a paged one
    // stand the next sequence's rows.
    if (p.splits == 1 && done > 0 && (!PAGED || ntok == tok_tile)) {
      unsigned char* to = sm + t * L::kQ;
      if (ok) stage_row<DP>(to, r, 0, tO, inv);
      tc::fence_async_smem();
      group_sync(9 + t, 128);
      if (ok && r == 0) {
        const int64_t first = (PAGED ? s.row0 : 0) + tok0 + t * tok_tile;
        for (int c = 0; c < kBlocks; ++c)
          tc::tma_store_4d(&maps.o, to + c * (kBM * 128), 64 * c, hk * G, (int)first, PAGED ? 0 : b);
        tc::bulk_commit_group();
        tc::bulk_wait_read_all();
      }
      if (!PAGED && p.o_low) {
        group_sync(9 + t, 128);  // the tile is read out
        if (ok) stage_row_low<DP>(to, r, tO, inv);
        tc::fence_async_smem();
        group_sync(9 + t, 128);
        if (ok && r == 0) {
          for (int c = 0; c < kBlocks; ++c)
            tc::tma_store_4d(&maps.o_low, to + c * (kBM * 128), 64 * c, hk * G, tok0 + t * tok_tile, b);
          tc::bulk_commit_group();
          tc::bulk_wait_read_all();
        }
      }
    } else if (ok && ntok > 0) {
#pragma unroll 1
      for (int c = 0; c < DP; c += 32) {
        float o[32];
        if (done > 0) {
          tc::tmem_ld32(tO + c, o);
          tc::tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = done > 0 && l != 0.f ? o[e] * inv : 0.f;
        if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            if (c + e < D) {
              if (p.splits > 1) {
                float* to = p.part_o + (split * total + at) * D + c + e;
                *reinterpret_cast<float4*>(to) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                *reinterpret_cast<float4*>(to + 4) = make_float4(o[e + 4], o[e + 5], o[e + 6], o[e + 7]);
              } else {
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + at * D + c + e) =
                    make_uint4(pack_bf16(o[e], o[e + 1]), pack_bf16(o[e + 2], o[e + 3]), pack_bf16(o[e + 4], o[e + 5]),
                               pack_bf16(o[e + 6], o[e + 7]));
              }
            }
          }
        }
      }
    }
    if (ok && live) {
      const float lse = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
      if (p.splits > 1) p.part_lse[split * total + at] = lse;
      else if (p.lse) p.lse[at] = lse;
    }
  }
  tc::tmem_fence_before();
  __syncthreads();
  tc::tmem_fence_after();
  if (warp == kMmaWarp) tc::tmem_dealloc(tb, 512);
}

int token_tile(const AttnParams& p) { return kBM / p.G; }

int64_t blocks_without_splits(const AttnParams& p) {
  const int64_t nq = p.table ? p.max_q : p.T;
  const int64_t per = 2 * token_tile(p);
  return (nq + per - 1) / per * p.Hkv * p.B;
}

template <int DP, bool PAGED>
cudaError_t launch_dp(const Maps& maps, const AttnParams& p, cudaStream_t stream) {
  cudaError_t e = set_smem_limit<attn_tc_kernel<DP, PAGED>>(Layout<DP>::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t blocks = blocks_without_splits(p);
  if (blocks * p.splits > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int npairs = (int)(blocks / ((int64_t)p.Hkv * p.B));
  attn_tc_kernel<DP, PAGED><<<(unsigned)(blocks * p.splits), kThreads, Layout<DP>::kBytes, stream>>>(maps, p, token_tile(p), npairs);
  return cudaGetLastError();
}

}  // namespace

bool attn_tc_supported(const AttnParams& p, rsm_dtype dtype) {
  if (dtype != RSM_BF16 || p.D > 128) return false;
  if (!p.table) return true;
  return p.num_pages > 0 && p.table_width > 0 && p.page % 8 == 0 && (kBN % p.page == 0 || p.page % kBN == 0);
}

// Blocks that share a row's keys: where the rows alone leave SMs idle, as many as fill them once, of at
// least four key tiles each by the table's width. Not more, to even out sequences of unequal length: with 128
// blocks of 4 x 512 tokens over 24181, 20657, 28506 and 31917 keys, 4 splits take 503 us against 525, but over
// equal 32768 keys 604 to 635 against 544 to 563, and over 2000 keys 100 against 47 (the join of the fp32 parts).
int attn_tc_splits(const AttnParams& p) {
  if (!p.table) return 1;
  int64_t keys = (int64_t)p.table_width * p.page;
  if (p.window > 0) keys = std::min<int64_t>(keys, (int64_t)p.window + p.sinks + p.max_q);
  const int64_t tiles = (keys + kBN - 1) / kBN;
  const int64_t want = device_sm_count() / std::max<int64_t>(1, blocks_without_splits(p));
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, tiles / 4, 64}));
}

cudaError_t launch_attn_tc(const AttnParams& p, cudaStream_t stream) {
  Maps maps;
  const uint64_t D = p.D, H = p.H, Hkv = p.Hkv;
  const bool paged = p.table != nullptr;
  const uint64_t T = p.T, B = paged ? 1 : p.B;
  const int tok = token_tile(p);
  bool ok = true;
  // (without o_low nothing is stored through its map)
  for (auto [m, base] : {std::pair<CUtensorMap*, const void*>{&maps.q, p.q}, {&maps.o, p.o},
                         {&maps.o_low, p.o_low ? p.o_low : p.o}})
    ok = ok && make_map_bf16(m, base, {D, H, T, B}, {D, H * D, T * H * D}, {64, (uint32_t)p.G, (uint32_t)tok, 1});
  if (paged) {
    const uint64_t page = p.page, pages = p.num_pages;
    const uint32_t rows = (uint32_t)std::min(p.page, kBN);
    for (auto [m, base] : {std::pair<CUtensorMap*, const void*>{&maps.k, p.k}, {&maps.v, p.v}})
      ok = ok && make_map_bf16(m, base, {D, Hkv, page, pages}, {D, Hkv * D, page * Hkv * D}, {64, 1, rows, 1});
  } else {
    for (auto [m, base] : {std::pair<CUtensorMap*, const void*>{&maps.k, p.k}, {&maps.v, p.v}})
      ok = ok && make_map_bf16(m, base, {D, Hkv, T, B}, {D, Hkv * D, T * Hkv * D}, {64, 1, (uint32_t)kBN, 1});
  }
  if (!ok) return cudaErrorInvalidValue;
  if (p.D <= 64) return paged ? launch_dp<64, true>(maps, p, stream) : launch_dp<64, false>(maps, p, stream);
  return paged ? launch_dp<128, true>(maps, p, stream) : launch_dp<128, false>(maps, p, stream);
}

}  // namespace rsm
