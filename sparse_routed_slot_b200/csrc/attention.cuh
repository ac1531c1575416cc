// attention.cuh -- what the attention kernels share (window and paged, forward and backward).
//
// Every kernel works on one key/value head at a time and packs the G = H / Hkv query heads that
// share it into the rows of one tile: packed row r of a sequence is token r / G, head r % G of the
// group. K and V are then read once per group, and a tile of R rows spans only R / G tokens, so
// fewer keys at the window's edges are computed and thrown away.
//
// Key j is seen from place p when j <= p and (p - j < window or j < sinks). Keys are walked in
// tiles of `bn` places: first the tiles that hold sinks, then those of the window.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace rsm {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// One sequence as a kernel sees it.
struct Seq {
  int64_t row0;  // first new token among all q rows
  int nq;        // new tokens
  int kv;        // keys in the sequence
  int pos0;      // place of the first new token (may be negative: such rows see nothing)
};

RSM_DEV Seq sequence(const AttnParams& p, int b) {
  Seq s;
  if (!p.table) {
    s.row0 = (int64_t)b * p.T;
    s.nq = p.T;
    s.kv = p.T;
    s.pos0 = 0;
    return s;
  }
  // offsets and lengths come from device memory: clamped, so that no wrong value leaves the buffers
  const int N = p.T;
  const int c0 = min(max(p.cu_q[b], 0), N), c1 = min(max(p.cu_q[b + 1], c0), N);
  const int len = max(p.kv_len[b], 0);
  const int64_t cap = (int64_t)p.table_width * p.page;
  s.row0 = c0;
  s.nq = c1 - c0;
  s.pos0 = len - s.nq;
  s.kv = (int64_t)len > cap ? (int)cap : len;
  return s;
}

// The keys that some place of [p0, p1] sees: [0, sinks) and [lo, end). A paged kernel takes the places of all its
// sequence's rows, and neither looks up nor reads another key, though it share a tile with a seen one: behind the
// window a cache may have given its pages back.
struct Seen {
  int sinks, lo, end;
  RSM_DEV bool has(int key) const { return key < end && (key >= lo || key < sinks); }
  // any, or all, of the n keys from k0 on
  RSM_DEV bool any(int k0, int n) const { return k0 < end && (k0 + n > lo || k0 < sinks); }
  RSM_DEV bool all(int k0, int n) const { return k0 + n <= end && (k0 >= lo || k0 + n <= sinks); }
};

RSM_DEV Seen keys_seen(int p0, int p1, int kv, int window, int sinks) {
  return {sinks, window > 0 && p0 >= window ? p0 - window + 1 : 0, min(p1 + 1, kv)};
}

// The key tiles that places [p0, p1] may see (p1 >= p0), as a walk over n tiles: the first `ns`
// are tiles 0..ns-1 (sinks), the others follow from tile `first`.
struct Walk {
  int n, ns, first;
  RSM_DEV int tile(int i) const { return i < ns ? i : first + (i - ns); }
};

RSM_DEV Walk key_walk(int p0, int p1, int kv, int window, int sinks, int bn) {
  Walk w;
  const Seen seen = keys_seen(p0, p1, kv, window, sinks);
  if (seen.end <= 0) return {0, 0, 0};
  const int last = (seen.end - 1) / bn;
  const int s = min(sinks, seen.end);
  w.ns = s > 0 ? (s - 1) / bn + 1 : 0;
  w.first = max(w.ns, seen.lo / bn);
  w.n = w.ns + max(0, last - w.first + 1);
  return w;
}

// The tokens [t0, t1) of a sequence of T that may see a key of [k0, k1] (dense attention only:
// token t stands at place t).
RSM_DEV void query_range(int k0, int k1, int T, int window, int sinks, int& t0, int& t1) {
  t0 = k0;
  t1 = k0 < sinks || window <= 0 ? T : (int)min((int64_t)T, (int64_t)k1 + window);
}

RSM_DEV bool sees(int pos, int key, int window, int sinks) {
  return key <= pos && (window <= 0 || pos - key < window || key < sinks);
}

// Address of key/value row `key` of sequence b, head hk (element offset into k or v), or -1 when
// the page table entry lies outside the cache (reported once per read).
RSM_DEV int64_t kv_offset(const AttnParams& p, int b, int hk, int key) {
  if (!p.table) return (((int64_t)b * p.T + key) * p.Hkv + hk) * p.D;
  const int pg = p.table[(int64_t)b * p.table_width + key / p.page];
  if ((unsigned)pg >= (unsigned)p.num_pages) {
    raise_status(RSM_ERR_BAD_PAGE);
    return -1;
  }
  return (((int64_t)pg * p.page + key % p.page) * p.Hkv + hk) * p.D;
}

}  // namespace attn
}  // namespace rsm
