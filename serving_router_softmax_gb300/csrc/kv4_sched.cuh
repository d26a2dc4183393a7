// Work split of the kv4 attention kernels.
//
// Sequence s has `nb` row blocks per kv head (its new tokens times the query
// heads of a kv head, in blocks of RB rows) and its slots in tiles.  An item
// (head, row block) counts one unit per tile and `extra` units more for what it
// costs to begin and end one; all units in order are split evenly over the CTAs,
// so ragged lengths balance by themselves.  The lengths are device data: every
// CTA forms the running sum over the sequences itself.
#pragma once

#include "kv4.cuh"

namespace moe {
namespace kv4 {

struct SeqShape {
  int q0, nq, base, total;  // first query token, tokens, context slots, slots in all
};

// Sequence s as its arrays give it; one that does not fit (a negative or
// falling q_start, a length outside its table) counts as having no tokens.
__device__ __forceinline__ SeqShape seq_shape(const Cache& c, const int32_t* q_start, const int32_t* base, int T, int s,
                                              int32_t* bad) {
  const int a = q_start[s], b = q_start[s + 1], n = base[s];
  const long long cap = static_cast<long long>(c.width) << c.page_log2;
  SeqShape r{a, b - a, n, n + (b - a)};
  if (a < 0 || b < a || b > T || n < 0 || static_cast<long long>(n) + (b - a) > cap) {
    *bad = MOE_DEV_CAPACITY;
    r.q0 = r.nq = r.base = r.total = 0;
  }
  return r;
}

// Fills cum[0..S] with the units before each sequence (rows per token G, row
// blocks of RB, tiles of `tile` slots, `extra` units an item).  All threads of the block; ends with
// a barrier.  scratch: 32 long longs.
__device__ __forceinline__ void build_units(const Cache& c, const int32_t* q_start, const int32_t* base, int T, int G,
                                            int RB, int tile, int extra, long long* cum, long long* scratch, int32_t* dev_err,
                                            bool report) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, nw = (blockDim.x + 31) >> 5;
  long long carry = 0;
  int32_t bad = 0;
  for (int s0 = 0; s0 < c.S; s0 += blockDim.x) {
    const int s = s0 + tid;
    long long u = 0;
    if (s < c.S) {
      const SeqShape q = seq_shape(c, q_start, base, T, s, &bad);
      const long long nb = (static_cast<long long>(q.nq) * G + RB - 1) / RB;
      u = static_cast<long long>(c.Hkv) * nb * ((q.total + tile - 1) / tile + extra);
    }
    long long incl = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      incl += lane >= o ? v : 0;
    }
    if (lane == 31) scratch[wid] = incl;
    __syncthreads();
    long long before = carry, all = 0;
    for (int w = 0; w < nw; ++w) {
      before += w < wid ? scratch[w] : 0;
      all += scratch[w];
    }
    if (s < c.S) cum[s] = before + incl - u;
    carry += all;
    __syncthreads();
  }
  if (tid == 0) cum[c.S] = carry;
  if (bad && report) flag_error(dev_err, bad);
  __syncthreads();
}

// Even shares of the units: share i of n begins at unit total * i / n, rounded down, so that one division finds the
// share of a unit (kv4_weigh on 16 sequences of up to 16k slots takes 47.4 us on the device so, with the
// longer shares at the front 46.0).  In divisions of 32 bits, but for totals beyond them: one of 64 bits is a long stretch of cold code in
// every CTA's prologue.
struct Shares {
  long long total, each;
  int n, rest;
  __device__ __forceinline__ Shares(long long units, int shares) : total(units), n(shares) {
    each = units < (1ll << 32) ? static_cast<uint32_t>(units) / static_cast<uint32_t>(shares) : units / shares;
    rest = static_cast<int>(units - each * shares);
  }
  __device__ __forceinline__ long long begin(int i) const {  // n < 65536
    return each * i + static_cast<uint32_t>(rest) * static_cast<uint32_t>(i) / static_cast<uint32_t>(n);
  }
  // The share that has unit u.
  __device__ __forceinline__ int of(long long u) const {
    const unsigned long long x = static_cast<unsigned long long>(u + 1) * n - 1;
    return static_cast<int>(x < (1ull << 32) && total < (1ll << 32) ? static_cast<uint32_t>(x) / static_cast<uint32_t>(total)
                                                                     : x / total);
  }
};

// The sequence that unit u (below cum[S]) belongs to.
__device__ __forceinline__ int find_seq(const long long* cum, int S, long long u) {
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cum[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A position in the unit order: the item and its next tile.
struct Cursor {
  int s, h, rb, tile, nt, nb;  // nt: units of an item, the first of them its tiles
  SeqShape q;
};

__device__ __forceinline__ void cursor_seq(Cursor& k, const Cache& c, const int32_t* q_start, const int32_t* base, int T,
                                           int G, int RB, int tile, int extra) {
  int32_t bad = 0;
  k.q = seq_shape(c, q_start, base, T, k.s, &bad);
  k.nb = static_cast<int>((static_cast<long long>(k.q.nq) * G + RB - 1) / RB);
  k.nt = (k.q.total + tile - 1) / tile + extra;
}

// The position of unit u (below cum[S]).
__device__ __forceinline__ void cursor_at(Cursor& k, const Cache& c, const int32_t* q_start, const int32_t* base, int T,
                                          int G, int RB, int tile, int extra, const long long* cum, long long u) {
  k.s = find_seq(cum, c.S, u);
  cursor_seq(k, c, q_start, base, T, G, RB, tile, extra);
  const long long rem = u - cum[k.s];
  long long item;
  if (rem < (1ll << 31)) item = static_cast<uint32_t>(rem) / static_cast<uint32_t>(k.nt);
  else item = rem / k.nt;
  k.tile = static_cast<int>(rem - item * k.nt);
  if (item < (1ll << 31)) k.h = static_cast<int>(static_cast<uint32_t>(item) / static_cast<uint32_t>(k.nb));
  else k.h = static_cast<int>(item / k.nb);
  k.rb = static_cast<int>(item - static_cast<long long>(k.h) * k.nb);
}

// On to the next item; there is one (the caller counts units).
__device__ __forceinline__ void cursor_next(Cursor& k, const Cache& c, const int32_t* q_start, const int32_t* base, int T,
                                            int G, int RB, int tile, int extra, const long long* cum) {
  k.tile = 0;
  if (++k.rb < k.nb) return;
  k.rb = 0;
  if (++k.h < c.Hkv) return;
  k.h = 0;
  do ++k.s;
  while (k.s + 1 < c.S && cum[k.s + 1] == cum[k.s]);
  cursor_seq(k, c, q_start, base, T, G, RB, tile, extra);
}

}  // namespace kv4
}  // namespace moe
