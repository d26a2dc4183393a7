// moe_prompt_attend: causal attention of packed prompts on the 5th-generation
// tensor cores.
//
// A CTA takes 256 query rows of one kv head, as two tiles of 128: the G query
// heads of floor(128 / G) tokens each, token by token, so that any number of
// heads fills the tiles and the heads share their keys.  Per 128 keys and tile:
//   S [128 x 128] = Q K^T           operands in shared memory, sums in TMEM
//   P = exp2(c S - r), l += row sums    a thread per row, P in TMEM as bf16
//   O [128 x D] += P V              P from TMEM, V as it lies ([keys][D])
// One tile's products run while the other's exponentials do.  At D = 64 TMEM has
// room for P beside S, and the next step's S is made while this one's exponentials
// run; at D = 128 P lies over S, and a step is a chain: S, exponentials, P V.
//
// The reference r of a row's exponentials need not be its maximum: any r gives
// the same quotient O / l.  It moves (and O and l are scaled to it) only when a
// score passes it by more than 8, so that powers stay below 2^8 and O is
// rewritten in a few steps of a row instead of all; bf16 and fp32 are as good
// anywhere in that range.  r is a product rounded to fp32, the exponents c S - r are
// not: past 2^31 the rounding alone takes P out of fp32's range, and such a row is NaN.
//
// Persistent, one CTA an SM: an item (such a block of a sequence and kv head)
// begins while the one before it ends, since a block's own beginning and end
// (13 us of launch, set-up, first loads and output) are longer than a short
// prompt's products.  Blocks of a sequence differ in work by their place in it;
// they are taken in falling order of it over all sequences, back and forth over
// the CTAs.  Rank x among the items is found by counting, with no plan in memory:
// F(b) = sum of max(0, blocks - b) items lie at block b of their sequence or later.
//
// What a row may not see: scores are replaced by -inf in the tiles that hold
// any; values there that are not finite would make 0 * v a NaN, so a warp looks
// through those value tiles, puts zeros in their place, and keeps for each
// dimension the first such key, which makes the output of the rows that see it
// NaN.
//
// Roles (512 threads): warps 0-3 and 4-7 softmax and output of a tile each, warps 8
// and 9 issue a tile's products each (the tensor core takes a product as it begins
// it, so one warp's waits and signals for both tiles, 1900 cycles a step, were not
// hidden by the 2050 of its products; at D = 64 warps 10 and 11 issue those with V),
// warp 12 loads by TMA, warp 13 looks at values, warp 14 finds the items, a few ahead.
// Every wait is bounded.
//
// Bound by a step's chain: at D = 128 some 3050 cycles, 2050 of them products of the
// two tiles, which take turns; at D = 64 2600 against 1110.  2 prompts of up to 12,001
// tokens, 32 query heads on 8, D 128: 1.28 ms, 1590 TFLOP/s; 24 ragged ones of up to
// 1500, 64 heads on 4: 0.36 ms, 1060; one of 8192, 32 on 8, D 64: 0.30 ms, 920.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "apart.cuh"
#include "kv4.cuh"
#include "tc_f16.cuh"
#include "tc_pair.cuh"

namespace moe {
namespace {

using tc::add2;
using tc::fma2;
using tc::mul2;

constexpr int kThreads = 512;
constexpr int kRows = 128;       // query rows of a tile, keys of a step
constexpr int kPanel = kRows * 128;  // bytes of 64 dimensions of a tile
constexpr float kSlack = 8.f;
constexpr float kFar = 2147483648.f;  // references from here on, either way: half a last place is 128 powers of two
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kMaxSeqs = 2048;
constexpr int kItems = 4;        // items found ahead

struct PromptArgs {
  const int32_t* start;
  uint16_t* out;
  float* lse;
  int32_t* dev_err;
  int T, S, Hq, Hkv, G, tokens;  // tokens: of a tile
  float c;                       // |scale| log2(e)
  int negative, wide, stall;     // scale < 0; out a multiple of 32 bytes; test hook
};

struct Item {
  int begin, len;  // the sequence: first row, rows
  int first;       // first token of the item, counted in the sequence
  int head;        // kv head
  int n[2];        // steps of each tile; n[0] < 0: no more items
};

template <int D>
struct Smem {
  static constexpr int kStages = D == 128 ? 4 : 8;
  alignas(1024) uint8_t q[2][D / 64][kPanel];
  alignas(1024) uint8_t kv[kStages][D / 64][kPanel];
  int blocks[kMaxSeqs], begin[kMaxSeqs], len[kMaxSeqs];  // of each sequence
  uint64_t full[kStages], empty[kStages], v_ok[kStages];
  uint64_t q_full[2], q_empty[2], s_full[2], s_read[2], p_full[2], pv_done[2], o_full[2], o_empty[2], item_full[kItems], item_empty[kItems], drain;
  Item item[kItems];
  int first_bad[kItems][D], bad[kItems];
  int most;
  uint32_t tmem;
  int abort, issuing;
};
template <int D>
constexpr size_t kSmemBytes = sizeof(Smem<D>) + 1024;
static_assert(kSmemBytes<128> <= 227 * 1024 && kSmemBytes<64> <= 227 * 1024, "shared memory");

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float2* e) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(e[0].x), "=f"(e[0].y), "=f"(e[1].x), "=f"(e[1].y), "=f"(e[2].x), "=f"(e[2].y), "=f"(e[3].x), "=f"(e[3].y),
        "=f"(e[4].x), "=f"(e[4].y), "=f"(e[5].x), "=f"(e[5].y), "=f"(e[6].x), "=f"(e[6].y), "=f"(e[7].x), "=f"(e[7].y),
        "=f"(e[8].x), "=f"(e[8].y), "=f"(e[9].x), "=f"(e[9].y), "=f"(e[10].x), "=f"(e[10].y), "=f"(e[11].x),
        "=f"(e[11].y), "=f"(e[12].x), "=f"(e[12].y), "=f"(e[13].x), "=f"(e[13].y), "=f"(e[14].x), "=f"(e[14].y),
        "=f"(e[15].x), "=f"(e[15].y)
      : "r"(taddr));
}
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// 32 bytes; `wide`: to an address that is a multiple of them.
__device__ __forceinline__ void store32(uint16_t* at, const uint32_t (&w)[8], int wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                 "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(at + 8) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Units u (bit kBit clear) and u + kBit of the four lanes of a quad: the lane whose number has the bit keeps u + kBit and takes the
// other lane's, the other one the lower ones.  With both bits, unit k of lane g is what was unit g of lane k.
template <int kBit>
__device__ __forceinline__ void turn4(uint32_t (&w)[4][8], int lane) {
  const bool high = lane & kBit;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (u & kBit) continue;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, high ? w[u][x] : w[u + kBit][x], kBit);
      if (high)
        w[u][x] = got;
      else
        w[u + kBit][x] = got;
    }
  }
}

// D[tmem] (+)= A[tmem] * B[smem], bf16.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  tc::mma_f16_ts(d, a, b, idesc, accumulate);
}
// V as the second operand: 64 dimensions side by side in a 128-byte row per key, 8 keys an atom of 1024 bytes, panels of 64
// dimensions kPanel bytes apart (the leading offset); the product's N goes along the row (bit 16 of the instruction).
__device__ __forceinline__ uint64_t value_desc(uint32_t addr) {
  return tc::smem_desc_sw128(addr) ^ (1ull << 16) ^ (static_cast<uint64_t>(kPanel >> 4) << 16);
}
constexpr uint32_t kValuesAlongN = 1u << 16, kNegateA = 1u << 13;

// Finds items by their rank: a warp's work.
struct Finder {
  const PromptArgs& a;
  const int *blocks, *begin, *len;
  int top;  // a level that no later rank lies above

  // F(b).
  __device__ __forceinline__ int at_or_above(int b, int lane) const {
    int v = 0;
    for (int s = lane; s < a.S; s += 32) v += max(0, blocks[s] - b);
    return __reduce_add_sync(0xFFFFFFFFu, v);
  }
  __device__ __forceinline__ bool find(int rank, Item* it, int lane) {
    const int r = rank / a.Hkv;
    if (r >= at_or_above(0, lane)) return false;
    // The last level lo with F(lo) > r.
    int lo = 0, hi = top, above = 0;  // F(hi) <= r: 0, or counted
    while (hi - lo > 1) {
      const int b = lo + (hi - lo) / 2, v = at_or_above(b, lane);
      if (v > r)
        lo = b;
      else
        hi = b, above = v;
    }
    if (hi == top) above = at_or_above(hi, lane);
    // The (r - F(lo + 1))-th sequence that has a block lo.
    int skip = r - above, seq = 0;
    for (int s0 = 0; s0 < a.S; s0 += 32) {
      const int s = s0 + lane;
      const uint32_t has = __ballot_sync(0xFFFFFFFFu, s < a.S && blocks[s] > lo);
      const int n = __popc(has);
      if (skip < n) {
        const bool me = ((has >> lane) & 1) && __popc(has & ((1u << lane) - 1)) == skip;
        seq = s0 + __ffs(__ballot_sync(0xFFFFFFFFu, me)) - 1;
        break;
      }
      skip -= n;
    }
    it->begin = begin[seq], it->len = len[seq];
    it->first = lo * 2 * a.tokens;
    it->head = rank - r * a.Hkv;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int from = it->first + t * a.tokens;  // a tile's last token sees itself
      it->n[t] = from >= it->len ? 0 : (min(from + a.tokens, it->len) + kRows - 1) / kRows;
    }
    return true;
  }
};

// Keys that tile t's last token sees.
__device__ __forceinline__ int seen_by(const PromptArgs& a, const Item& it, int t) { return min(it.first + (t + 1) * a.tokens, it.len); }

// acc += 0 * x, on two bf16.
__device__ __forceinline__ void zero_times(uint32_t& acc, uint32_t x) {
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
}

// A tile's products are issued as a block: taken from two warps one by one in turn, both tiles' blocks take twice as long, end
// together, and the tiles' exponentials then run at the same time as well (418 instead of 354 us for 24 ragged prompts).
// Only the order depends on it, so who waits too long goes ahead.
__device__ __forceinline__ void issue_alone(int* issuing) {
  for (int n = 0; n < (1 << 20) && atomicCAS(issuing, 0, 1); ++n) {
  }
}
__device__ __forceinline__ void issue_done(int* issuing) { atomicExch(issuing, 0); }

// A role's place in the ring of items.
struct Turn {
  int i = 0;
  __device__ __forceinline__ int slot() const { return i % kItems; }
  __device__ __forceinline__ uint32_t parity() const { return (i / kItems) & 1; }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const PromptArgs a) {
  using Sm = Smem<D>;
  constexpr int NS = Sm::kStages, P = D / 64;
  constexpr bool kApart = D == 64;  // P beside S
  // TMEM columns: S of both tiles, P (beside or over it), O.
  constexpr int kPCol = kApart ? 256 : 0, kPStep = kApart ? 64 : 128, kOCol = kApart ? 384 : 256;
  extern __shared__ uint8_t raw[];
  Sm& sm = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) tc::mbar_init(&sm.full[i], 1), tc::mbar_init(&sm.empty[i], 2), tc::mbar_init(&sm.v_ok[i], 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.q_full[i], 1), tc::mbar_init(&sm.q_empty[i], 1);
      tc::mbar_init(&sm.s_full[i], 1), tc::mbar_init(&sm.s_read[i], 4), tc::mbar_init(&sm.pv_done[i], 1);
      tc::mbar_init(&sm.p_full[i], 4);
      tc::mbar_init(&sm.o_full[i], 1), tc::mbar_init(&sm.o_empty[i], 4);
    }
    for (int i = 0; i < kItems; ++i) {
      tc::mbar_init(&sm.item_full[i], 1), tc::mbar_init(&sm.item_empty[i], kApart ? 14 : 12);  // softmax, products, loads, values
      sm.bad[i] = 0;
    }
    tc::mbar_init(&sm.drain, kApart ? 4 : 2);
    sm.abort = sm.most = sm.issuing = 0;
    tc::fence_mbar_init();
  }
  for (int d = tid; d < kItems * D; d += kThreads) (&sm.first_bad[0][0])[d] = 0x7FFFFFFF;
  if (warp == 8) {
    tc::tmem_alloc(&sm.tmem, 512);
    tc::tmem_relinquish();
  }
  const int per = 2 * a.tokens;
  int most = 0, out_of_order = 0;
  for (int s = tid; s < a.S; s += kThreads) {
    const int b = a.start[s], e = a.start[s + 1];
    const bool wrong = b < 0 || e > a.T || b > e;
    out_of_order |= wrong;
    const int n = wrong ? 0 : (e - b + per - 1) / per;
    sm.blocks[s] = n, sm.begin[s] = b, sm.len[s] = e - b;
    most = max(most, n);
  }
  tc::tc_fence_before();
  out_of_order = __syncthreads_or(out_of_order);
  tc::tc_fence_after();
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (lane == 0 && most > 0) atomicMax(&sm.most, most);
  __syncthreads();
  if (out_of_order && blockIdx.x == 0 && tid == 0) flag_error(a.dev_err, MOE_DEV_CAPACITY);
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sm.tmem, 0);
  volatile int* gave_up = &sm.abort;
  bool ok = true;
  Turn turn;
  // The next item, for the roles that are told of it.
  auto next_item = [&]() -> Item {
    ok = tc::mbar_sleep<true>(&sm.item_full[turn.slot()], turn.parity(), gave_up, kWaitNs);
    Item it = sm.item[turn.slot()];
    if (!ok) it.n[0] = -1;
    return it;
  };
  auto item_done = [&] {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sm.item_empty[turn.slot()]);
    ++turn.i;
  };

  if (warp < 8) {
    // ---------------------------------------------------------- softmax, output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int t = warp >> 2, r = (warp & 3) * 32 + lane, tok = r / a.G, in_group = r % a.G;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + t * 128, tp = tmem + lanes + kPCol + t * kPStep, to = tmem + lanes + kOCol + t * D;
    const float2 c2 = make_float2(a.c, a.c);
    int step = 0, items = 0;  // of this tile
    while (true) {
      const Item it = next_item();
      if (it.n[0] < 0) break;
      const int steps = t ? it.n[1] : it.n[0];
      if (steps == 0) {
        item_done();
        continue;
      }
      const int from = it.first + t * a.tokens, pos = from + tok;
      const bool real = tok < a.tokens && pos < it.len;
      const int limit = real ? pos + 1 : 0;  // keys that the row sees
      float ref = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f), k2 = make_float2(0.f, 0.f);
      for (int j = 0; j < steps; ++j, ++step) {
        ok = tc::mbar_sleep<true>(&sm.s_full[t], step & 1, gave_up, kWaitNs);
        if (!ok) break;
        tc::tc_fence_after();
        float2 s[64];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, s + 16 * i);
        tc::tmem_ld_wait();
        if (kApart) {
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.s_read[t]);
        }
        if ((j + 1) * kRows > from + 1) {
          // (Code that runs once an item comes from far: only the groups of 32 keys that some row does not see.)
          const int see = limit - j * kRows;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            if (__all_sync(0xFFFFFFFFu, see >= 32 * g + 32)) continue;
#pragma unroll
            for (int i = 16 * g; i < 16 * g + 16; ++i) {
              s[i].x = 2 * i < see ? s[i].x : -INFINITY;
              s[i].y = 2 * i + 1 < see ? s[i].y : -INFINITY;
            }
          }
        }
        float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 64; ++i) m[i & 3] = kv4::max3(m[i & 3], s[i].x, s[i].y);
        const float top = fmaxf(kv4::max3(m[0], m[1], m[2]), m[3]) * a.c;
        const bool move = top > ref + kSlack;
        if (kApart && j > 0) {  // the products of the step before (D = 128: the scores came after them)
          ok = tc::mbar_sleep<true>(&sm.pv_done[t], (step - 1) & 1, gave_up, kWaitNs);
          if (!ok) break;
          tc::tc_fence_after();
        }
        if (__any_sync(0xFFFFFFFFu, move)) {
          const float f = move ? kv4::ex2(ref - top) : 1.f;  // (0 from -inf)
          if (move) ref = top;
          const float2 f2 = make_float2(f, f);
          l2 = mul2(l2, f2), k2 = mul2(k2, f2);
          if (j > 0) {
#pragma unroll 1
            for (int i = 0; i < D; i += 16) {
              float o[16];
              tc::tmem_ld16(to + i, o);
              tc::tmem_ld_wait();
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * f);
              tc::tmem_st16(to + i, w);
            }
          }
        }
        const float neg = ref <= -kFar ? 0.f : -ref;  // (P is then 0)
        const float2 r2 = make_float2(neg, neg);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 x = fma2(s[16 * i + e], c2, r2);
            x.x = kv4::ex2(x.x), x.y = kv4::ex2(x.y);
            if (e & 1)
              k2 = add2(k2, x);
            else
              l2 = add2(l2, x);
            w[e] = pack_bf(x.x, x.y);
          }
          tc::tmem_st16(tp + 16 * i, w);
        }
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.p_full[t]);
      }
      if (ok) ok = tc::mbar_sleep<true>(&sm.o_full[t], items & 1, gave_up, kWaitNs);
      if (kApart && ok) ok = tc::mbar_sleep<true>(&sm.pv_done[t], (step - 1) & 1, gave_up, kWaitNs);  // (its phases are all seen)
      if (!ok) break;
      ++items;
      tc::tc_fence_after();
      const float l = fabsf(ref) >= kFar && ref != -INFINITY ? NAN : (l2.x + l2.y) + (k2.x + k2.y);
      const float inv = l == 0.f ? 0.f : kv4::rcp(l);
      const bool some_bad = sm.bad[turn.slot()] != 0;
      const int* bad = sm.first_bad[turn.slot()];
      const size_t row0 = static_cast<size_t>(it.begin + from) * a.Hq + it.head * a.G;
      if (real && a.lse)
        a.lse[row0 + tok * a.Hq + in_group] = l == 0.f ? -INFINITY : ((ref == -INFINITY ? 0.f : ref) + kv4::lg2(l)) * kv4::kLn2;
      // A lane has a whole row.  Four lanes turn their rows' 128 bytes about, so that a store takes whole lines: 8 rows' 128 bytes
      // (32 bytes of each of 32 rows to a store: 3300 cycles an item).  The loop stays a loop: code that runs once an item comes
      // from far.
      const int mine = real ? tok * a.Hq * D + in_group * D : -1, quarter = lane & 3;
      uint16_t* out = a.out + row0 * D + quarter * 16;
      int at[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) at[k] = __shfl_sync(0xFFFFFFFFu, mine, (lane & ~3) + k);
#pragma unroll 1
      for (int i = 0; i < D; i += 64) {
        uint32_t w[4][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2 o[16];
          tmem_ld32(to + i + 32 * h, o);
          tc::tmem_ld_wait();
          if (some_bad) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              if (bad[i + 32 * h + 2 * e] < limit) o[e].x = NAN;
              if (bad[i + 32 * h + 2 * e + 1] < limit) o[e].y = NAN;
            }
          }
#pragma unroll
          for (int x = 0; x < 16; ++x) w[2 * h + x / 8][x % 8] = l == 0.f ? 0u : pack_bf(o[x].x * inv, o[x].y * inv);
        }
        if (i + 64 == D) {
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.o_empty[t]);
        }
        turn4<1>(w, lane);
        turn4<2>(w, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (at[k] >= 0) store32(out + at[k] + i, w[k], a.wide);
      }
      item_done();
    }
    if (!ok && lane == 0) flag_error(a.dev_err, MOE_DEV_TIMEOUT);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  }
  if (warp < 8) {
  } else if (warp < (kApart ? 12 : 10)) {
    // ---------------------------------------------------------- products
    const int t = __shfl_sync(0xFFFFFFFFu, warp & 1, 0);
    const bool with_k = warp < 10, with_v = !kApart || !with_k;  // S = Q K^T, O += P V
    const uint32_t neg = a.negative ? kNegateA : 0u;
    const uint32_t iv = tc::idesc_bf16_f32(kRows, D) | kValuesAlongN;
    constexpr int kTile = P * kPanel >> 4;
    const uint64_t qd = tc::smem_desc_sw128(tc::smem_u32(sm.q[0][0])) + t * kTile, kd = tc::smem_desc_sw128(tc::smem_u32(sm.kv[0][0]));
    const uint64_t vd = value_desc(tc::smem_u32(sm.kv[0][0]));
    const uint32_t ts = tmem + t * 128, tp = tmem + kPCol + t * kPStep, to = tmem + kOCol + t * D;
    int place = 0;                          // in the ring's order: keys, values, keys, ...
    int steps_done = 0, items_done = 0;     // of this tile
    auto wait = [&](uint64_t* bar, int index) {  // its index-th phase
      if (ok) ok = tc::mbar_sleep<true>(bar, index & 1, gave_up, kWaitNs);
    };
    // (within one elected thread)  The scores of the first `keys` keys, a multiple of 16.
    auto scores = [&](int stage, int keys, bool last) {
      const uint32_t is = tc::idesc_bf16_f32(kRows, keys) | neg;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        tc::mma_bf16(ts, qd + (i / 4) * (kPanel >> 4) + 2 * (i % 4), kd + stage * kTile + (i / 4) * (kPanel >> 4) + 2 * (i % 4), is, i > 0);
      tc::mma_commit(&sm.s_full[t]);
      tc::mma_commit(&sm.empty[stage]);
      if (last) tc::mma_commit(&sm.q_empty[t]);
    };
    auto values = [&](int stage, int parts, int j) {
      if (parts == kRows / 16) {
#pragma unroll
        for (int i = 0; i < kRows / 16; ++i) mma_bf16_ts(to, tp + 8 * i, vd + stage * kTile + i * (2048 >> 4), iv, j > 0 || i > 0);
      } else {
        for (int i = 0; i < parts; ++i) mma_bf16_ts(to, tp + 8 * i, vd + stage * kTile + i * (2048 >> 4), iv, j > 0 || i > 0);
      }
    };
    // An item's first scores; keys and values that only the other tile uses are handed back as they are seen.
    auto start = [&](const Item& it, int at) {
      const int st = at % NS, steps = t ? it.n[1] : it.n[0];
      wait(&sm.full[st], at / NS);
      if (steps == 0) {
        if (ok && lane == 0) tc::mbar_arrive(&sm.empty[st]);
        return;
      }
      wait(&sm.q_full[t], items_done);
      if (kApart && steps_done) wait(&sm.s_read[t], steps_done - 1);
      tc::tc_fence_after();
      if (ok && tc::elect_one()) scores(st, min(kRows, (seen_by(a, it, t) + 15) & ~15), steps == 1);
      __syncwarp();
    };
    Item it = next_item();
    if (with_k && it.n[0] >= 0) start(it, 0);
    while (it.n[0] >= 0 && ok) {
      const int n = max(it.n[0], it.n[1]), steps = t ? it.n[1] : it.n[0], seen = seen_by(a, it, t);
      for (int j = 0; j < n && ok; ++j) {
        const int v = place + 2 * j + 1, k = v + 1, sv = v % NS, sk = k % NS;  // this step's values, the next one's keys
        const bool more = j + 1 < steps, other = j + 1 < n;
        const int keys = min(kRows, (seen - (j + 1) * kRows + 15) & ~15);      // of the next step
        if (with_k && other) wait(&sm.full[sk], k / NS);
        if (kApart && with_k) {
          if (more) {
            wait(&sm.s_read[t], steps_done);
            tc::tc_fence_after();
            if (ok && tc::elect_one()) {
              issue_alone(&sm.issuing);
              scores(sk, keys, j + 2 == steps);
              issue_done(&sm.issuing);
            }
            __syncwarp();
          } else if (other && ok && lane == 0) {
            tc::mbar_arrive(&sm.empty[sk]);
          }
        }
        if (with_v) {
          wait(&sm.v_ok[sv], v / NS);
          if (j < steps) {
            if (j == 0) wait(&sm.o_empty[t], items_done + 1);  // (the first passes)
            wait(&sm.p_full[t], steps_done);
            tc::tc_fence_after();
            if (ok && tc::elect_one()) {
              issue_alone(&sm.issuing);
              values(sv, more ? kRows / 16 : (seen - j * kRows + 15) / 16, j);
              if (kApart) tc::mma_commit(&sm.pv_done[t]);
              if (!kApart && more) scores(sk, keys, j + 2 == steps);
              if (!more) tc::mma_commit(&sm.o_full[t]);
              tc::mma_commit(&sm.empty[sv]);
              issue_done(&sm.issuing);
            }
            __syncwarp();
            if (!kApart && !more && other && ok && lane == 0) tc::mbar_arrive(&sm.empty[sk]);
          } else if (ok && lane == 0) {
            tc::mbar_arrive(&sm.empty[sv]);
            if (!kApart && other) tc::mbar_arrive(&sm.empty[sk]);
          }
        }
        steps_done += j < steps;
      }
      if (!ok) break;
      items_done += steps > 0;
      place += 2 * n;
      item_done();
      it = next_item();
      if (with_k && it.n[0] >= 0) start(it, place);
    }
    if (!ok) {
      if (lane == 0) flag_error(a.dev_err, MOE_DEV_TIMEOUT);
      if (tc::elect_one()) {
        tc::mma_commit(&sm.drain);
        int never = 0;
        tc::mbar_wait_bounded(&sm.drain, 0, &never, kWaitNs / 100);
      }
      __syncwarp();
    }
  } else if (warp == 12) {
    // ---------------------------------------------------------- loads
    int place = 0, q_used[2] = {0, 0};
    while (true) {
      const Item it = next_item();
      if (it.n[0] < 0) break;
      const int row = it.begin + it.first, n = max(it.n[0], it.n[1]);
      for (int x = 0; x < 2 * n && ok; ++x, ++place) {
        const int s = place % NS;
        ok = tc::mbar_sleep<true>(&sm.empty[s], (place / NS + 1) & 1, gave_up, kWaitNs);
        if (ok && tc::elect_one()) {
          tc::mbar_arrive_expect_tx(&sm.full[s], P * kPanel);
          if (!(a.stall && x == 2 * n - 2)) {
            for (int p = 0; p < P; ++p)
              tc::tma_load(sm.kv[s][p], x & 1 ? &vmap : &kmap, 64 * p, it.head, it.begin + (x >> 1) * kRows, &sm.full[s]);
          }
        }
        __syncwarp();
        if (x > 0) continue;
        // (Behind the first keys: the queries' place is free a step later than theirs.)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (it.n[t] == 0) continue;
          if (ok) ok = tc::mbar_sleep<true>(&sm.q_empty[t], (q_used[t] + 1) & 1, gave_up, kWaitNs);
          ++q_used[t];
          if (ok && tc::elect_one()) {
            tc::mbar_arrive_expect_tx(&sm.q_full[t], P * a.G * a.tokens * 128);
            for (int p = 0; p < P; ++p) tc::tma_load(sm.q[t][p], &qmap, 64 * p, it.head * a.G, row + t * a.tokens, &sm.q_full[t]);
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      item_done();
    }
    // The last products' arrivals are seen before the CTA may leave.
    for (int i = 0; i < NS && ok; ++i, ++place) ok = tc::mbar_sleep<true>(&sm.empty[place % NS], (place / NS + 1) & 1, gave_up, kWaitNs);
    for (int t = 0; t < 2 && ok; ++t) ok = tc::mbar_sleep<true>(&sm.q_empty[t], (q_used[t] + 1) & 1, gave_up, kWaitNs);
    if (!ok) {
      // Copies in flight land in microseconds.
      if (lane == 0) {
        flag_error(a.dev_err, MOE_DEV_TIMEOUT);
        const uint64_t t0 = tc::globaltimer_ns();
        while (tc::globaltimer_ns() - t0 < 5000000ull) __nanosleep(1000);
      }
      __syncwarp();
    }
  } else if (warp == 13) {
    // ---------------------------------------------------------- values that a row may not see
    int place = 0;
    while (true) {
      const Item it = next_item();
      if (it.n[0] < 0) break;
      const int n = max(it.n[0], it.n[1]), slot = turn.slot();
      for (int j = 0; j < n; ++j) {
        const int v = place + 2 * j + 1, s = v % NS;
        ok = tc::mbar_sleep<true>(&sm.full[s], (v / NS) & 1, gave_up, kWaitNs);
        if (!ok) break;
        // Keys from the first one that some row does not see to the last that a product takes.
        const int lo = max(0, it.first + 1 - j * kRows) & ~7, hi = min(kRows, (seen_by(a, it, 1) - j * kRows + 15) & ~15);
        if (lo < hi) {
          // 0 * x + 0 is NaN for an x that is not finite, two values at a time.
          uint32_t odd[4] = {0, 0, 0, 0};
#pragma unroll
          for (int p = 0; p < P; ++p) {
            const uint4* at = reinterpret_cast<const uint4*>(sm.kv[s][p] + lo * 128) + lane;
#pragma unroll 8
            for (int i = 0; i < (hi - lo) * 8; i += 32) {
              const uint4 w = at[i];
              zero_times(odd[0], w.x), zero_times(odd[1], w.y), zero_times(odd[2], w.z), zero_times(odd[3], w.w);
            }
          }
          if (__any_sync(0xFFFFFFFFu, ((odd[0] | odd[1] | odd[2] | odd[3]) & 0x7FFF7FFFu) != 0)) {
            for (int i = lane; i < P * (hi - lo) * 64; i += 32) {
              const int d = i % (P * 64), row = lo + i / (P * 64);
              uint16_t* e = reinterpret_cast<uint16_t*>(sm.kv[s][d / 64] + row * 128 + ((((d & 63) >> 3) ^ (row & 7)) << 4)) + (d & 7);
              if ((*e & 0x7F80) == 0x7F80) {
                *e = 0;
                atomicMin(&sm.first_bad[slot][d], j * kRows + row);
                sm.bad[slot] = 1;
              }
            }
            tc::fence_async_smem();
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.v_ok[s]);
      }
      if (!ok) break;
      place += 2 * n;
      item_done();
    }
    if (!ok && lane == 0) flag_error(a.dev_err, MOE_DEV_TIMEOUT);
    __syncwarp();
  } else if (warp == 14) {
    // ---------------------------------------------------------- items
    Finder finder{a, sm.blocks, sm.begin, sm.len, sm.most};
    for (int i = 0;; ++i) {  // (ranks stay below 2^27)
      ok = tc::mbar_sleep<true>(&sm.item_empty[turn.slot()], turn.parity() ^ 1, gave_up, kWaitNs);
      if (!ok) break;
      const int slot = turn.slot();
      Item it = {};
      if (out_of_order || !finder.find(static_cast<int>(i * gridDim.x + (i & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x)), &it, lane)) it.n[0] = -1;
      if (sm.bad[slot]) {
        for (int d = lane; d < D; d += 32) sm.first_bad[slot][d] = 0x7FFFFFFF;
        __syncwarp();
        if (lane == 0) sm.bad[slot] = 0;
      }
      if (lane == 0) sm.item[slot] = it;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.item_full[slot]);
      ++turn.i;
      if (it.n[0] < 0) break;
    }
    if (!ok && lane == 0) flag_error(a.dev_err, MOE_DEV_TIMEOUT);
    __syncwarp();
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 8) tc::tmem_dealloc(tmem, 512);
}

// A stride over n tokens or heads.
bool stride_ok(long long st, int n) { return n <= 1 || (st > 0 && st % 8 == 0 && st < (1ll << 38)); }

// [T][heads][D] rows, in boxes of 64 dimensions of h heads and t tokens.
bool rows_map(CUtensorMap* m, const void* p, int T, int heads, int D, long long ts, long long hs, uint32_t h, uint32_t t) {
  const uint64_t d[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(heads), static_cast<uint64_t>(T)};
  const uint64_t s[2] = {2ull * (heads > 1 ? hs : D), 2ull * (T > 1 ? ts : D)};
  const uint32_t b[3] = {64, h, t};
  return tc::make_bf16_map(m, p, 3, d, s, b);
}

template <int D>
int launch(const moe_prompt_cfg& c, const void* q, const void* k, const void* v, PromptArgs a, cudaStream_t s) {
  CUtensorMap qm, km, vm;
  if (!rows_map(&qm, q, c.T, c.n_q_heads, D, c.q_token_stride, c.q_head_stride, a.G, a.tokens) ||
      !rows_map(&km, k, c.T, c.n_kv_heads, D, c.k_token_stride, c.k_head_stride, 1, kRows) ||
      !rows_map(&vm, v, c.T, c.n_kv_heads, D, c.v_token_stride, c.v_head_stride, 1, kRows))
    return MOE_ERR_CUDA;
  const int e = allow_smem<prompt_kernel<D>>(kSmemBytes<D>);
  if (e != MOE_OK) return e;
  // Blocks of a kv head, one more for each sequence at most.
  const long long items = (c.T / (2 * a.tokens) + static_cast<long long>(c.n_seq)) * c.n_kv_heads;
  LaunchScope ls(kProfPrompt, s);
  prompt_kernel<D><<<static_cast<unsigned>(std::min<long long>(items, sm_count())), kThreads, kSmemBytes<D>, s>>>(qm, km, vm, a);
  return check_launch();
}

}  // namespace
}  // namespace moe

extern "C" int moe_prompt_attend(const void* q, const void* k, const void* v, const int32_t* start,
                                 const moe_prompt_cfg* cfg, void* out, float* lse, int32_t* dev_err, void* stream) {
  using namespace moe;
  if (!cfg) return MOE_ERR_ARG;
  const moe_prompt_cfg& c = *cfg;
  if (c.T < 0 || c.n_seq < 0 || c.n_q_heads < 1 || c.n_kv_heads < 1 || !std::isfinite(c.scale * kv4::kLog2e)) return MOE_ERR_ARG;
  if (c.n_q_heads % c.n_kv_heads) return MOE_ERR_ARG;
  if (c.head_dim != 64 && c.head_dim != 128) return MOE_ERR_UNSUPPORTED;
  if (c.T > (1 << 24) || c.n_seq > kMaxSeqs || c.n_q_heads > 1024 || c.n_q_heads / c.n_kv_heads > 128) return MOE_ERR_UNSUPPORTED;
  if (!stride_ok(c.q_token_stride, c.T) || !stride_ok(c.q_head_stride, c.n_q_heads) || !stride_ok(c.k_token_stride, c.T) ||
      !stride_ok(c.k_head_stride, c.n_kv_heads) || !stride_ok(c.v_token_stride, c.T) || !stride_ok(c.v_head_stride, c.n_kv_heads))
    return MOE_ERR_UNSUPPORTED;
  if (c.T == 0 || c.n_seq == 0) return MOE_OK;
  if (!q || !k || !v || !start || !out) return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
       reinterpret_cast<uintptr_t>(out)) & 15 ||
      (reinterpret_cast<uintptr_t>(start) | reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(dev_err)) & 3)
    return MOE_ERR_ARG;
  auto rows = [&](const void* p, int H, long long ts, long long hs) {
    return Rows{reinterpret_cast<uintptr_t>(p), c.T, 2 * ts, H, 2 * hs, 2ll * c.head_dim};
  };
  const long long n_rows = static_cast<long long>(c.T) * c.n_q_heads;
  const Rows o = whole(out, n_rows * 2 * c.head_dim), z = whole(lse, lse ? n_rows * 4 : 0);
  for (const Rows& r : {rows(q, c.n_q_heads, c.q_token_stride, c.q_head_stride), rows(k, c.n_kv_heads, c.k_token_stride, c.k_head_stride),
                        rows(v, c.n_kv_heads, c.v_token_stride, c.v_head_stride)})
    if (!rows_apart(r, o) || !rows_apart(r, z)) return MOE_ERR_ARG;
  if (!rows_apart(o, z)) return MOE_ERR_ARG;
  PromptArgs a = {};
  a.start = start, a.out = static_cast<uint16_t*>(out), a.lse = lse, a.dev_err = dev_err;
  a.T = c.T, a.S = c.n_seq, a.Hq = c.n_q_heads, a.Hkv = c.n_kv_heads, a.G = c.n_q_heads / c.n_kv_heads;
  a.tokens = kRows / a.G;
  a.c = std::fmax(std::fabs(c.scale) * kv4::kLog2e, 1.17549435e-38f);  // (not 0: what is left out is -inf times this)
  a.negative = c.scale < 0.f;
  a.wide = reinterpret_cast<uintptr_t>(out) % 32 == 0;
  a.stall = (test_stall_mask() & MOE_TEST_STALL_PROMPT) != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return c.head_dim == 64 ? launch<64>(c, q, k, v, a, s) : launch<128>(c, q, k, v, a, s);
}
