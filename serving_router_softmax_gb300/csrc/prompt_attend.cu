// moe_prompt_attend: causal attention of packed prompts on the 5th-generation
// tensor cores.
//
// A CTA takes 256 query rows of one kv head, as two tiles of 128: the G query
// heads of floor(128 / G) tokens each, token by token, so that any number of
// heads fills the tiles and the heads share their keys.  Per 128 keys and tile:
//   S [128 x 128] = Q K^T           operands in shared memory, sums in TMEM
//   P = exp2(c S - r), l += row sums    a thread per row, P over S in TMEM as bf16
//   O [128 x D] += P V              P from TMEM, V as it lies ([keys][D])
// One tile's products run while the other's exponentials do.
//
// The reference r of a row's exponentials need not be its maximum: any r gives
// the same quotient O / l.  It moves (and O and l are scaled to it) only when a
// score passes it by more than 8, so that powers stay below 2^8 and O is
// rewritten in a few steps of a row instead of all; bf16 and fp32 are as good
// anywhere in that range.
//
// Blocks of one sequence differ in work by their place in it.  The grid takes
// them in falling order of it over all sequences: rank x among the items is
// found by counting, with no plan in memory: F(b) = sum of max(0, blocks - b)
// items lie at block b of their sequence or later.
//
// What a row may not see: scores are replaced by -inf in the tiles that hold
// any; values there that are not finite would make 0 * v a NaN, so two warps
// look through those value tiles, put zeros in their place, and keep for each
// dimension the first such key, which makes the output of the rows that see it
// NaN.
//
// Roles (384 threads): warps 0-3 and 4-7 softmax and output of a tile each,
// warp 8 issues the products, warp 9 loads by TMA, warps 10-11 look at values.
// Every wait is bounded.
#include <cuda_bf16.h>

#include <cmath>

#include "kv4.cuh"
#include "tc_f16.cuh"
#include "tc_pair.cuh"

namespace moe {
namespace {

using tc::add2;
using tc::fma2;
using tc::mul2;

constexpr int kThreads = 384;
constexpr int kRows = 128;       // query rows of a tile, keys of a step
constexpr int kPanel = kRows * 128;  // bytes of 64 dimensions of a tile
constexpr float kSlack = 8.f;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kMaxSeqs = 4096;

struct PromptArgs {
  const int32_t* start;
  uint16_t* out;
  float* lse;
  int32_t* dev_err;
  int T, S, Hq, Hkv, G, tokens;  // tokens: of a tile
  float c;                       // |scale| log2(e)
  int negative, stall;           // scale < 0; test hook
};

template <int D>
struct Smem {
  static constexpr int kStages = D == 128 ? 4 : 8;
  alignas(1024) uint8_t q[2][D / 64][kPanel];
  alignas(1024) uint8_t kv[kStages][D / 64][kPanel];  // first: blocks of each sequence
  uint64_t q_full, full[kStages], empty[kStages], v_ok[kStages], s_full[2], p_full[2], o_full[2], drain;
  int first_bad[D], bad;
  int sum[12], found;
  uint32_t tmem;
  int abort;
};
template <int D>
constexpr size_t kSmemBytes = sizeof(Smem<D>) + 1024;
static_assert(kSmemBytes<128> <= 227 * 1024 && kSmemBytes<64> <= 227 * 1024, "shared memory");
static_assert(sizeof(Smem<64>::kv) >= kMaxSeqs * 4, "room for the sequences' blocks");

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

// Sum over the block; every thread gets it.
__device__ __forceinline__ int block_sum(int v, int* part) {
  v = __reduce_add_sync(0xFFFFFFFFu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += part[i];
  return s;
}

struct Item {
  int begin, end, first;  // rows of the sequence; its first token here, counted in the sequence
};

// Item of this rank; false if there are fewer, or if the starts are out of order.
template <int D>
__device__ __forceinline__ bool find_item(const PromptArgs& a, Smem<D>& sm, int rank, Item* it) {
  int* blocks = reinterpret_cast<int*>(&sm.kv[0][0][0]);
  const int per = 2 * a.tokens;
  int most = 0, bad = 0;
  for (int s = threadIdx.x; s < a.S; s += kThreads) {
    const int b = a.start[s], e = a.start[s + 1];
    bad |= b < 0 || e > a.T || b > e;
    const int n = bad ? 0 : (e - b + per - 1) / per;
    blocks[s] = n;
    most = max(most, n);
  }
  if (threadIdx.x == 0) sm.found = 0;
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(a.dev_err, MOE_DEV_CAPACITY);
    return false;
  }
  atomicMax(&sm.found, __reduce_max_sync(0xFFFFFFFFu, most));
  __syncthreads();
  // The last b with F(b) > rank.
  int lo = -1, hi = sm.found, above = 0;  // F(hi) <= rank
  while (hi - lo > 1) {
    const int b = lo + (hi - lo) / 2;
    int v = 0;
    for (int s = threadIdx.x; s < a.S; s += kThreads) v += max(0, blocks[s] - b);
    v = block_sum(v, sm.sum);
    if (v > rank)
      lo = b;
    else
      hi = b, above = v;
  }
  if (lo < 0) return false;
  // The (rank - F(lo + 1))-th sequence that has a block lo.
  int skip = rank - above;
  __syncthreads();
  if (threadIdx.x < 32) {
    int seq = -1;
    for (int s0 = 0; s0 < a.S && seq < 0; s0 += 32) {
      const int s = s0 + threadIdx.x;
      const uint32_t has = __ballot_sync(0xFFFFFFFFu, s < a.S && blocks[s] > lo);
      const int n = __popc(has);
      if (skip < n) {
        const bool me = ((has >> threadIdx.x) & 1) && __popc(has & ((1u << threadIdx.x) - 1)) == skip;
        seq = s0 + __ffs(__ballot_sync(0xFFFFFFFFu, me)) - 1;
      }
      skip -= n;
    }
    if (threadIdx.x == 0) sm.found = seq;
  }
  __syncthreads();
  const int s = sm.found;
  it->begin = a.start[s], it->end = a.start[s + 1], it->first = lo * per;
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const PromptArgs a) {
  using Sm = Smem<D>;
  constexpr int NS = Sm::kStages, P = D / 64;
  extern __shared__ uint8_t raw[];
  Sm& sm = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kvh = blockIdx.x % a.Hkv;
  Item it;
  if (!find_item<D>(a, sm, blockIdx.x / a.Hkv, &it)) return;

  if (tid == 0) {
    tc::mbar_init(&sm.q_full, 1);
    for (int i = 0; i < NS; ++i) tc::mbar_init(&sm.full[i], 1), tc::mbar_init(&sm.empty[i], 1), tc::mbar_init(&sm.v_ok[i], 2);
    for (int i = 0; i < 2; ++i) tc::mbar_init(&sm.s_full[i], 1), tc::mbar_init(&sm.p_full[i], 4), tc::mbar_init(&sm.o_full[i], 1);
    tc::mbar_init(&sm.drain, 1);
    sm.abort = sm.bad = 0;
    tc::fence_mbar_init();
  }
  for (int d = tid; d < D; d += kThreads) sm.first_bad[d] = 0x7FFFFFFF;
  if (warp == 8) {
    tc::tmem_alloc(&sm.tmem, 512);
    tc::tmem_relinquish();
  }
  // (The sequences' blocks lay where the copies go.)
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sm.tmem, 0);
  volatile int* gave_up = &sm.abort;
  // Steps of a tile: its last token sees itself.
  const int len = it.end - it.begin;
  auto steps_of = [&](int t) {
    const int from = it.first + t * a.tokens;
    return from >= len ? 0 : (min(from + a.tokens, len) + kRows - 1) / kRows;
  };
  const int n0 = steps_of(0), n1 = steps_of(1), n = max(n0, n1);

  if (warp < 8) {
    // ---------------------------------------------------------- softmax, output
    const int t = warp >> 2, r = (warp & 3) * 32 + lane, steps = t ? n1 : n0;
    const int tok = r / a.G, pos = it.first + t * a.tokens + tok;
    const bool real = tok < a.tokens && pos < len;
    const int limit = real ? pos + 1 : 0;  // keys that the row sees
    const int all_see = it.first + t * a.tokens + 1;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * D;
    float ref = -INFINITY;
    float2 l2 = make_float2(0.f, 0.f);
    bool ok = true;
    const float2 c2 = make_float2(a.c, a.c);
    for (int j = 0; j < steps; ++j) {
      ok = tc::mbar_sleep<true>(&sm.s_full[t], j & 1, gave_up, kWaitNs);
      if (!ok) break;
      tc::tc_fence_after();
      float2 s[64];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, s + 16 * i);
      tc::tmem_ld_wait();
      if ((j + 1) * kRows > all_see) {
        const int see = limit - j * kRows;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          s[i].x = 2 * i < see ? s[i].x : -INFINITY;
          s[i].y = 2 * i + 1 < see ? s[i].y : -INFINITY;
        }
      }
      float m0 = fmaxf(s[0].x, s[0].y), m1 = fmaxf(s[1].x, s[1].y), m2 = fmaxf(s[2].x, s[2].y), m3 = fmaxf(s[3].x, s[3].y);
#pragma unroll
      for (int i = 4; i < 64; i += 4) {
        m0 = kv4::max3(m0, s[i].x, s[i].y), m1 = kv4::max3(m1, s[i + 1].x, s[i + 1].y);
        m2 = kv4::max3(m2, s[i + 2].x, s[i + 2].y), m3 = kv4::max3(m3, s[i + 3].x, s[i + 3].y);
      }
      const float top = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * a.c;
      const bool move = top > ref + kSlack;
      if (__any_sync(0xFFFFFFFFu, move)) {
        const float f = move ? kv4::ex2(ref - top) : 1.f;  // (0 from -inf)
        if (move) ref = top;
        const float2 f2 = make_float2(f, f);
        l2 = mul2(l2, f2);
        if (j > 0) {  // (the products of the step before are over: the scores came after them)
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            float2 o[16];
            tmem_ld32(to + 32 * i, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 x = mul2(o[8 * h + e], f2);
                w[2 * e] = __float_as_uint(x.x), w[2 * e + 1] = __float_as_uint(x.y);
              }
              tc::tmem_st16(to + 32 * i + 16 * h, w);
            }
          }
        }
      }
      const float neg = ref == -INFINITY ? 0.f : -ref;
      const float2 r2 = make_float2(neg, neg);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float2 x = fma2(s[16 * i + e], c2, r2);
          x.x = kv4::ex2(x.x), x.y = kv4::ex2(x.y);
          l2 = add2(l2, x);
          w[e] = pack_bf(x.x, x.y);
        }
        tc::tmem_st16(ts + 16 * i, w);
      }
      tc::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.p_full[t]);
    }
    if (ok && steps > 0) ok = tc::mbar_sleep<true>(&sm.o_full[t], 0, gave_up, kWaitNs);
    if (!ok) {
      if (lane == 0) flag_error(a.dev_err, MOE_DEV_TIMEOUT);
    } else if (steps > 0) {
      tc::tc_fence_after();
      const float l = l2.x + l2.y;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const bool some_bad = sm.bad != 0;
      // A lane's row goes to the tile's query panel in 16-byte parts, swizzled, and from there to its place in whole rows.
      uint8_t* stage = &sm.q[t][0][0] + (warp & 3) * 32 * D * 2;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float2 o[16];
        tmem_ld32(to + 32 * i, o);
        tc::tmem_ld_wait();
        if (some_bad) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (sm.first_bad[32 * i + 2 * e] < limit) o[e].x = NAN;
            if (sm.first_bad[32 * i + 2 * e + 1] < limit) o[e].y = NAN;
          }
        }
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) w[x] = l == 0.f ? 0u : pack_bf(o[e + x].x * inv, o[e + x].y * inv);
          const int part = 4 * i + e / 4;
          *reinterpret_cast<uint4*>(stage + lane * (D * 2) + ((part ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      const int head = r % a.G;
      const int mine = real ? tok * a.Hq * D + head * D : -1;
      const size_t row0 = (static_cast<size_t>(it.begin + it.first + t * a.tokens)) * a.Hq + kvh * a.G;
      uint16_t* out = a.out + row0 * D;
      if (real && a.lse) a.lse[row0 + tok * a.Hq + head] = l == 0.f ? -INFINITY : (ref == -INFINITY ? 0.f : ref) * kv4::kLn2 + logf(l);
      __syncwarp();
      constexpr int kParts = D / 8, kAtOnce = 32 / kParts;  // 16-byte parts of a row, rows a pass
#pragma unroll 4
      for (int i = 0; i < 32; i += kAtOnce) {
        const int row = i + lane / kParts, part = lane % kParts;
        const int at = __shfl_sync(0xFFFFFFFFu, mine, row);
        if (at >= 0)
          *reinterpret_cast<uint4*>(out + at + part * 8) =
              *reinterpret_cast<const uint4*>(stage + row * (D * 2) + ((part ^ (row & 7)) << 4));
      }
    }
  } else if (warp == 8) {
    // ---------------------------------------------------------- products
    const uint32_t is = tc::idesc_bf16_f32(kRows, kRows) | (a.negative ? kNegateA : 0u);
    const uint32_t iv = tc::idesc_bf16_f32(kRows, D) | kValuesAlongN;
    const uint64_t qd = tc::smem_desc_sw128(tc::smem_u32(sm.q[0][0])), kd = tc::smem_desc_sw128(tc::smem_u32(sm.kv[0][0]));
    const uint64_t vd = value_desc(tc::smem_u32(sm.kv[0][0]));
    constexpr int kTile = P * kPanel >> 4;
    bool ok = tc::mbar_sleep<true>(&sm.q_full, 0, gave_up, kWaitNs);
    auto wait = [&](uint64_t* bar, int index) {  // its index-th phase
      if (ok) ok = tc::mbar_sleep<true>(bar, index & 1, gave_up, kWaitNs);
      tc::tc_fence_after();
    };
    auto scores = [&](int t, int stage) {
      if (ok && tc::elect_one()) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          tc::mma_bf16(tmem + t * 128, qd + t * kTile + (i / 4) * (kPanel >> 4) + 2 * (i % 4), kd + stage * kTile + (i / 4) * (kPanel >> 4) + 2 * (i % 4),
                       is, i > 0);
        tc::mma_commit(&sm.s_full[t]);
      }
      __syncwarp();
    };
    auto values = [&](int t, int stage, int j) {
      if (ok && tc::elect_one()) {
#pragma unroll
        for (int i = 0; i < kRows / 16; ++i)
          mma_bf16_ts(tmem + 256 + t * D, tmem + t * 128 + 8 * i, vd + stage * kTile + i * (2048 >> 4), iv, j > 0 || i > 0);
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (ok && tc::elect_one()) tc::mma_commit(bar);
      __syncwarp();
    };
    wait(&sm.full[0], 0);
    if (n0) scores(0, 0);
    if (n1) scores(1, 0);
    commit(&sm.empty[0]);
    for (int j = 0; j < n && ok; ++j) {
      const int v = 2 * j + 1, k = 2 * j + 2;  // places in the ring's order of this step's values and the next one's keys
      const bool more = j + 1 < n;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int steps = t ? n1 : n0;
        if (j >= steps) continue;
        wait(&sm.p_full[t], j);
        wait(&sm.v_ok[v % NS], v / NS);
        values(t, v % NS, j);
        if (j + 1 < steps) {
          wait(&sm.full[k % NS], k / NS);
          scores(t, k % NS);
        } else {
          commit(&sm.o_full[t]);
        }
      }
      commit(&sm.empty[v % NS]);
      if (more) commit(&sm.empty[k % NS]);
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
  } else if (warp == 9) {
    // ---------------------------------------------------------- loads
    if (tc::elect_one()) {
      const int row = it.begin + it.first;
      const int tiles = n1 ? 2 : 1;
      tc::mbar_arrive_expect_tx(&sm.q_full, tiles * P * a.G * a.tokens * 128);
      for (int t = 0; t < tiles; ++t)
        for (int p = 0; p < P; ++p) tc::tma_load(sm.q[t][p], &qmap, 64 * p, kvh * a.G, row + t * a.tokens, &sm.q_full);
    }
    __syncwarp();
    bool ok = true;
    for (int i = 0; i < 2 * n; ++i) {
      const int s = i % NS;
      ok = tc::mbar_sleep<true>(&sm.empty[s], (i / NS + 1) & 1, gave_up, kWaitNs);
      if (!ok) break;
      if (tc::elect_one()) {
        tc::mbar_arrive_expect_tx(&sm.full[s], P * kPanel);
        if (!(a.stall && i == 2 * n - 2)) {
          for (int p = 0; p < P; ++p)
            tc::tma_load(sm.kv[s][p], i & 1 ? &vmap : &kmap, 64 * p, kvh, it.begin + (i >> 1) * kRows, &sm.full[s]);
        }
      }
      __syncwarp();
    }
    if (!ok) {
      // Copies in flight land in microseconds.
      if (lane == 0) {
        flag_error(a.dev_err, MOE_DEV_TIMEOUT);
        const uint64_t t0 = tc::globaltimer_ns();
        while (tc::globaltimer_ns() - t0 < 5000000ull) __nanosleep(1000);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------- values that a row may not see
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int v = 2 * j + 1, s = v % NS;
      ok = tc::mbar_sleep<true>(&sm.full[s], (v / NS) & 1, gave_up, kWaitNs);
      if (!ok) break;
      if ((j + 1) * kRows > it.first + 1) {
        bool wrote = false;
        for (int i = tid - 320; i < P * kPanel / 16; i += 64) {
          uint4* at = reinterpret_cast<uint4*>(&sm.kv[s][0][0]) + i;
          const uint4 w = *at;
          auto odd = [](uint32_t x) { return ((x & 0x7F807F80u) + 0x00800080u) & 0x80008000u; };  // exponents of ones carry over
          if (odd(w.x) | odd(w.y) | odd(w.z) | odd(w.w)) {
            const int row = (i >> 3) & (kRows - 1), part = (i & 7) ^ (row & 7), d0 = (i / (kPanel / 16)) * 64 + part * 8;
            uint16_t e[8];
            *reinterpret_cast<uint4*>(e) = w;
            for (int x = 0; x < 8; ++x) {
              if ((e[x] & 0x7F80) == 0x7F80) {
                e[x] = 0;
                atomicMin(&sm.first_bad[d0 + x], j * kRows + row);
                sm.bad = 1;
              }
            }
            *at = *reinterpret_cast<const uint4*>(e);
            wrote = true;
          }
        }
        if (__any_sync(0xFFFFFFFFu, wrote)) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.v_ok[s]);
    }
    if (!ok && lane == 0) flag_error(a.dev_err, MOE_DEV_TIMEOUT);
    __syncwarp();
  }
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
  if (items > 0x7FFFFFFFll) return MOE_ERR_UNSUPPORTED;
  LaunchScope ls(kProfPrompt, s);
  prompt_kernel<D><<<static_cast<unsigned>(items), kThreads, kSmemBytes<D>, s>>>(qm, km, vm, a);
  return check_launch();
}

}  // namespace
}  // namespace moe

extern "C" int moe_prompt_attend(const void* q, const void* k, const void* v, const int32_t* start,
                                 const moe_prompt_cfg* cfg, void* out, float* lse, int32_t* dev_err, void* stream) {
  using namespace moe;
  if (!cfg) return MOE_ERR_ARG;
  const moe_prompt_cfg& c = *cfg;
  if (c.T < 0 || c.n_seq < 0 || c.n_q_heads < 1 || c.n_kv_heads < 1 || !std::isfinite(c.scale)) return MOE_ERR_ARG;
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
  PromptArgs a = {};
  a.start = start, a.out = static_cast<uint16_t*>(out), a.lse = lse, a.dev_err = dev_err;
  a.T = c.T, a.S = c.n_seq, a.Hq = c.n_q_heads, a.Hkv = c.n_kv_heads, a.G = c.n_q_heads / c.n_kv_heads;
  a.tokens = kRows / a.G;
  a.c = std::fmax(std::fabs(c.scale) * kv4::kLog2e, 1.17549435e-38f);  // (not 0: what is left out is -inf times this)
  a.negative = c.scale < 0.f;
  a.stall = (test_stall_mask() & MOE_TEST_STALL_PROMPT) != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return c.head_dim == 64 ? launch<64>(c, q, k, v, a, s) : launch<128>(c, q, k, v, a, s);
}
