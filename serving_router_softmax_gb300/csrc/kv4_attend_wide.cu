// kv4_attend for many query rows per kv head (a tree of several tokens times
// the query heads of its kv head, a chunk of a prompt): blocks of 128 rows on
// the 5th-generation tensor cores.
//
// Per tile of 64 slots: S [128 x 64] = Q K^T with Q as the TMEM operand and
// the key codes unpacked to fp16 in shared memory, a softmax thread per row,
// O [128 x D] += P V with P as the TMEM operand (over S's columns) and the
// value codes unpacked to fp16, transposed.  Both stay bare codes, their nibbles
// being fp16 numbers already (see kv4.cuh); the scales and zeros enter per slot in
// the softmax, in fp32.  P holds the probability times its slot's value scale,
// 2^(t + log2 vs - m), with the row's running maximum m over that exponent: the
// row's own largest product is what fp16's range lies around, whatever
// the scales of the slots are, and of those it does not see.
//
// Roles: warps 0-3 softmax and output (a thread per row), warps 4-7 unpack,
// warp 8 issues the products, warp 9 copies tiles.  The scores of a tile come in two halves of 32 slots, each with its own
// columns (its P over its S), so that one half's products run while the other's
// exponentials do.  256 TMEM columns (Q, S / P, O), half the shared memory and 96
// registers a thread: two CTAs share an SM.  The exponentials (32 a clock and SM) would allow 4 clocks per slot of
// 128 rows, the products (D = 64) 5; it takes about 30, in the chain of a half (scores out of TMEM, maximum,
// exponentials, P into TMEM, product), which two CTAs do not hide: 145 us for 2 chunks of up to 500 tokens of 32 query heads on
// up to 6000 slots of 8 kv heads, D = 64 (294 TFLOP/s, issue slots 51% busy, tensor pipe 14%).
#include "kv4_attend.cuh"
#include "tc_f16.cuh"

namespace moe {
namespace kv4 {
namespace {

using tc::add2;
using tc::fma2;
using tc::idesc_f16;
using tc::mul2;
using tc::tmem_st16;
using tc::tmem_st_wait;

constexpr int kThreads = 320;
constexpr int kRaw = 3;       // tiles in flight
constexpr uint32_t kTmemCols = 256;
constexpr int kHalf = kTile / 2;
constexpr int kMinUnits = 4;

template <int D>
struct Smem {
  alignas(1024) uint8_t k16[2][kTile * D * 2];  // panels of 64 dimensions: [64 slots][128 B], 128-byte swizzle
  alignas(1024) uint8_t v16[2][D * kTile * 2];  // [D rows][64 slots]
  Tile<D> raw[kRaw];
  alignas(16) float ks[2][kTile];
  alignas(16) float kz[2][kTile];
  alignas(16) float lv[2][kTile];               // log2 of the value scale vs
  alignas(16) float rs[2][kTile];               // 1 / vs
  alignas(16) float zr[2][kTile];               // vz / vs
  uint32_t raw_groups[kRaw], groups[2];
  uint2 bad[2];                                  // slots whose values are not finite: the even ones, the odd ones
  uint64_t raw_full[kRaw], raw_empty[kRaw], kv_full[2], kv_empty[2], q_full, s_full[2], p_full[2], pv_done[2];
  long long scratch[32];
  uint32_t tmem;
  int abort, never;
  long long cum[1];                              // [S + 1]
};

// 32 columns of the thread's lane, waited for.
__device__ __forceinline__ void tmem_ld_pairs(uint32_t taddr, float2 (&e)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(e[0].x), "=f"(e[0].y), "=f"(e[1].x), "=f"(e[1].y), "=f"(e[2].x), "=f"(e[2].y), "=f"(e[3].x), "=f"(e[3].y),
        "=f"(e[4].x), "=f"(e[4].y), "=f"(e[5].x), "=f"(e[5].y), "=f"(e[6].x), "=f"(e[6].y), "=f"(e[7].x), "=f"(e[7].y),
        "=f"(e[8].x), "=f"(e[8].y), "=f"(e[9].x), "=f"(e[9].y), "=f"(e[10].x), "=f"(e[10].y), "=f"(e[11].x),
        "=f"(e[11].y), "=f"(e[12].x), "=f"(e[12].y), "=f"(e[13].x), "=f"(e[13].y), "=f"(e[14].x), "=f"(e[14].y),
        "=f"(e[15].x), "=f"(e[15].y)
      : "r"(taddr));
  tc::tmem_ld_wait();
}

// Ring position of a pipeline of N stages.
template <int N>
struct Ring {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) i = 0, phase ^= 1;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2) attend_wide_kernel(const AttendArgs a) {
  constexpr int W = D / 8;                  // code words of a row
  constexpr uint32_t kQCol = 0, kSCol = D / 2, kOCol = D / 2 + kTile;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kRaw; ++i) {
      tc::mbar_init(&sm.raw_full[i], arrivals_of_stage(a, i));
      tc::mbar_init(&sm.raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.kv_full[i], 128);
      tc::mbar_init(&sm.kv_empty[i], 1);
      tc::mbar_init(&sm.s_full[i], 1);
      tc::mbar_init(&sm.p_full[i], 128);
      tc::mbar_init(&sm.pv_done[i], 1);
    }
    tc::mbar_init(&sm.q_full, 128);
    sm.abort = sm.never = 0;
    tc::fence_mbar_init();
  }
  if (warp == 8) {
    tc::tmem_alloc(&sm.tmem, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  pdl_wait();
  build_units(a.c, a.q_start, a.base, a.T, a.G, kWideRows, kTile, kItemUnits, sm.cum, sm.scratch, a.dev_err, blockIdx.x == 0);
  tc::tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = sm.tmem;
  const long long total = sm.cum[a.c.S];
  const int ncta = used_ctas(total, kMinUnits), cta = blockIdx.x;
  const Shares shares(total, max(ncta, 1));
  const long long u0 = cta < ncta ? shares.begin(cta) : 0, u1 = cta < ncta ? shares.begin(cta + 1) : 0;
  volatile int* abort_flag = &sm.abort;
  Cursor k;
  if (u0 < u1) cursor_at(k, a.c, a.q_start, a.base, a.T, a.G, kWideRows, kTile, kItemUnits, sm.cum, u0);
  // Waits give up together: the first to run out tells the others.
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_phase<false>(bar, parity, abort_flag); };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) { return wait_phase<true>(bar, parity, abort_flag); };

  if (warp < 4) {
    // ---------------------------------------------------------- softmax, output
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tq = tmem + lanes + kQCol, ts = tmem + lanes + kSCol, to = tmem + lanes + kOCol;
    if (tid < 8) a.meta[static_cast<size_t>(cta) * 8 + tid] = 0;
    Ring<2> kv;
    uint32_t sp = 0;  // parity of s_full, p_full and pv_done
    for (long long u = u0; u < u1;) {
      const Span s = span_of<kWideRows>(a, k, u, u1);
      if (s.tiles == 0) {
        u += s.n;
        if (u < u1) cursor_next(k, a.c, a.q_start, a.base, a.T, a.G, kWideRows, kTile, kItemUnits, sm.cum);
        continue;
      }
      // Token and query head of row x of the block (small numbers: a multiplication finds the quotient).
      const int tok0 = s.row0 / a.G, g0 = s.row0 - tok0 * a.G;
      const float inv_g = 1.f / static_cast<float>(a.G);
      auto token = [&](int x) { return static_cast<int>((static_cast<float>(g0 + x) + 0.5f) * inv_g); };
      const bool real = tid < s.rows;
      const int tok_rel = token(min(tid, s.rows - 1)), tok = tok0 + tok_rel;
      const int head = k.h * a.G + g0 + tid - tok_rel * a.G;
      const uint64_t bits = a.visible ? a.visible[k.q.q0 + tok] : 0;
      if (a.visible && k.q.nq > kMaxTree && tid == 0) flag_error(a.dev_err, MOE_DEV_CAPACITY);
      float m = 0.f, l = 0.f, z = 0.f, cq = 0.f, cqs = 0.f;
      {
        // The warp's 32 rows of q, scaled by powers of two (see prep_q), into TMEM.  In a half of 16
        // rows lane 4 a + x takes word x (8 dimensions) of every 32 of rows a and a + 8, which is how the 16 x 256 bit
        // store wants them: of the 16 columns of 32 dimensions, word x has 2 x, 2 x + 1 (its pairs (0, 4) and
        // (1, 5)/16) and 8 + 2 x, 9 + 2 x ((2, 6) and (3, 7)/16).
        const int lr = lane >> 2, x = lane & 3;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          constexpr int C = D / 32;
          uint4 v[2][C];
          float f[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int rr = warp * 32 + 16 * half + 8 * i + lr, tr = token(rr);
            const uint16_t* src = a.q + (k.q.q0 + tok0 + tr) * a.q_ts + (k.h * a.G + g0 + rr - tr * a.G) * a.q_hs + 8 * x;
#pragma unroll
            for (int c = 0; c < C; ++c)
              v[i][c] = rr < s.rows ? *reinterpret_cast<const uint4*>(src + 32 * c) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t mag = 0;  // largest magnitudes of the low and the high halves, as bf16
            float2 both = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < C; ++c) {
              const uint32_t w[4] = {v[i][c].x, v[i][c].y, v[i][c].z, v[i][c].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                mag = __vmaxu2(mag, w[j] & 0x7FFF7FFFu);
                both = add2(both, make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u)));
              }
            }
            float sum = both.x + both.y;
            mag = __vmaxu2(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 1));
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            mag = __vmaxu2(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 2));
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
            // (Below 2^-113 a row's largest magnitude lands below 2^14; its scores are zero all the same.)
            const int ex = static_cast<int>(max(mag >> 16, mag & 0xFFFFu) >> 7);
            const int e = ex > 0 && ex < 255 ? min(14 + 127 - ex, 127) : 0;
            f[i] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            // The lane of the row keeps its factors.
            const int es = __shfl_sync(0xFFFFFFFFu, e, 4 * (lane & 7));
            const float ss = __shfl_sync(0xFFFFFFFFu, sum, 4 * (lane & 7));
            if (lane >> 3 == 2 * half + i) {
              const int y = 24 - es;  // the codes carry 2^-24; two factors, as y may pass one fp32's range
              cq = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + (y >> 1)) << 23) *
                   __uint_as_float(static_cast<uint32_t>(127 + y - (y >> 1)) << 23);
              cqs = a.scale_log2 * ss;
            }
          }
#pragma unroll
          for (int c = 0; c < C; ++c) {
            uint32_t o[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint4 u = v[i][c];
              const float f16 = f[i] * 0.0625f;
              auto pair = [](uint32_t lo, uint32_t hi, float by) {
                const float2 y = mul2(make_float2(__uint_as_float(lo), __uint_as_float(hi)), make_float2(by, by));
                return pack_h2(y.x, y.y);
              };
              o[i][0] = pair(u.x << 16, u.z << 16, f[i]);
              o[i][1] = pair(u.x & 0xFFFF0000u, u.z & 0xFFFF0000u, f16);
              o[i][2] = pair(u.y << 16, u.w << 16, f[i]);
              o[i][3] = pair(u.y & 0xFFFF0000u, u.w & 0xFFFF0000u, f16);
            }
            asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                             tq + (static_cast<uint32_t>(16 * half) << 16) + 16 * c),
                         "r"(o[0][0]), "r"(o[0][1]), "r"(o[1][0]), "r"(o[1][1]), "r"(o[0][2]), "r"(o[0][3]), "r"(o[1][2]),
                         "r"(o[1][3])
                         : "memory");
          }
        }
        tmem_st_wait();
        tc::tc_fence_before();
        tc::mbar_arrive(&sm.q_full);
      }
      bool dead = false;
      for (int it = 0; it < s.tiles && !dead; ++it) {
        const int j0 = (k.tile + it) * kTile;
        if (!wait_warp(&sm.kv_full[kv.i], kv.phase)) {
          dead = true;
          break;
        }
        const uint32_t groups = sm.groups[kv.i];
        const bool edge = j0 + kTile > k.q.base || groups != 15u;
        uint64_t see = 0;
        if (edge) see = sees(k.q, a.visible != nullptr, bits, tok, j0) & group_mask(groups);
        const uint2 bad = sm.bad[kv.i];
        if (bad.x | bad.y) {
          // Values that are not finite reach the outputs of the rows that see them, and nothing else.
          const uint64_t sight = edge ? see : ~0ull;
          for (int i = 0; i < 32; ++i)
            if (((bad.x >> i) & (sight >> (2 * i)) & 1) || ((bad.y >> i) & (sight >> (2 * i + 1)) & 1)) z = __uint_as_float(0x7FC00000u);
        }
        for (int h = 0; h < 2; ++h) {
          if (!wait_warp(&sm.s_full[h], sp)) {
            dead = true;
            break;
          }
          tc::tc_fence_after();
          const uint32_t tsh = ts + h * kHalf;
          const float4* ks4 = reinterpret_cast<const float4*>(sm.ks[kv.i] + h * kHalf);
          const float4* kz4 = reinterpret_cast<const float4*>(sm.kz[kv.i] + h * kHalf);
          const float4* lv4 = reinterpret_cast<const float4*>(sm.lv[kv.i] + h * kHalf);
          const float4* rs4 = reinterpret_cast<const float4*>(sm.rs[kv.i] + h * kHalf);
          const float4* zr4 = reinterpret_cast<const float4*>(sm.zr[kv.i] + h * kHalf);
          const float2 cq2 = make_float2(cq, cq), cqs2 = make_float2(cqs, cqs), off2 = make_float2(-m, -m);
          float2 d[kHalf / 2];
          tmem_ld_pairs(tsh, d);
#pragma unroll
          for (int i = 0; i < kHalf / 2; i += 2) {
            const float4 s4 = ks4[i / 2], z4 = kz4[i / 2], v4 = lv4[i / 2];
            d[i] = fma2(make_float2(s4.x, s4.y), mul2(d[i], cq2),
                        fma2(make_float2(z4.x, z4.y), cqs2, add2(make_float2(v4.x, v4.y), off2)));
            d[i + 1] = fma2(make_float2(s4.z, s4.w), mul2(d[i + 1], cq2),
                            fma2(make_float2(z4.z, z4.w), cqs2, add2(make_float2(v4.z, v4.w), off2)));
          }
          if (edge) {
            const uint32_t w = static_cast<uint32_t>(h ? see >> 32 : see);
#pragma unroll
            for (int i = 0; i < kHalf / 2; ++i) {
              if (!((w >> (2 * i)) & 1)) d[i].x = -INFINITY;
              if (!((w >> (2 * i + 1)) & 1)) d[i].y = -INFINITY;
            }
          }
          float mx[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = fmaxf(d[i].x, d[i].y);
#pragma unroll
          for (int i = 4; i < kHalf / 2; ++i) mx[i & 3] = max3(mx[i & 3], d[i].x, d[i].y);
          const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
          // A row's first visible slots set its maximum; later ones move it when it lags too far.
          const bool first = l == 0.f && top > -INFINITY;
          if (__any_sync(0xFFFFFFFFu, first || top > kLazy)) {
            const float by = first ? top : fmaxf(top, 0.f);
            const float f = first ? 1.f : ex2(-by);
            const float2 by2 = make_float2(-by, -by);
            m += by;
            l *= f;
            z *= f;
#pragma unroll
            for (int i = 0; i < kHalf / 2; ++i) d[i] = add2(d[i], by2);
            if (it > 0 || h > 0) {
              // The half before has been summed into O first.
              if (!wait_warp(&sm.pv_done[h ^ 1], h ? sp : sp ^ 1)) {
                dead = true;
                break;
              }
              tc::tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                float v[16];
                uint32_t x[16];
                tc::tmem_ld16(to + c, v);
                tc::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(v[i] * f);
                tmem_st16(to + c, x);
              }
            }
          }
          float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0, z0 = sum0, z1 = sum0;
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float2 x = make_float2(ex2(d[i].x), ex2(d[i].y));
            const float2 y = make_float2(ex2(d[i + 1].x), ex2(d[i + 1].y));
            const float4 zz = zr4[i / 2], rr = rs4[i / 2];
            sum0 = fma2(x, make_float2(rr.x, rr.y), sum0);
            sum1 = fma2(y, make_float2(rr.z, rr.w), sum1);
            z0 = fma2(x, make_float2(zz.x, zz.y), z0);
            z1 = fma2(y, make_float2(zz.z, zz.w), z1);
            p[i] = pack_h2(x.x, x.y);
            p[i + 1] = pack_h2(y.x, y.y);
          }
          tmem_st16(tsh, p);
          sum0 = add2(sum0, sum1);
          z0 = add2(z0, z1);
          z += z0.x + z0.y;
          l += sum0.x + sum0.y;
          tmem_st_wait();
          tc::tc_fence_before();
          tc::mbar_arrive(&sm.p_full[h]);
        }
        kv.next();
        sp ^= 1;
      }
      if (dead) break;
      // The item's products have been summed when pv_done is at the parity of its last tile.
      if (!wait_warp(&sm.pv_done[0], sp ^ 1) || !wait_warp(&sm.pv_done[1], sp ^ 1)) break;
      tc::tc_fence_after();
      const bool whole = s.whole;
      const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      float* P = a.part + (static_cast<size_t>(cta) * 2 + (u == u0 ? 0 : 1)) * part_floats<D, kWideRows>();
      const size_t at = (static_cast<size_t>(k.q.q0) + tok) * a.Hq + head;
      // TMEM column n * W + w is dimension 8 w + n.  (Loops that run once an item stay rolled: a cold
      // instruction costs about 10 clocks.)
#pragma unroll 1
      for (int w0 = 0; w0 < W; w0 += 4) {
        float o[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          uint32_t x[4];
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                       : "r"(to + n * W + w0));
#pragma unroll
          for (int j = 0; j < 4; ++j) o[n][j] = __uint_as_float(x[j]);
        }
        tc::tmem_ld_wait();
        if (!real) continue;
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[n][j] = fmaf(o[n][j], (n & 1) ? 1048576.f : 16777216.f, z);
        if (!whole) {
          // Lanes are rows: a column of the block is 128 floats side by side.
#pragma unroll
          for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) P[(n * W + w0 + j) * kWideRows + tid] = o[n][j];
          continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          {
            uint32_t b[4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b[n]) : "f"(o[2 * n + 1][j] * inv), "f"(o[2 * n][j] * inv));
            *reinterpret_cast<uint4*>(a.out + at * D + 8 * (w0 + j)) = make_uint4(b[0], b[1], b[2], b[3]);
          }
        }
      }
      if (real) {
        if (whole) {
          if (a.lse) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        } else {
          P[kWideRows * D + tid] = l == 0.f ? kNone : m;
          P[kWideRows * D + kWideRows + tid] = l;
        }
      }
      if (!whole && s.first && tid == 0) note_cut(a, cta, shares, k, s, u, u == u0 ? 0 : 1);
      tc::tc_fence_before();
      u += s.n;
      if (u < u1) cursor_next(k, a.c, a.q_start, a.base, a.T, a.G, kWideRows, kTile, kItemUnits, sm.cum);
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------- unpack
    const int x = tid - 128;
    Ring<kRaw> raw;
    Ring<2> kv;
    bool dead = false;
    const TileMap<D> map(a.c);
    for (long long u = u0; u < u1 && !dead;) {
      const Span s = span_of<kWideRows>(a, k, u, u1);
      for (int it = 0; it < s.tiles; ++it) {
        const int j0 = (k.tile + it) * kTile;
        if (!wait_warp(&sm.raw_full[raw.i], raw.phase) || !wait_warp(&sm.kv_empty[kv.i], kv.phase ^ 1)) {
          dead = true;
          break;
        }
        const uint8_t* t = sm.raw[raw.i].b;
        const uint32_t groups = sm.raw_groups[raw.i];
        if (warp == 4) {
          // Parameters of slots 2 lane and 2 lane + 1.
          const uint64_t ok = group_mask(groups) & low_ones(static_cast<long long>(k.q.total) - j0);
          const uint4 pr = *reinterpret_cast<const uint4*>(t + map.p(2 * lane));
          const float2 ka = __half22float2(*reinterpret_cast<const __half2*>(&pr.x));
          const float2 kb = __half22float2(*reinterpret_cast<const __half2*>(&pr.z));
          float2 va = __half22float2(*reinterpret_cast<const __half2*>(&pr.y));
          float2 vb = __half22float2(*reinterpret_cast<const __half2*>(&pr.w));
          // A value row that is not finite must not reach other rows through 0 * NaN: it counts as
          // zeros here, and the softmax threads add it to the rows that see it.
          const bool fa = va.x - va.x == 0.f && va.y - va.y == 0.f, fb = vb.x - vb.x == 0.f && vb.y - vb.y == 0.f;
          if (!fa || !((ok >> (2 * lane)) & 1)) va = make_float2(0.f, 0.f);
          if (!fb || !((ok >> (2 * lane + 1)) & 1)) vb = make_float2(0.f, 0.f);
          const float sa = fmaxf(va.x, kMinScale), sb = fmaxf(vb.x, kMinScale), ra = rcp(sa), rb = rcp(sb);
          const uint2 bad = make_uint2(__ballot_sync(0xFFFFFFFFu, !fa), __ballot_sync(0xFFFFFFFFu, !fb));
          *reinterpret_cast<float2*>(&sm.ks[kv.i][2 * lane]) = make_float2(ka.x, kb.x);
          *reinterpret_cast<float2*>(&sm.kz[kv.i][2 * lane]) = make_float2(ka.y, kb.y);
          *reinterpret_cast<float2*>(&sm.lv[kv.i][2 * lane]) = make_float2(lg2(sa), lg2(sb));
          *reinterpret_cast<float2*>(&sm.rs[kv.i][2 * lane]) = make_float2(ra, rb);
          *reinterpret_cast<float2*>(&sm.zr[kv.i][2 * lane]) = make_float2(va.y * ra, vb.y * rb);
          if (lane == 0) {
            sm.groups[kv.i] = groups;
            sm.bad[kv.i] = bad;
          }
        }
        // Keys: 16 bytes of a row (32 codes) make four 16-byte pieces.
#pragma unroll
        for (int q0 = 0; q0 < D / 32; q0 += 2) {
          const int row = x & 63, q = q0 + (x >> 6);
          const uint4 w = *reinterpret_cast<const uint4*>(t + map.k(row) + 16 * q);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
          uint8_t* dst = sm.k16[kv.i] + (row >> 3) * 1024 + (row & 7) * 128 + (q >> 1) * (kTile * 128);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // In the order of Q's columns: first the pairs (0, 4) and (1, 5) of the four words, then the others.
            const uint32_t y = ww[2 * (i & 1)], z = ww[2 * (i & 1) + 1];
            *reinterpret_cast<uint4*>(dst + (((4 * (q & 1) + i) ^ (row & 7)) << 4)) =
                i < 2 ? make_uint4(nibbles<0>(y), nibbles<1>(y), nibbles<0>(z), nibbles<1>(z))
                      : make_uint4(nibbles<2>(y), nibbles<3>(y), nibbles<2>(z), nibbles<3>(z));
          }
        }
        // Values: a word of each of KP slots makes, for its 8 dimensions, KP fp16 numbers side by side.
        {
          constexpr int KP = D == 128 ? 8 : 4;
          const int w = x % W, k0 = (x / W) * KP;
          const int swap = (lane / W) & 1;  // lanes of two slot groups read rows of opposite parity
          const uint32_t sel_lo = swap ? 0x1054u : 0x5410u, sel_hi = swap ? 0x3276u : 0x7632u;
          const uint8_t* tv = t + map.v(k0) + 4 * w;
          uint32_t lo[KP / 2], hi[KP / 2];
#pragma unroll
          for (int i = 0; i < KP / 2; ++i) {
            const uint32_t y0 = *reinterpret_cast<const uint32_t*>(tv + (2 * i + swap) * (D / 2));
            const uint32_t y1 = *reinterpret_cast<const uint32_t*>(tv + (2 * i + (swap ^ 1)) * (D / 2));
            lo[i] = __byte_perm(y0, y1, sel_lo);
            hi[i] = __byte_perm(y0, y1, sel_hi);
          }
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            uint32_t y[KP / 2];
#pragma unroll
            for (int i = 0; i < KP / 2; ++i) {
              const uint32_t z = n < 4 ? lo[i] : hi[i];
              y[i] = ((n & 2) ? z >> 8 : z) & ((n & 1) ? 0x00F000F0u : 0x000F000Fu);
            }
            const int row = n * W + w;
            uint8_t* dst = sm.v16[kv.i] + (row >> 3) * 1024 + (row & 7) * 128 + (((k0 / 8) ^ (row & 7)) << 4);
            if constexpr (KP == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
            else *reinterpret_cast<uint2*>(dst + (k0 & 4) * 2) = make_uint2(y[0], y[1]);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc::mbar_arrive(&sm.kv_full[kv.i]);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.raw_empty[raw.i]);
        raw.next();
        kv.next();
      }
      u += s.n;
      if (u < u1) cursor_next(k, a.c, a.q_start, a.base, a.T, a.G, kWideRows, kTile, kItemUnits, sm.cum);
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------- copies
    TileLoader<D> loader(a.c);
    Ring<kRaw> raw;
    int issued = 0;  // (only its remainder and whether it passed kRaw matter)
    bool dead = false;
    for (long long u = u0; u < u1 && !dead;) {
      const Span s = span_of<kWideRows>(a, k, u, u1);
      const int tiles = copied_tiles(a, s, u + s.n == u1);
      for (int it = 0; it < tiles; ++it) {
        if (!wait_warp(&sm.raw_empty[raw.i], raw.phase ^ 1)) {
          dead = true;
          break;
        }
        loader.load(a, k, sm.raw[raw.i], &sm.raw_groups[raw.i], &sm.raw_full[raw.i]);
        ++k.tile;
        issued = min(issued + 1, kRaw);
        raw.next();
      }
      u += s.n;
      if (u < u1) cursor_next(k, a.c, a.q_start, a.base, a.T, a.G, kWideRows, kTile, kItemUnits, sm.cum);
    }
    // Copies in flight land before the CTA's shared memory goes.
    for (int i = 0; i < issued; ++i) {
      raw.i = raw.i ? raw.i - 1 : kRaw - 1;
      if (raw.i == kRaw - 1) raw.phase ^= 1;
      wait_phase<true>(&sm.raw_full[raw.i], raw.phase, &sm.never, 100000000ull);
    }
  } else if (lane == 0) {
    // ---------------------------------------------------------- products
    const uint32_t is = idesc_f16(kWideRows, kHalf), io = idesc_f16(kWideRows, D);
    const uint64_t kd0 = tc::smem_desc_sw128(tc::smem_u32(sm.k16)), vd0 = tc::smem_desc_sw128(tc::smem_u32(sm.v16));
    Ring<2> kv;
    uint32_t qp = 0, sp = 0;
    bool dead = false, any = false;
    // Scores of half h of the tile in unpacked buffer b.
    auto scores = [&](int h, int b) {
      const uint64_t kd = kd0 + b * (sizeof(sm.k16[0]) >> 4) + h * (kHalf * 128 >> 4);
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
        tc::mma_f16_ts(tmem + kSCol + h * kHalf, tmem + kQCol + 8 * t, kd + (t >> 2) * (kTile * 128 >> 4) + (t & 3) * 2, is, t > 0);
      tc::mma_commit(&sm.s_full[h]);
    };
    for (long long u = u0; u < u1 && !dead;) {
      const Span s = span_of<kWideRows>(a, k, u, u1);
      if (s.tiles > 0) {
        if (!wait(&sm.q_full, qp) || !wait(&sm.kv_full[kv.i], kv.phase)) {
          dead = true;
          break;
        }
        qp ^= 1;
        any = true;
        tc::tc_fence_after();
        scores(0, kv.i);
        scores(1, kv.i);
      }
      for (int it = 0; it < s.tiles && !dead; ++it) {
        const int b = kv.i;
        kv.next();
        for (int h = 0; h < 2; ++h) {
          if (!wait(&sm.p_full[h], sp)) {
            dead = true;
            break;
          }
          tc::tc_fence_after();
          const uint64_t vd = vd0 + b * (sizeof(sm.v16[0]) >> 4) + h * (kHalf * 2 >> 4);
#pragma unroll
          for (int t = 0; t < kHalf / 16; ++t)
            tc::mma_f16_ts(tmem + kOCol, tmem + kSCol + h * kHalf + 8 * t, vd + t * 2, io, it > 0 || h > 0 || t > 0);
          if (h) tc::mma_commit(&sm.kv_empty[b]);
          tc::mma_commit(&sm.pv_done[h]);
          if (it + 1 < s.tiles) {
            // The next tile's scores go over this P once its product is done.
            if ((h == 0 && !wait(&sm.kv_full[kv.i], kv.phase)) || !wait(&sm.pv_done[h], sp)) {
              dead = true;
              break;
            }
            tc::tc_fence_after();
            scores(h, kv.i);
          }
        }
        sp ^= 1;
      }
      u += s.n;
      if (u < u1) cursor_next(k, a.c, a.q_start, a.base, a.T, a.G, kWideRows, kTile, kItemUnits, sm.cum);
    }
    // Products in flight end before TMEM is freed.
    if (dead) {
      const uint64_t t0 = tc::globaltimer_ns();
      while (tc::globaltimer_ns() - t0 < 1000000ull) {}
    } else if (any) {
      wait_phase<false>(&sm.pv_done[1], sp ^ 1, &sm.never, 100000000ull);
    }
  }
  __syncthreads();
  if (tid == 0 && *abort_flag) flag_error(a.dev_err, MOE_DEV_TIMEOUT);
  if (warp == 8) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
int launch(const AttendArgs& a, int grid, cudaStream_t s) {
  const size_t smem = sizeof(Smem<D>) + static_cast<size_t>(a.c.S) * 8;
  int st = allow_smem<attend_wide_kernel<D>>(smem);
  if (st != MOE_OK) return st;
  {
    LaunchScope ls(kProfKv4Attend, s);
    st = launch_k(attend_wide_kernel<D>, dim3(grid), dim3(kThreads), smem, s, false, a);
  }
  if (st != MOE_OK) return st;
  return launch_combine<D, kWideRows, true>(a, grid, s);
}

}  // namespace

int wide_grid() { return 2 * sm_count(); }

int wide_launch(const AttendArgs& a, int grid, cudaStream_t s) {
  return a.c.D == 128 ? launch<128>(a, grid, s) : launch<64>(a, grid, s);
}

}  // namespace kv4
}  // namespace moe
