// kv4_attend for many query rows per kv head (a tree of several tokens times
// the query heads of its kv head, a chunk of a prompt): blocks of 128 rows on
// the 5th-generation tensor cores.
//
// Per tile of 64 slots: S [128 x 64] = Q K^T with Q as the TMEM operand and
// the key codes unpacked to fp16 in shared memory, a softmax thread per row,
// O [128 x D] += P V with P as the TMEM operand (over S's columns) and the
// value codes unpacked to fp16, transposed.  Keys stay bare codes (their nibbles
// are fp16 numbers already, see kv4.cuh); their scales and zeros, and the values'
// zeros, enter per slot in the softmax, in fp32.  Value codes are multiplied by
// their scale while they are unpacked (one rounding to fp16, relative 2^-11)
// and by the power of two 2^-E that brings the tile's largest scale to [1, 2), so
// that no magnitude leaves fp16's range; the exponential takes E back: p' =
// 2^(t - m + E).
//
// Roles: warps 0-3 softmax and output (a thread per row), warps 4-7 unpack,
// warp 8 copies tiles, warp 9 issues the products.  256 TMEM columns (Q, S / P,
// O) and half the shared memory: two CTAs share an SM, and one's products
// run while the other's exponentials do.  Bound by the exponentials (16 a
// clock and SM: 8 clocks per slot of 128 rows) and as much by the products (8).
#include "kv4_attend.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr int kThreads = 384;
constexpr int kRaw = 4;       // tiles in flight
constexpr uint32_t kTmemCols = 256;

template <int D>
struct Smem {
  alignas(1024) uint8_t k16[2][kTile * D * 2];  // panels of 64 dimensions: [64 slots][128 B], 128-byte swizzle
  alignas(1024) uint8_t v16[2][D * kTile * 2];  // [D rows][64 slots]
  Tile<D> raw[kRaw];
  alignas(16) float ks[2][kTile];
  alignas(16) float kz[2][kTile];
  alignas(16) float vz[2][kTile];               // times 2^-E
  float e[2];                                    // the tile's E
  uint32_t raw_groups[kRaw], groups[2];
  alignas(16) uint32_t vs[4][kTile / 2];         // per unpacking warp: scales times 2^-E of slot pairs
  uint64_t raw_full[kRaw], raw_empty[kRaw], kv_full[2], kv_empty[2], q_full, s_full, p_full, pv_done;
  long long scratch[32];
  uint32_t tmem;
  int abort, never;
  long long cum[1];                              // [S + 1]
};

// D[tmem] (+)= A[tmem] * B[smem]^T, fp16 operands, fp32 sums.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of kind::f16 with fp16 A/B, fp32 D, both K-major.
constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

template <int N>
__device__ __forceinline__ void set_regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void set_regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// The part of the unit order that a CTA does in one item.
struct Span {
  Cursor k;
  int row0, rows;
  int n;              // units of the item that are this CTA's
  int tiles;          // of them, those that a row of the block can see
  long long item_end;
};
__device__ __forceinline__ Span span_at(const AttendArgs& a, const long long* cum, long long u, long long u1) {
  Span s;
  cursor_at(s.k, a.c, a.q_start, a.base, a.T, a.G, kWideRows, kTile, cum, u);
  s.item_end = s.k.item0 + s.k.nt;
  s.n = static_cast<int>((s.item_end < u1 ? s.item_end : u1) - u);
  s.row0 = s.k.rb * kWideRows;
  s.rows = min(kWideRows, s.k.q.nq * a.G - s.row0);
  int need = s.k.nt;
  if (!a.visible) need = (min(s.k.q.total, s.k.q.base + (s.row0 + s.rows - 1) / a.G + 1) + kTile - 1) / kTile;
  s.tiles = max(0, min(s.n, need - s.k.tile));
  return s;
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
      tc::mbar_init(&sm.raw_full[i], 1);
      tc::mbar_init(&sm.raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.kv_full[i], 128);
      tc::mbar_init(&sm.kv_empty[i], 1);
    }
    tc::mbar_init(&sm.q_full, 128);
    tc::mbar_init(&sm.s_full, 1);
    tc::mbar_init(&sm.p_full, 128);
    tc::mbar_init(&sm.pv_done, 1);
    sm.abort = sm.never = 0;
    tc::fence_mbar_init();
  }
  if (warp == 8) {
    tc::tmem_alloc(&sm.tmem, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  pdl_wait();
  build_units(a.c, a.q_start, a.base, a.T, a.G, kWideRows, kTile, sm.cum, sm.scratch, a.dev_err, blockIdx.x == 0);
  tc::tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = sm.tmem;
  const long long total = sm.cum[a.c.S];
  const int ncta = static_cast<int>(total < gridDim.x ? total : gridDim.x), cta = blockIdx.x;
  const long long u0 = cta < ncta ? total * cta / ncta : 0, u1 = cta < ncta ? total * (cta + 1) / ncta : 0;
  volatile int* abort_flag = &sm.abort;
  // Waits give up together: the first to run out tells the others.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (tc::mbar_wait_bounded(bar, parity, abort_flag, kWaitBudgetNs)) return true;
    *abort_flag = 1;
    return false;
  };

  if (warp < 4) {
    // ---------------------------------------------------------- softmax, output
    set_regs_up<136>();
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tq = tmem + lanes + kQCol, ts = tmem + lanes + kSCol, to = tmem + lanes + kOCol;
    if (tid < 8) a.meta[static_cast<size_t>(cta) * 8 + tid] = 0;
    Ring<2> kv;
    uint32_t sp = 0;  // parity of s_full, p_full and pv_done
    for (long long u = u0; u < u1;) {
      const Span s = span_at(a, sm.cum, u, u1);
      const int r = s.row0 + tid;
      const bool real = tid < s.rows;
      const int tok = (s.row0 + min(tid, s.rows - 1)) / a.G;
      const uint64_t bits = a.visible ? a.visible[s.k.q.q0 + tok] : 0;
      if (a.visible && s.k.q.nq > kMaxTree && tid == 0) flag_error(a.dev_err, MOE_DEV_CAPACITY);
      float m = 0.f, l = 0.f, z = 0.f, cq = 0.f, cqs = 0.f;
      if (s.tiles > 0) {
        // The row of q, scaled by a power of two and permuted as the key words are (see prep_q), into TMEM.
        const uint4* src = real ? reinterpret_cast<const uint4*>(q_row(a, s.k.q, s.k.h, r)) : nullptr;
        float mx = 0.f, sum = 0.f;
        if (real) {
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const uint4 x = src[i];
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xFFFF0000u);
              mx = fmaxf(mx, fmaxf(fabsf(lo), fabsf(hi)));
              sum += lo + hi;
            }
          }
        }
        const int ex = static_cast<int>(__float_as_uint(mx) >> 23);
        const int e = mx > 0.f && ex < 255 ? 14 + 127 - (ex > 0 ? ex : 1) : 0;
        const float f1 = __uint_as_float(static_cast<uint32_t>(127 + e / 2) << 23);
        const float f2 = __uint_as_float(static_cast<uint32_t>(127 + e - e / 2) << 23);
        cq = ldexpf(a.scale_log2, 24 - e);
        cqs = a.scale_log2 * sum;
#pragma unroll
        for (int i = 0; i < W; i += 4) {
          uint32_t c[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 x = real ? src[i + j] : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            float v[8];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              v[2 * t] = __uint_as_float(w[t] << 16) * f1 * f2;
              v[2 * t + 1] = __uint_as_float(w[t] & 0xFFFF0000u) * f1 * f2;
            }
            c[4 * j] = pack_h2(v[0], v[4]);
            c[4 * j + 1] = pack_h2(v[1] * 0.0625f, v[5] * 0.0625f);
            c[4 * j + 2] = pack_h2(v[2], v[6]);
            c[4 * j + 3] = pack_h2(v[3] * 0.0625f, v[7] * 0.0625f);
          }
          tmem_st16(tq + 4 * i, c);
        }
        tmem_st_wait();
        tc::tc_fence_before();
        tc::mbar_arrive(&sm.q_full);
      }
      bool dead = false;
      for (int it = 0; it < s.tiles; ++it) {
        const int j0 = (s.k.tile + it) * kTile;
        if (!wait(&sm.kv_full[kv.i], kv.phase) || !wait(&sm.s_full, sp)) {
          dead = true;
          break;
        }
        tc::tc_fence_after();
        const float E = sm.e[kv.i];
        const float4* ks4 = reinterpret_cast<const float4*>(sm.ks[kv.i]);
        const float4* kz4 = reinterpret_cast<const float4*>(sm.kz[kv.i]);
        const float off = E - m;
        const float2 cq2 = make_float2(cq, cq), cqs2 = make_float2(cqs, cqs), off2 = make_float2(off, off);
        float2 d[kTile / 2];
#pragma unroll
        for (int c = 0; c < kTile; c += 16) {
          float v[16];
          tc::tmem_ld16(ts + c, v);
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 s4 = ks4[(c + i) / 4], z4 = kz4[(c + i) / 4];
            d[(c + i) / 2] = fma2(make_float2(s4.x, s4.y), mul2(make_float2(v[i], v[i + 1]), cq2),
                                  fma2(make_float2(z4.x, z4.y), cqs2, off2));
            d[(c + i) / 2 + 1] = fma2(make_float2(s4.z, s4.w), mul2(make_float2(v[i + 2], v[i + 3]), cq2),
                                      fma2(make_float2(z4.z, z4.w), cqs2, off2));
          }
        }
        const uint32_t groups = sm.groups[kv.i];
        if (j0 + kTile > s.k.q.base || groups != 15u) {
          const uint64_t see = sees(s.k.q, a.visible != nullptr, bits, tok, j0) & group_mask(groups);
          const uint32_t lo = static_cast<uint32_t>(see), hi = static_cast<uint32_t>(see >> 32);
#pragma unroll
          for (int i = 0; i < kTile / 2; ++i) {
            const uint32_t w = i < 16 ? lo : hi;
            if (!((w >> (2 * i & 31)) & 1)) d[i].x = -INFINITY;
            if (!((w >> ((2 * i + 1) & 31)) & 1)) d[i].y = -INFINITY;
          }
        }
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = fmaxf(d[i].x, d[i].y);
#pragma unroll
        for (int i = 4; i < kTile / 2; ++i) mx[i & 3] = fmaxf(mx[i & 3], fmaxf(d[i].x, d[i].y));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // A row's first visible tile sets its maximum; later ones move it when it lags too far.
        const bool first = l == 0.f && top > -INFINITY;
        if (__any_sync(0xFFFFFFFFu, first || top > kLazy)) {
          const float by = first ? top : fmaxf(top, 0.f);
          const float f = first ? 1.f : ex2(-by);
          const float2 by2 = make_float2(-by, -by);
          m += by;
          l *= f;
          z *= f;
#pragma unroll
          for (int i = 0; i < kTile / 2; ++i) d[i] = add2(d[i], by2);
          if (it > 0) {
#pragma unroll
            for (int c = 0; c < D; c += 8) {
              float v[8];
              tmem_ld8(to + c, v);
              tc::tmem_ld_wait();
              asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(to + c),
                           "f"(v[0] * f), "f"(v[1] * f), "f"(v[2] * f), "f"(v[3] * f), "f"(v[4] * f), "f"(v[5] * f),
                           "f"(v[6] * f), "f"(v[7] * f)
                           : "memory");
            }
          }
        }
        float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0, z0 = sum0, z1 = sum0;
        const float4* vz4 = reinterpret_cast<const float4*>(sm.vz[kv.i]);
#pragma unroll
        for (int c = 0; c < kTile / 2; c += 16) {
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float2 x = make_float2(ex2(d[c + i].x), ex2(d[c + i].y));
            const float2 y = make_float2(ex2(d[c + i + 1].x), ex2(d[c + i + 1].y));
            const float4 zz = vz4[(c + i) / 2];
            sum0 = add2(sum0, x);
            sum1 = add2(sum1, y);
            z0 = fma2(x, make_float2(zz.x, zz.y), z0);
            z1 = fma2(y, make_float2(zz.z, zz.w), z1);
            p[i] = pack_h2(x.x, x.y);
            p[i + 1] = pack_h2(y.x, y.y);
          }
          tmem_st16(ts + c, p);
        }
        sum0 = add2(sum0, sum1);
        z0 = add2(z0, z1);
        z += z0.x + z0.y;
        l = fmaf(sum0.x + sum0.y, ex2(-E), l);
        tmem_st_wait();
        tc::tc_fence_before();
        tc::mbar_arrive(&sm.p_full);
        kv.next();
        sp ^= 1;
      }
      if (dead) break;
      // The item's last product has been summed when pv_done is at the parity of its last tile.
      if (s.tiles > 0) {
        if (!wait(&sm.pv_done, sp ^ 1)) break;
        tc::tc_fence_after();
      }
      const bool whole = u == s.k.item0 && u + s.n == s.item_end;
      const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      float* P = a.part + (static_cast<size_t>(cta) * 2 + (u == u0 ? 0 : 1)) * part_floats<D, kWideRows>();
      const size_t at = (static_cast<size_t>(s.k.q.q0) + tok) * a.Hq + s.k.h * a.G + r % a.G;
      // TMEM column n * W + w is dimension 8 w + n.
#pragma unroll
      for (int w0 = 0; w0 < W; w0 += 4) {
        float o[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          uint32_t x[4] = {0, 0, 0, 0};
          if (s.tiles > 0)
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
          for (int j = 0; j < 4; ++j) o[n][j] += z;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (whole) {
            uint32_t b[4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b[n]) : "f"(o[2 * n + 1][j] * inv), "f"(o[2 * n][j] * inv));
            *reinterpret_cast<uint4*>(a.out + at * D + 8 * (w0 + j)) = make_uint4(b[0], b[1], b[2], b[3]);
          } else {
            float4* x = reinterpret_cast<float4*>(P + tid * D + 8 * (w0 + j));
            x[0] = make_float4(o[0][j], o[1][j], o[2][j], o[3][j]);
            x[1] = make_float4(o[4][j], o[5][j], o[6][j], o[7][j]);
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
      if (!whole && u == s.k.item0 && tid == 0)
        note_cut(a, cta, ncta, total, s.k, s.row0, s.rows, s.item_end, u == u0 ? 0 : 1);
      tc::tc_fence_before();
      u += s.n;
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------- unpack
    set_regs_down<64>();
    const int x = tid - 128;
    Ring<kRaw> raw;
    Ring<2> kv;
    bool dead = false;
    for (long long u = u0; u < u1 && !dead;) {
      const Span s = span_at(a, sm.cum, u, u1);
      for (int it = 0; it < s.tiles; ++it) {
        const int j0 = (s.k.tile + it) * kTile;
        if (!wait(&sm.raw_full[raw.i], raw.phase) || !wait(&sm.kv_empty[kv.i], kv.phase ^ 1)) {
          dead = true;
          break;
        }
        const Tile<D>& t = sm.raw[raw.i];
        const uint32_t groups = sm.raw_groups[raw.i];
        // Parameters of slots 2 lane and 2 lane + 1, in every warp.
        {
          const uint64_t ok = group_mask(groups) & low_ones(static_cast<long long>(s.k.q.total) - j0);
          const uint4 pr = *reinterpret_cast<const uint4*>(t.p + 16 * lane);
          const float2 ka = __half22float2(*reinterpret_cast<const __half2*>(&pr.x));
          const float2 kb = __half22float2(*reinterpret_cast<const __half2*>(&pr.z));
          float2 va = __half22float2(*reinterpret_cast<const __half2*>(&pr.y));
          float2 vb = __half22float2(*reinterpret_cast<const __half2*>(&pr.w));
          // A value row that is not finite must not reach other rows through 0 * NaN: it counts as
          // zeros, and its key makes the rows that see it NaN.
          const bool fa = va.x - va.x == 0.f && va.y - va.y == 0.f, fb = vb.x - vb.x == 0.f && vb.y - vb.y == 0.f;
          if (!fa || !((ok >> (2 * lane)) & 1)) va = make_float2(0.f, 0.f);
          if (!fb || !((ok >> (2 * lane + 1)) & 1)) vb = make_float2(0.f, 0.f);
          const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fmaxf(va.x, vb.x)));
          const int E = top ? static_cast<int>(top >> 23) - 127 : -30;
          const float f = __uint_as_float(static_cast<uint32_t>(127 - E) << 23);
          sm.vs[warp - 4][lane] = pack_h2(va.x * f, vb.x * f);
          if (warp == 4) {
            const float nan = __uint_as_float(0x7FC00000u);
            *reinterpret_cast<float2*>(&sm.ks[kv.i][2 * lane]) = make_float2(fa ? ka.x : nan, fb ? kb.x : nan);
            *reinterpret_cast<float2*>(&sm.kz[kv.i][2 * lane]) = make_float2(ka.y, kb.y);
            *reinterpret_cast<float2*>(&sm.vz[kv.i][2 * lane]) = make_float2(va.y * f, vb.y * f);
            if (lane == 0) {
              sm.e[kv.i] = static_cast<float>(E);
              sm.groups[kv.i] = groups;
            }
          }
        }
        // Keys: 16 bytes of a row (32 codes) make four 16-byte pieces.
#pragma unroll
        for (int q0 = 0; q0 < D / 32; q0 += 2) {
          const int row = x & 63, q = q0 + (x >> 6);
          const uint4 w = *reinterpret_cast<const uint4*>(t.k + row * (D / 2) + 16 * q);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
          uint8_t* dst = sm.k16[kv.i] + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = 4 * q + i;
            *reinterpret_cast<uint4*>(dst + (c >> 3) * (kTile * 128) + (((c & 7) ^ (row & 7)) << 4)) =
                make_uint4(nibbles<0>(ww[i]), nibbles<1>(ww[i]), nibbles<2>(ww[i]), nibbles<3>(ww[i]));
          }
        }
        __syncwarp();
        // Values: a word of each of KP slots makes, for its 8 dimensions, KP fp16 numbers side by side.
        {
          constexpr int KP = D == 128 ? 8 : 4;
          const int w = x % W, k0 = (x / W) * KP;
          const int swap = (lane / W) & 1;  // lanes of two slot groups read rows of opposite parity
          const uint32_t sel_lo = swap ? 0x1054u : 0x5410u, sel_hi = swap ? 0x3276u : 0x7632u;
          uint32_t lo[KP / 2], hi[KP / 2];
          __half2 sc[KP / 2], off[KP / 2];  // scale, -1024 scale
#pragma unroll
          for (int i = 0; i < KP / 2; ++i) {
            const uint32_t y0 = *reinterpret_cast<const uint32_t*>(t.v + (k0 + 2 * i + swap) * (D / 2) + 4 * w);
            const uint32_t y1 = *reinterpret_cast<const uint32_t*>(t.v + (k0 + 2 * i + (swap ^ 1)) * (D / 2) + 4 * w);
            lo[i] = __byte_perm(y0, y1, sel_lo);
            hi[i] = __byte_perm(y0, y1, sel_hi);
            sc[i] = *reinterpret_cast<const __half2*>(&sm.vs[warp - 4][k0 / 2 + i]);
            off[i] = __hmul2(sc[i], __float2half2_rn(-1024.f));
          }
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            uint32_t y[KP / 2];
#pragma unroll
            for (int i = 0; i < KP / 2; ++i) {
              const uint32_t z = n < 4 ? lo[i] : hi[i];
              const uint32_t b = ((z >> (4 * (n & 3))) & 0x000F000Fu) | 0x64006400u;  // 1024 + code
              const __half2 val = __hfma2(*reinterpret_cast<const __half2*>(&b), sc[i], off[i]);
              y[i] = *reinterpret_cast<const uint32_t*>(&val);
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
    }
  } else {
    set_regs_down<40>();
    if (warp == 8) {
      // -------------------------------------------------------- copies
      TileLoader<D> loader;
      Ring<kRaw> raw;
      long long issued = 0;
      bool dead = false;
      for (long long u = u0; u < u1 && !dead;) {
        Span s = span_at(a, sm.cum, u, u1);
        for (int it = 0; it < s.tiles; ++it) {
          if (__any_sync(0xFFFFFFFFu, !wait(&sm.raw_empty[raw.i], raw.phase ^ 1))) {
            dead = true;
            break;
          }
          loader.load(a, s.k, sm.raw[raw.i], &sm.raw_groups[raw.i], &sm.raw_full[raw.i]);
          ++s.k.tile;
          ++issued;
          raw.next();
        }
        u += s.n;
      }
      // Copies in flight land before the CTA's shared memory goes.
      for (long long i = issued > kRaw ? issued - kRaw : 0; i < issued; ++i)
        tc::mbar_wait_bounded(&sm.raw_full[i % kRaw], static_cast<uint32_t>((i / kRaw) & 1), &sm.never, 100000000ull);
    } else if (warp == 9 && lane == 0) {
      // -------------------------------------------------------- products
      const uint32_t is = idesc_f16(kWideRows, kTile), io = idesc_f16(kWideRows, D);
      Ring<2> kv;
      uint32_t qp = 0, sp = 0;
      bool dead = false, any = false;
      for (long long u = u0; u < u1 && !dead;) {
        const Span s = span_at(a, sm.cum, u, u1);
        if (s.tiles > 0) {
          if (!wait(&sm.q_full, qp)) break;
          qp ^= 1;
        }
        for (int it = 0; it < s.tiles; ++it) {
          // S shares its columns with the last tile's P: that product comes first.
          if (!wait(&sm.kv_full[kv.i], kv.phase) || (any && !wait(&sm.pv_done, sp ^ 1))) {
            dead = true;
            break;
          }
          tc::tc_fence_after();
          const uint32_t kb = tc::smem_u32(sm.k16[kv.i]), vb = tc::smem_u32(sm.v16[kv.i]);
#pragma unroll
          for (int t = 0; t < D / 16; ++t)
            mma_ts(tmem + kSCol, tmem + kQCol + 8 * t, tc::smem_desc_sw128(kb + (t >> 2) * (kTile * 128) + (t & 3) * 32), is,
                   t > 0);
          tc::mma_commit(&sm.s_full);
          if (!wait(&sm.p_full, sp)) {
            dead = true;
            break;
          }
          tc::tc_fence_after();
#pragma unroll
          for (int t = 0; t < kTile / 16; ++t)
            mma_ts(tmem + kOCol, tmem + kSCol + 8 * t, tc::smem_desc_sw128(vb + t * 32), io, it > 0 || t > 0);
          tc::mma_commit(&sm.kv_empty[kv.i]);
          tc::mma_commit(&sm.pv_done);
          any = true;
          kv.next();
          sp ^= 1;
        }
        u += s.n;
      }
      // Products in flight end before TMEM is freed.
      if (any || dead) {
        if (dead) {
          tc::mma_commit(&sm.kv_empty[0]);
          const uint64_t t0 = tc::globaltimer_ns();
          while (tc::globaltimer_ns() - t0 < 1000000ull) {}
        } else {
          tc::mbar_wait_bounded(&sm.pv_done, sp ^ 1, &sm.never, 100000000ull);
        }
      }
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
  if (cudaFuncSetAttribute(attend_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  LaunchScope ls(kProfKv4Attend, s);
  return launch_k(attend_wide_kernel<D>, dim3(grid), dim3(kThreads), smem, s, false, a);
}

}  // namespace

int wide_grid() { return 2 * sm_count(); }

int wide_launch(const AttendArgs& a, int grid, cudaStream_t s) {
  return a.c.D == 128 ? launch<128>(a, grid, s) : launch<64>(a, grid, s);
}

}  // namespace kv4
}  // namespace moe
