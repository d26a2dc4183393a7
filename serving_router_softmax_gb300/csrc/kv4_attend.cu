// kv4_attend: attention of a batch's new tokens over the 4-bit paged cache.
//
// One pass over the cache with a running softmax maximum and sum, in the
// transposed form: scores S^T [slots x query rows] = C_k Q^T with the key codes as
// the row operand straight from their nibbles, output O^T [D x query rows] =
// C_v^T P^T with the value codes.  The query rows of a kv head (its new tokens
// times the query heads that share it) are the narrow side, in steps of 8, so
// a single decoded token of 8 query heads wastes nothing.
//
// Each CTA owns an even share of all (sequence, head, row block, tile) units;
// a producer warp keeps a ring of tiles in flight (bulk copies), two consumer
// warps take 32 slots of each tile, two groups of 16 beside each other.  An item cut between CTAs leaves its
// partial sums in the workspace and the combine kernel joins them in CTA
// order, so results do not depend on timing.
#include "kv4_attend.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr int kConsumerWarps = 2;
constexpr int kGroups = kTile / 16 / kConsumerWarps;  // 16-slot groups of a tile that a warp takes
constexpr int kMinUnits = 1;
constexpr int kThreads = 32 * (kConsumerWarps + 1);
// CTAs that an SM holds, by their registers.
constexpr int ctas_per_sm(int nt) { return nt <= 2 ? 4 : 2; }

template <int D, int NT, int NS>
struct Smem {
  static constexpr int RB = 8 * NT;
  Tile<D> st[NS];
  uint4 frag[NT * (D / 32) * 32];
  float o[RB][D + 4];
  float cq[RB], cqs[RB];
  float m[kConsumerWarps][RB], l[kConsumerWarps][RB], z[kConsumerWarps][RB];
  uint64_t mask[RB];
  uint64_t full[NS], empty[NS];
  uint32_t groups[NS];  // bit g: the page of slots 16g..16g+15 of the tile is valid
  long long scratch[32];
  int abort, never;
  long long cum[1];     // [S + 1]
};

// MMA layouts: see kv4.cuh.
template <int D, int NT, int NS>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NT)) attend_kernel(const AttendArgs a) {
  using SM = Smem<D, NT, NS>;
  constexpr int RB = SM::RB;
  constexpr int J = NT == 4 ? 1 : kGroups;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  SM& sm = *reinterpret_cast<SM*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(&sm.full[i], 1);
      tc::mbar_init(&sm.empty[i], kConsumerWarps);
    }
    sm.abort = sm.never = 0;
    tc::fence_mbar_init();
  }
  pdl_wait();
  build_units(a.c, a.q_start, a.base, a.T, a.G, RB, kTile, kItemUnits, sm.cum, sm.scratch, a.dev_err, blockIdx.x == 0);
  pdl_trigger();
  const long long total = sm.cum[a.c.S];
  const int ncta = used_ctas(total, kMinUnits), cta = blockIdx.x;
  const long long u0 = cta < ncta ? total * cta / ncta : 0, u1 = cta < ncta ? total * (cta + 1) / ncta : 0;
  volatile int* abort_flag = &sm.abort;

  if (warp == kConsumerWarps) {
    // ---------------------------------------------------------- producer
    Cursor k;
    TileLoader<D> loader(a.c);
    int stage = 0, phase = 0;
    long long issued = 0;
    if (u0 < u1) cursor_at(k, a.c, a.q_start, a.base, a.T, a.G, RB, kTile, kItemUnits, sm.cum, u0);
    bool dead = false;
    for (long long u = u0; u < u1 && !dead;) {
     const Span sp = span_of<RB>(a, k, u, u1);
     for (int it = 0; it < sp.tiles; ++it) {
      const bool ok = tc::mbar_wait_bounded(&sm.empty[stage], phase ^ 1, abort_flag, kWaitBudgetNs);
      if (__any_sync(0xFFFFFFFFu, !ok)) {
        *abort_flag = 1;
        dead = true;
        break;
      }
      loader.load(a, k, sm.st[stage], &sm.groups[stage], &sm.full[stage]);
      ++issued;
      ++k.tile;
      if (++stage == NS) stage = 0, phase ^= 1;
     }
     u += sp.n;
     if (u < u1) cursor_next(k, a.c, a.q_start, a.base, a.T, a.G, RB, kTile, kItemUnits, sm.cum);
    }
    if (*abort_flag) {
      // Copies in flight land before the CTA's shared memory goes.
      for (long long i = issued > NS ? issued - NS : 0; i < issued; ++i)
        tc::mbar_wait_bounded(&sm.full[i % NS], static_cast<uint32_t>((i / NS) & 1), &sm.never, 100000000ull);
      if (lane == 0) flag_error(a.dev_err, MOE_DEV_TIMEOUT);
    }
    return;
  }

  // ------------------------------------------------------------ consumers
  const int g = lane >> 2, c = lane & 3;
  const int s0 = slot_of_row(g), s1 = slot_of_row(g + 8);
  const TileMap<D> map(a.c);
  int k_at[kGroups], v_at[kGroups], p_at[kGroups];
#pragma unroll
  for (int x = 0; x < kGroups; ++x) {
    const int r = 16 * (kGroups * warp + x);
    k_at[x] = map.k(r);
    v_at[x] = map.v(r);
    p_at[x] = map.p(r);
  }
  int stage = 0, phase = 0;
  if (tid < 8) a.meta[static_cast<size_t>(cta) * 8 + tid] = 0;
  Cursor k;
  if (u0 < u1) cursor_at(k, a.c, a.q_start, a.base, a.T, a.G, RB, kTile, kItemUnits, sm.cum, u0);
  for (long long u = u0; u < u1;) {
    const Span sp = span_of<RB>(a, k, u, u1);
    const int n = sp.tiles, row0 = sp.row0, rows = sp.rows;
    if (n == 0) {
      u += sp.n;
      if (u < u1) cursor_next(k, a.c, a.q_start, a.base, a.T, a.G, RB, kTile, kItemUnits, sm.cum);
      continue;
    }
    prep_q<D>([&](int r) { return r < rows ? q_row(a, k.q, k.h, row0 + r) : (const uint16_t*)nullptr; }, RB, a.scale_log2, sm.frag, sm.cq,
              sm.cqs, tid, 32 * kConsumerWarps);
    if (tid < RB && a.visible) sm.mask[tid] = a.visible[k.q.q0 + (row0 + min(tid, rows - 1)) / a.G];
    if (a.visible && k.q.nq > kMaxTree && tid == 0) flag_error(a.dev_err, MOE_DEV_CAPACITY);
    tc::named_bar_sync(1, 32 * kConsumerWarps);

    float o[D / 16][NT][4];
    float m[NT][2], l[NT][2], z[NT][2], cq[NT][2], cqs[NT][2];
    uint32_t fresh = (1u << (2 * NT)) - 1;  // rows (of this lane's columns) that have seen nothing
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[t][e] = l[t][e] = z[t][e] = 0.f;
        cq[t][e] = sm.cq[8 * t + 2 * c + e];
        cqs[t][e] = sm.cqs[8 * t + 2 * c + e];
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][t][e] = 0.f;
    }

    for (int it = 0; it < n; ++it) {
      const int j0 = (k.tile + it) * kTile + 16 * kGroups * warp;  // first slot of this warp's groups
      if (!tc::mbar_wait_bounded(&sm.full[stage], phase, abort_flag, kWaitBudgetNs)) *abort_flag = 1;
      __syncwarp();
      const uint8_t* st = sm.st[stage].b;
      const uint32_t groups = sm.groups[stage] >> (kGroups * warp);
      const bool edge = j0 + 16 * kGroups > k.q.base || (groups & ((1u << kGroups) - 1)) != (1u << kGroups) - 1;
      // J groups of 16 slots at a time, their chains beside each other.
#pragma unroll
      for (int x0 = 0; x0 < kGroups; x0 += J) {
        float d[J][NT][4], rs[J][2], zr[J][2];
#pragma unroll
        for (int x = 0; x < J; ++x) {
          uint32_t ka[D / 32], kb[D / 32];
          load_k_words<D>(st + k_at[x0 + x] + s0 * (D / 2), c, ka);
          load_k_words<D>(st + k_at[x0 + x] + s1 * (D / 2), c, kb);
          const uint2 ra = *reinterpret_cast<const uint2*>(st + p_at[x0 + x] + s0 * 8);
          const uint2 rb = *reinterpret_cast<const uint2*>(st + p_at[x0 + x] + s1 * 8);
          float ks[2], kz[2], lv[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint2 r = e ? rb : ra;
            const float2 kp = __half22float2(*reinterpret_cast<const __half2*>(&r.x));
            const float2 vp = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
            const float se = fmaxf(vp.x, kMinScale);
            ks[e] = kp.x;
            kz[e] = kp.y;
            lv[e] = lg2(se);
            rs[x][e] = rcp(se);
            zr[x][e] = vp.y * rs[x][e];
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            qk_16x8<D>(acc, ka, kb, sm.frag + t * (D / 32) * 32);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int kk = e >> 1, y = e & 1;
              d[x][t][e] = fmaf(ks[kk], acc[e] * cq[t][y], fmaf(kz[kk], cqs[t][y], lv[kk] - m[t][y]));
            }
          }
        }
        // Where slots may be out of sight (or out of range): their exponents are -inf, and
        // what their parameters hold (NaN, say) must not reach the sums.
        uint32_t seen = 0xFFFFFFFFu;  // bit 4 (NT x + t) + e
        if (edge) {
          seen = 0;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int r = 8 * t + 2 * c + y;
#pragma unroll
              for (int x = 0; x < J; ++x) {
                uint64_t v = 0;
                if ((groups >> (x0 + x)) & 1)
                  v = sees(k.q, a.visible != nullptr, sm.mask[r], (row0 + min(r, rows - 1)) / a.G, j0 + 16 * (x0 + x));
                if ((v >> s0) & 1) seen |= 1u << (4 * (NT * x + t) + y);
                else d[x][t][y] = -INFINITY;
                if ((v >> s1) & 1) seen |= 1u << (4 * (NT * x + t) + 2 + y);
                else d[x][t][2 + y] = -INFINITY;
              }
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int x = 0; x < J; ++x)
#pragma unroll
          for (int t = 0; t < NT; ++t) top = max3(max3(top, d[x][t][0], d[x][t][1]), d[x][t][2], d[x][t][3]);
        if (__any_sync(0xFFFFFFFFu, top > kLazy || fresh != 0)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float mx = -INFINITY;
#pragma unroll
              for (int x = 0; x < J; ++x) mx = max3(mx, d[x][t][y], d[x][t][2 + y]);
              mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
              // A row's first visible slots set its maximum; later ones only raise it.
              const bool first = (fresh >> (2 * t + y)) & 1, none = mx == -INFINITY;
              const float by = none ? 0.f : first ? mx : fmaxf(mx, 0.f);
              const float f = first ? 1.f : ex2(-by);
              if (!none) fresh &= ~(1u << (2 * t + y));
              m[t][y] += by;
              l[t][y] *= f;
              z[t][y] *= f;
#pragma unroll
              for (int x = 0; x < J; ++x) {
                d[x][t][y] -= by;
                d[x][t][2 + y] -= by;
              }
#pragma unroll
              for (int j = 0; j < D / 16; ++j) {
                o[j][t][y] *= f;
                o[j][t][2 + y] *= f;
              }
            }
        }
        uint2 pf[J][NT];
#pragma unroll
        for (int x = 0; x < J; ++x)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              p[e] = ex2(d[x][t][e]);
              if (!edge || ((seen >> (4 * (NT * x + t) + e)) & 1)) {
                l[t][e & 1] = fmaf(p[e], rs[x][e >> 1], l[t][e & 1]);
                z[t][e & 1] = fmaf(p[e], zr[x][e >> 1], z[t][e & 1]);
              }
            }
            pf[x][t] = make_uint2(transpose_8x8(pack_h2(p[0], p[1])), transpose_8x8(pack_h2(p[2], p[3])));
          }
        // Values: lane (g, c) owns k indices 2c, 2c+1, 2c+8, 2c+9 and the
        // dimensions g * D/8 ..; one byte permute pairs two slots' halves.
        const int v0 = slot_of_row(2 * c), v1 = slot_of_row(2 * c + 1);
#pragma unroll
        for (int x = 0; x < J; ++x) {
          const uint8_t* vb = st + v_at[x0 + x] + g * (D / 16);
          if constexpr (D == 128) {
            uint2 w[4];
            w[0] = *reinterpret_cast<const uint2*>(vb + v0 * (D / 2));
            w[1] = *reinterpret_cast<const uint2*>(vb + v1 * (D / 2));
            w[2] = *reinterpret_cast<const uint2*>(vb + (8 + v0) * (D / 2));
            w[3] = *reinterpret_cast<const uint2*>(vb + (8 + v1) * (D / 2));
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t sel = hf ? 0x7632u : 0x5410u;
              const uint32_t xa = __byte_perm(w[0].x, w[1].x, sel), ya = __byte_perm(w[0].y, w[1].y, sel);
              const uint32_t xb = __byte_perm(w[2].x, w[3].x, sel), yb = __byte_perm(w[2].y, w[3].y, sel);
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                mma_f16(o[4 * hf + 0][t], nibbles<0>(xa), nibbles<0>(ya), nibbles<0>(xb), nibbles<0>(yb), pf[x][t]);
                mma_f16(o[4 * hf + 1][t], nibbles<1>(xa), nibbles<1>(ya), nibbles<1>(xb), nibbles<1>(yb), pf[x][t]);
                mma_f16(o[4 * hf + 2][t], nibbles<2>(xa), nibbles<2>(ya), nibbles<2>(xb), nibbles<2>(yb), pf[x][t]);
                mma_f16(o[4 * hf + 3][t], nibbles<3>(xa), nibbles<3>(ya), nibbles<3>(xb), nibbles<3>(yb), pf[x][t]);
              }
            }
          } else {
            uint32_t w[4];
            w[0] = *reinterpret_cast<const uint32_t*>(vb + v0 * (D / 2));
            w[1] = *reinterpret_cast<const uint32_t*>(vb + v1 * (D / 2));
            w[2] = *reinterpret_cast<const uint32_t*>(vb + (8 + v0) * (D / 2));
            w[3] = *reinterpret_cast<const uint32_t*>(vb + (8 + v1) * (D / 2));
            const uint32_t xa = __byte_perm(w[0], w[1], 0x5410u), ya = __byte_perm(w[0], w[1], 0x7632u);
            const uint32_t xb = __byte_perm(w[2], w[3], 0x5410u), yb = __byte_perm(w[2], w[3], 0x7632u);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              mma_f16(o[0][t], nibbles<0>(xa), nibbles<0>(ya), nibbles<0>(xb), nibbles<0>(yb), pf[x][t]);
              mma_f16(o[1][t], nibbles<1>(xa), nibbles<1>(ya), nibbles<1>(xb), nibbles<1>(yb), pf[x][t]);
              mma_f16(o[2][t], nibbles<2>(xa), nibbles<2>(ya), nibbles<2>(xb), nibbles<2>(yb), pf[x][t]);
              mma_f16(o[3][t], nibbles<3>(xa), nibbles<3>(ya), nibbles<3>(xb), nibbles<3>(yb), pf[x][t]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.empty[stage]);
      if (++stage == NS) stage = 0, phase ^= 1;
    }

    // ---- join the warps' sums
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int sft = 4; sft < 32; sft <<= 1) {
          l[t][x] += __shfl_xor_sync(0xFFFFFFFFu, l[t][x], sft);
          z[t][x] += __shfl_xor_sync(0xFFFFFFFFu, z[t][x], sft);
        }
        if ((fresh >> (2 * t + x)) & 1) m[t][x] = kNone;
        if (g == 0) {
          sm.m[warp][8 * t + 2 * c + x] = m[t][x];
          sm.l[warp][8 * t + 2 * c + x] = l[t][x];
          sm.z[warp][8 * t + 2 * c + x] = z[t][x];
        }
      }
    tc::named_bar_sync(1, 32 * kConsumerWarps);
    float f[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = 8 * t + 2 * c + x;
        float mm = sm.m[0][r];
#pragma unroll
        for (int w = 1; w < kConsumerWarps; ++w) mm = fmaxf(mm, sm.m[w][r]);
        f[t][x] = ex2(m[t][x] - mm);
      }
    // Share (warp + p) % kConsumerWarps of the dimensions in phase p.
    constexpr int QT = D / 16 / kConsumerWarps;
    for (int p = 0; p < kConsumerWarps; ++p) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        if (j / QT != (warp + p) % kConsumerWarps) continue;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // accumulator row g (+ 8 for e >= 2) of tile j is this dimension
            const int d = D == 128 ? 16 * g + 8 * (e >> 1) + j : 8 * g + 4 * (e >> 1) + j;
            const int r = 8 * t + 2 * c + (e & 1);
            const float val = (o[j][t][e] * ((j & 1) ? 1048576.f : 16777216.f) + z[t][e & 1]) * f[t][e & 1];
            if (p == 0) sm.o[r][d] = val;
            else sm.o[r][d] += val;
          }
      }
      tc::named_bar_sync(1, 32 * kConsumerWarps);
    }
    const bool whole = sp.whole;
    for (int i = tid; i < rows * (D / 2); i += 32 * kConsumerWarps) {
      const int r = i / (D / 2), d = 2 * (i % (D / 2));
      float mm = sm.m[0][r];
#pragma unroll
      for (int w = 1; w < kConsumerWarps; ++w) mm = fmaxf(mm, sm.m[w][r]);
      float ll = 0.f;
#pragma unroll
      for (int w = 0; w < kConsumerWarps; ++w) ll += sm.l[w][r] * ex2(sm.m[w][r] - mm);
      float x = sm.o[r][d], y = sm.o[r][d + 1];
      if (whole) {
        const int ri = row0 + r, tok = ri / a.G, hd = k.h * a.G + ri % a.G;
        const size_t at = (static_cast<size_t>(k.q.q0) + tok) * a.Hq + hd;
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        x *= inv;
        y *= inv;
        uint32_t b;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(y), "f"(x));
        *reinterpret_cast<uint32_t*>(a.out + at * D + d) = b;
        if (d == 0 && a.lse) a.lse[at] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
      } else {
        float* P = a.part + (static_cast<size_t>(cta) * 2 + (u == u0 ? 0 : 1)) * part_floats<D, RB>();
        *reinterpret_cast<float2*>(P + r * D + d) = make_float2(x, y);
        if (d == 0) {
          P[RB * D + r] = mm;
          P[RB * D + RB + r] = ll;
        }
      }
    }
    if (!whole && sp.first && tid == 0) note_cut(a, cta, ncta, total, k, sp, u, u == u0 ? 0 : 1);
    tc::named_bar_sync(1, 32 * kConsumerWarps);
    u += sp.n;
    if (u < u1) cursor_next(k, a.c, a.q_start, a.base, a.T, a.G, RB, kTile, kItemUnits, sm.cum);
  }
}

// Ring depth: about 43 KB of tiles, so that the CTAs of an SM keep more than
// 100 KB in flight.
template <int D> constexpr int stages() { return D == 128 ? 5 : 9; }

// Rows of a sequence and kv head up to which the kernel here is used.
constexpr int kNarrowRows = 32;

struct Plan {
  int rb, grid;
};

// Row block: the fewest steps of 8 rows (up to 32) that hold a sequence's
// rows, or 128 and the tcgen05 kernel.
Plan plan_of(const kv4_attn_cfg& cfg, const Cache& c) {
  const long long rows = static_cast<long long>(cfg.max_q) * (cfg.n_q_heads / c.Hkv);
  Plan p;
  p.rb = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= kNarrowRows ? 32 : kWideRows;
  p.grid = p.rb == kWideRows ? wide_grid() : sm_count() * ctas_per_sm(p.rb / 8);
  return p;
}

size_t part_bytes(const Plan& p, const Cache& c) { return align_up(static_cast<size_t>(p.grid) * 2 * p.rb * (c.D + 2) * 4, 256); }

template <int D, int NT>
int launch_attend(const AttendArgs& a, const Plan& p, cudaStream_t s) {
  using SM = Smem<D, NT, stages<D>()>;
  const size_t smem = sizeof(SM) + static_cast<size_t>(a.c.S) * 8;
  constexpr auto k = attend_kernel<D, NT, stages<D>()>;
  int st = allow_smem<k>(smem);
  if (st != MOE_OK) return st;
  {
    LaunchScope ls(kProfKv4Attend, s);
    st = launch_k(k, dim3(p.grid), dim3(kThreads), smem, s, false, a);
  }
  if (st != MOE_OK) return st;
  return launch_combine<D, 8 * NT, false>(a, p.grid, s);
}

}  // namespace

int attn_validate(const kv4_attn_cfg* cfg, const Cache& c) {
  if (!cfg || cfg->T < 0 || cfg->n_q_heads < 1 || cfg->max_q < 1) return MOE_ERR_ARG;
  if (cfg->n_q_heads % c.Hkv) return MOE_ERR_ARG;
  if (!(cfg->scale == cfg->scale) || cfg->scale - cfg->scale != 0.f) return MOE_ERR_ARG;
  if (cfg->n_q_heads > 4096 || static_cast<long long>(cfg->T) * cfg->n_q_heads > (1ll << 30)) return MOE_ERR_UNSUPPORTED;
  if (cfg->q_token_stride < 0 || cfg->q_head_stride < 0 || cfg->q_token_stride % 8 || cfg->q_head_stride % 8)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace kv4
}  // namespace moe

extern "C" size_t kv4_attend_workspace(const kv4_cache* cache, const kv4_attn_cfg* cfg) {
  using namespace moe;
  using namespace moe::kv4;
  Cache c;
  if (cache_validate(cache, &c) != MOE_OK || attn_validate(cfg, c) != MOE_OK) return 0;
  const Plan p = plan_of(*cfg, c);
  return part_bytes(p, c) + align_up(static_cast<size_t>(p.grid) * 32, 256);
}

extern "C" int kv4_attend(const kv4_cache* cache, const void* q, const int32_t* q_start, const int32_t* base,
                          const uint64_t* visible, const kv4_attn_cfg* cfg, void* out, float* lse, void* workspace,
                          size_t workspace_bytes, int32_t* dev_err, void* stream) {
  using namespace moe;
  using namespace moe::kv4;
  Cache c;
  int st = cache_validate(cache, &c);
  if (st != MOE_OK || (st = attn_validate(cfg, c)) != MOE_OK) return st;
  if (cfg->T == 0 || c.S == 0) return MOE_OK;
  if (!q || !q_start || !base || !out) return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(q) & 15) || (reinterpret_cast<uintptr_t>(out) & 15) ||
      (reinterpret_cast<uintptr_t>(visible) & 7) ||
      ((reinterpret_cast<uintptr_t>(q_start) | reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(lse)) & 3))
    return MOE_ERR_ARG;
  const size_t need = kv4_attend_workspace(cache, cfg);
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255)) return MOE_ERR_WORKSPACE;
  const Plan p = plan_of(*cfg, c);
  AttendArgs a{c, static_cast<const uint16_t*>(q), cfg->q_token_stride, cfg->q_head_stride, q_start, base, visible,
               static_cast<uint16_t*>(out), lse, cfg->T, cfg->n_q_heads, cfg->n_q_heads / c.Hkv, cfg->scale * kLog2e,
               static_cast<float*>(workspace),
               reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + part_bytes(p, c)), dev_err};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.rb == kWideRows) return wide_launch(a, p.grid, s);
  if (c.D == 128)
    return p.rb == 8 ? launch_attend<128, 1>(a, p, s) : p.rb == 16 ? launch_attend<128, 2>(a, p, s) : launch_attend<128, 4>(a, p, s);
  return p.rb == 8 ? launch_attend<64, 1>(a, p, s) : p.rb == 16 ? launch_attend<64, 2>(a, p, s) : launch_attend<64, 4>(a, p, s);
}
