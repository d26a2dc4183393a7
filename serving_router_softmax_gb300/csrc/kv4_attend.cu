// kv4_attend: attention of a batch's new tokens over the 4-bit paged cache.
//
// One pass over the cache with a running softmax maximum and sum, in the
// transposed form: scores S^T [slots x query rows] = C_k Q^T with the key codes as
// the row operand straight from their nibbles, output O^T [D x query rows] =
// C_v^T P^T with the value codes.  The query rows of a kv head (its new tokens
// times the query heads that share it) are the narrow side, in blocks of 8, so
// a single decoded token of 8 query heads wastes nothing.  More blocks read the
// cache again, out of L2 where it fits; from where that costs more, the
// kernel of kv4_attend_wide.cu takes over (see wide_pays).
//
// Each CTA owns an even share of all (sequence, head, row block, tile) units;
// a producer warp keeps a ring of tiles in flight (bulk copies), two consumer
// warps take 32 slots of each tile, two groups of 16 beside each other, whose
// chains of products and exponentials fill each other's waits.  An item cut
// between CTAs leaves its partial sums in the workspace and the combine kernel
// joins them in CTA order, so results do not depend on timing.
//
// Bound by memory for long contexts (48 sequences of 8k to 32k slots, 64 query
// heads on 8: 1.09 GB in 201 us with the joining, 79% of the copy rate); what keeps it
// from more is the unpacking's integer operations (the ALU pipe is 59% busy, the issue slots 55%) and
// the registers, which hold four CTAs an SM.
#include "kv4_attend.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr int kRows = 8;
constexpr int kConsumerWarps = 2;
constexpr int kThreads = 32 * (kConsumerWarps + 1);
constexpr int kGroups = kTile / 16 / kConsumerWarps;  // 16-slot groups of a tile that a warp takes
constexpr int kMinUnits = 1;
constexpr int kCtasPerSm = 4;  // the above on the device: 199 us; with five, which spill registers, 306, with three 250

// About 43 KB of tiles in flight a CTA.
template <int D> constexpr int stages() { return D == 128 ? 5 : 9; }

template <int D>
struct Smem {
  static constexpr int NS = stages<D>();
  Tile<D> st[NS];
  uint4 frag[(D / 32) * 32];
  float o[kRows][D + 4];
  float cq[kRows], cqs[kRows];
  float m[kConsumerWarps][kRows], l[kConsumerWarps][kRows], z[kConsumerWarps][kRows];
  uint64_t mask[kRows];
  uint64_t full[NS], empty[NS];
  uint32_t groups[NS];  // bit g: the page of slots 16g..16g+15 of the tile is valid
  long long scratch[32];
  int abort, never;
  long long cum[1];     // [S + 1]
};

// MMA layouts: see kv4.cuh.
template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) attend_kernel(const AttendArgs a) {
  constexpr int NS = Smem<D>::NS;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(&sm.full[i], arrivals_of_stage(a, i));
      tc::mbar_init(&sm.empty[i], kConsumerWarps);
    }
    sm.abort = sm.never = 0;
    tc::fence_mbar_init();
  }
  pdl_wait();
  build_units(a.c, a.q_start, a.base, a.T, a.G, kRows, kTile, kItemUnits, sm.cum, sm.scratch, a.dev_err, blockIdx.x == 0);
  pdl_trigger();
  const long long total = sm.cum[a.c.S];
  const int ncta = used_ctas(total, kMinUnits), cta = blockIdx.x;
  const Shares shares(total, max(ncta, 1));
  const long long u0 = cta < ncta ? shares.begin(cta) : 0, u1 = cta < ncta ? shares.begin(cta + 1) : 0;
  volatile int* abort_flag = &sm.abort;
  Cursor k;
  if (u0 < u1) cursor_at(k, a.c, a.q_start, a.base, a.T, a.G, kRows, kTile, kItemUnits, sm.cum, u0);

  if (warp == kConsumerWarps) {
    // ---------------------------------------------------------- producer
    TileLoader<D> loader(a.c);
    int stage = 0, issued = 0;  // issued: up to NS
    uint32_t phase = 0;
    bool dead = false;
    for (long long u = u0; u < u1 && !dead;) {
      const Span sp = span_of<kRows>(a, k, u, u1);
      const int tiles = copied_tiles(a, sp, u + sp.n == u1);
      for (int it = 0; it < tiles; ++it) {
        if (__any_sync(0xFFFFFFFFu, !tc::mbar_wait_bounded(&sm.empty[stage], phase ^ 1, abort_flag, kWaitBudgetNs))) {
          *abort_flag = 1;
          dead = true;
          break;
        }
        loader.load(a, k, sm.st[stage], &sm.groups[stage], &sm.full[stage]);
        ++k.tile;
        issued = min(issued + 1, NS);
        if (++stage == NS) stage = 0, phase ^= 1;
      }
      u += sp.n;
      if (u < u1) cursor_next(k, a.c, a.q_start, a.base, a.T, a.G, kRows, kTile, kItemUnits, sm.cum);
    }
    // A consumer may give up long after the last copy has been started, so this warp stays until they are done.
    tc::named_bar_sync(2, kThreads);
    if (*abort_flag) {
      // Copies in flight land before the CTA's shared memory goes.
      for (int i = 0; i < issued; ++i) {
        if (--stage < 0) stage = NS - 1, phase ^= 1;
        tc::mbar_wait_bounded(&sm.full[stage], phase, &sm.never, 100000000ull);
      }
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
  int stage = 0;
  uint32_t phase = 0;
  bool lost = false;  // a tile has not come: no later one is looked at, nor a stage freed that may still be filling
  if (tid < 8) a.meta[static_cast<size_t>(cta) * 8 + tid] = 0;
  for (long long u = u0; u < u1;) {
    const Span sp = span_of<kRows>(a, k, u, u1);
    const int n = sp.tiles, row0 = sp.row0, rows = sp.rows;
    if (n == 0) {
      u += sp.n;
      if (u < u1) cursor_next(k, a.c, a.q_start, a.base, a.T, a.G, kRows, kTile, kItemUnits, sm.cum);
      continue;
    }
    prep_q<D>([&](int r) { return r < rows ? q_row(a, k.q, k.h, row0 + r) : (const uint16_t*)nullptr; }, kRows, a.scale_log2,
              sm.frag, sm.cq, sm.cqs, tid, 32 * kConsumerWarps);
    if (tid < kRows && a.visible) sm.mask[tid] = a.visible[k.q.q0 + (row0 + min(tid, rows - 1)) / a.G];
    if (a.visible && k.q.nq > kMaxTree && tid == 0) flag_error(a.dev_err, MOE_DEV_CAPACITY);
    tc::named_bar_sync(1, 32 * kConsumerWarps);

    // This lane's columns: rows 2c and 2c + 1.
    float o[D / 16][4], m[2] = {}, l[2] = {}, z[2] = {};
    const float cq[2] = {sm.cq[2 * c], sm.cq[2 * c + 1]}, cqs[2] = {sm.cqs[2 * c], sm.cqs[2 * c + 1]};
    uint32_t fresh = 3;  // columns that have seen nothing
#pragma unroll
    for (int j = 0; j < D / 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

    for (int it = 0; it < n && !lost; ++it) {
      const int j0 = (k.tile + it) * kTile + 16 * kGroups * warp;  // first slot of this warp's groups
      if (__any_sync(0xFFFFFFFFu, !tc::mbar_wait_bounded(&sm.full[stage], phase, abort_flag, kWaitBudgetNs))) {
        *abort_flag = 1;
        lost = true;
        break;
      }
      const uint8_t* st = sm.st[stage].b;
      const uint32_t groups = sm.groups[stage] >> (kGroups * warp);
      const bool edge = j0 + 16 * kGroups > k.q.base || (groups & ((1u << kGroups) - 1)) != (1u << kGroups) - 1;
      float d[kGroups][4], rs[kGroups][2], zr[kGroups][2];
#pragma unroll
      for (int x = 0; x < kGroups; ++x) {
        uint32_t ka[D / 32], kb[D / 32];
        load_k_words<D>(st + k_at[x] + s0 * (D / 2), c, ka);
        load_k_words<D>(st + k_at[x] + s1 * (D / 2), c, kb);
        const uint2 ra = *reinterpret_cast<const uint2*>(st + p_at[x] + s0 * 8);
        const uint2 rb = *reinterpret_cast<const uint2*>(st + p_at[x] + s1 * 8);
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
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        qk_16x8<D>(acc, ka, kb, sm.frag);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int kk = e >> 1, y = e & 1;
          d[x][e] = fmaf(ks[kk], acc[e] * cq[y], fmaf(kz[kk], cqs[y], lv[kk] - m[y]));
        }
      }
      // Where slots may be out of sight (or out of range): their exponents are -inf, and
      // what their parameters hold (NaN, say) must not reach the sums.
      uint32_t seen = 0xFFFFFFFFu;  // bit 4 x + e
      if (edge) {
        seen = 0;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int r = 2 * c + y;
#pragma unroll
          for (int x = 0; x < kGroups; ++x) {
            uint64_t v = 0;
            if ((groups >> x) & 1)
              v = sees(k.q, a.visible != nullptr, sm.mask[r], (row0 + min(r, rows - 1)) / a.G, j0 + 16 * x);
            if ((v >> s0) & 1) seen |= 1u << (4 * x + y);
            else d[x][y] = -INFINITY;
            if ((v >> s1) & 1) seen |= 1u << (4 * x + 2 + y);
            else d[x][2 + y] = -INFINITY;
          }
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int x = 0; x < kGroups; ++x) top = max3(max3(top, d[x][0], d[x][1]), d[x][2], d[x][3]);
      if (__any_sync(0xFFFFFFFFu, top > kLazy || fresh != 0)) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float mx = -INFINITY;
#pragma unroll
          for (int x = 0; x < kGroups; ++x) mx = max3(mx, d[x][y], d[x][2 + y]);
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
          // A row's first visible slots set its maximum; later ones only raise it.
          const bool first = (fresh >> y) & 1, none = mx == -INFINITY;
          const float by = none ? 0.f : first ? mx : fmaxf(mx, 0.f);
          const float f = first ? 1.f : ex2(-by);
          if (!none) fresh &= ~(1u << y);
          m[y] += by;
          l[y] *= f;
          z[y] *= f;
#pragma unroll
          for (int x = 0; x < kGroups; ++x) {
            d[x][y] -= by;
            d[x][2 + y] -= by;
          }
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            o[j][y] *= f;
            o[j][2 + y] *= f;
          }
        }
      }
      uint2 pf[kGroups];
#pragma unroll
      for (int x = 0; x < kGroups; ++x) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = ex2(d[x][e]);
          if (!edge || ((seen >> (4 * x + e)) & 1)) {
            l[e & 1] = fmaf(p[e], rs[x][e >> 1], l[e & 1]);
            z[e & 1] = fmaf(p[e], zr[x][e >> 1], z[e & 1]);
          }
        }
        pf[x] = make_uint2(transpose_8x8(pack_h2(p[0], p[1])), transpose_8x8(pack_h2(p[2], p[3])));
      }
      // Values: lane (g, c) owns k indices 2c, 2c+1, 2c+8, 2c+9 and the
      // dimensions g * D/8 ..; one byte permute pairs two slots' halves.
      const int v0 = slot_of_row(2 * c), v1 = slot_of_row(2 * c + 1);
#pragma unroll
      for (int x = 0; x < kGroups; ++x) {
        const uint8_t* vb = st + v_at[x] + g * (D / 16);
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
            mma_f16(o[4 * hf + 0], nibbles<0>(xa), nibbles<0>(ya), nibbles<0>(xb), nibbles<0>(yb), pf[x]);
            mma_f16(o[4 * hf + 1], nibbles<1>(xa), nibbles<1>(ya), nibbles<1>(xb), nibbles<1>(yb), pf[x]);
            mma_f16(o[4 * hf + 2], nibbles<2>(xa), nibbles<2>(ya), nibbles<2>(xb), nibbles<2>(yb), pf[x]);
            mma_f16(o[4 * hf + 3], nibbles<3>(xa), nibbles<3>(ya), nibbles<3>(xb), nibbles<3>(yb), pf[x]);
          }
        } else {
          uint32_t w[4];
          w[0] = *reinterpret_cast<const uint32_t*>(vb + v0 * (D / 2));
          w[1] = *reinterpret_cast<const uint32_t*>(vb + v1 * (D / 2));
          w[2] = *reinterpret_cast<const uint32_t*>(vb + (8 + v0) * (D / 2));
          w[3] = *reinterpret_cast<const uint32_t*>(vb + (8 + v1) * (D / 2));
          const uint32_t xa = __byte_perm(w[0], w[1], 0x5410u), ya = __byte_perm(w[0], w[1], 0x7632u);
          const uint32_t xb = __byte_perm(w[2], w[3], 0x5410u), yb = __byte_perm(w[2], w[3], 0x7632u);
          mma_f16(o[0], nibbles<0>(xa), nibbles<0>(ya), nibbles<0>(xb), nibbles<0>(yb), pf[x]);
          mma_f16(o[1], nibbles<1>(xa), nibbles<1>(ya), nibbles<1>(xb), nibbles<1>(yb), pf[x]);
          mma_f16(o[2], nibbles<2>(xa), nibbles<2>(ya), nibbles<2>(xb), nibbles<2>(yb), pf[x]);
          mma_f16(o[3], nibbles<3>(xa), nibbles<3>(ya), nibbles<3>(xb), nibbles<3>(yb), pf[x]);
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.empty[stage]);
      if (++stage == NS) stage = 0, phase ^= 1;
    }

    // ---- join the warps' sums
#pragma unroll
    for (int y = 0; y < 2; ++y) {
#pragma unroll
      for (int sft = 4; sft < 32; sft <<= 1) {
        l[y] += __shfl_xor_sync(0xFFFFFFFFu, l[y], sft);
        z[y] += __shfl_xor_sync(0xFFFFFFFFu, z[y], sft);
      }
      if ((fresh >> y) & 1) m[y] = kNone;
      if (g == 0) {
        sm.m[warp][2 * c + y] = m[y];
        sm.l[warp][2 * c + y] = l[y];
        sm.z[warp][2 * c + y] = z[y];
      }
    }
    tc::named_bar_sync(1, 32 * kConsumerWarps);
    float f[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float mm = sm.m[0][2 * c + y];
#pragma unroll
      for (int w = 1; w < kConsumerWarps; ++w) mm = fmaxf(mm, sm.m[w][2 * c + y]);
      f[y] = ex2(m[y] - mm);
    }
    // Share (warp + p) % kConsumerWarps of the dimensions in phase p.
    constexpr int QT = D / 16 / kConsumerWarps;
    for (int p = 0; p < kConsumerWarps; ++p) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        if (j / QT != (warp + p) % kConsumerWarps) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // accumulator row g (+ 8 for e >= 2) of tile j is this dimension
          const int dim = D == 128 ? 16 * g + 8 * (e >> 1) + j : 8 * g + 4 * (e >> 1) + j;
          const int r = 2 * c + (e & 1);
          const float val = (o[j][e] * ((j & 1) ? 1048576.f : 16777216.f) + z[e & 1]) * f[e & 1];
          if (p == 0) sm.o[r][dim] = val;
          else sm.o[r][dim] += val;
        }
      }
      tc::named_bar_sync(1, 32 * kConsumerWarps);
    }
    for (int i = tid; i < rows * (D / 2); i += 32 * kConsumerWarps) {
      const int r = i / (D / 2), dim = 2 * (i % (D / 2));
      float mm = sm.m[0][r];
#pragma unroll
      for (int w = 1; w < kConsumerWarps; ++w) mm = fmaxf(mm, sm.m[w][r]);
      float ll = 0.f;
#pragma unroll
      for (int w = 0; w < kConsumerWarps; ++w) ll += sm.l[w][r] * ex2(sm.m[w][r] - mm);
      float x = sm.o[r][dim], y = sm.o[r][dim + 1];
      if (sp.whole) {
        const int ri = row0 + r, tok = ri / a.G, hd = k.h * a.G + ri % a.G;
        const size_t at = (static_cast<size_t>(k.q.q0) + tok) * a.Hq + hd;
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        x *= inv;
        y *= inv;
        uint32_t b;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(y), "f"(x));
        *reinterpret_cast<uint32_t*>(a.out + at * D + dim) = b;
        if (dim == 0 && a.lse) a.lse[at] = ll == 0.f ? -INFINITY : (mm + lg2(ll)) * kLn2;
      } else {
        float* P = a.part + (static_cast<size_t>(cta) * 2 + (u == u0 ? 0 : 1)) * part_floats<D, kRows>();
        *reinterpret_cast<float2*>(P + r * D + dim) = make_float2(x, y);
        if (dim == 0) {
          P[kRows * D + r] = mm;
          P[kRows * D + kRows + r] = ll;
        }
      }
    }
    if (!sp.whole && sp.first && tid == 0) note_cut(a, cta, shares, k, sp, u, u == u0 ? 0 : 1);
    tc::named_bar_sync(1, 32 * kConsumerWarps);
    u += sp.n;
    if (u < u1) cursor_next(k, a.c, a.q_start, a.base, a.T, a.G, kRows, kTile, kItemUnits, sm.cum);
  }
  tc::named_bar_sync(2, kThreads);  // (the producer waits for it)
}

// Whether blocks of 128 rows on the tcgen05 kernel take less time than blocks of
// 8 here, which read the cache once a block.  Measured on the device in us
// (here / wide), rows of a sequence and kv head against sequences x longest
// context (lengths and tokens ragged but in the last column, 8 kv heads, the
// table as wide as the longest context):
//            rows    2 x 2,000     1 x 30,000     16 x 8,192    16 x 8,192, all full
//   D = 128    24   13.8 / 20.2   30.2 / 47.4    68.0 /  83.9     87.1 / 127.5
//              32   14.0 / 20.7   33.7 / 47.9    69.2 /  79.1    112.0 / 127.8
//              40   13.8 / 20.4   39.4 / 48.8    90.4 /  89.6    135.8 / 128.8
//              48   14.0 / 20.9   44.1 / 49.1   111.2 /  85.3    163.0 / 129.3
//              64   16.0 / 21.4   54.0 / 49.2   183.6 /  93.8    213.2 / 130.8
//             128   20.7 / 24.3   98.1 / 54.1   294.8 / 101.1    414.0 / 139.8
//   D = 64     24   11.9 / 17.8   23.8 / 42.2    45.5 /  67.9     61.8 / 106.3
//              32   12.0 / 18.1   26.4 / 42.3    47.1 /  63.4     78.4 / 106.2
//              40   12.0 / 17.9   30.3 / 43.0    60.7 /  71.5     95.8 / 106.5
//              48   11.8 / 18.0   33.6 / 43.0    73.6 /  67.7    113.6 / 106.5
//              64   13.0 / 18.2   40.6 / 43.1   115.6 /  73.7    148.5 / 106.8
//             128   16.1 / 21.1   71.1 / 46.5   192.7 /  71.7    288.0 / 111.0
// The rule below takes up to 18% more there than the better one.  The lengths are
// device data, so it goes by the slots that the table can hold: a table far
// wider than what is in use costs more (32 rows, 4 x 2,000 slots, a table of
// 131,072 slots: 22.0 us where the kernel here takes 14.2).
bool wide_pays(long long rows, const Cache& c) {
  const double slots = static_cast<double>(c.S) * c.Hkv * (static_cast<double>(c.width) * c.page_size);
  return rows > 24 && slots * static_cast<double>(rows - 24) * c.D >= 576e6;
}

struct Plan {
  int rb, grid;
};

Plan plan_of(const kv4_attn_cfg& cfg, const Cache& c) {
  const bool wide = wide_pays(static_cast<long long>(cfg.max_q) * (cfg.n_q_heads / c.Hkv), c);
  return wide ? Plan{kWideRows, wide_grid()} : Plan{kRows, kCtasPerSm * sm_count()};
}

size_t part_bytes(const Plan& p, const Cache& c) { return align_up(static_cast<size_t>(p.grid) * 2 * p.rb * (c.D + 2) * 4, 256); }

template <int D>
int launch_attend(const AttendArgs& a, const Plan& p, cudaStream_t s) {
  const size_t smem = sizeof(Smem<D>) + static_cast<size_t>(a.c.S) * 8;
  int st = allow_smem<attend_kernel<D>>(smem);
  if (st != MOE_OK) return st;
  {
    LaunchScope ls(kProfKv4Attend, s);
    st = launch_k(attend_kernel<D>, dim3(p.grid), dim3(kThreads), smem, s, false, a);
  }
  if (st != MOE_OK) return st;
  return launch_combine<D, kRows, false>(a, p.grid, s);
}

}  // namespace

int attn_validate(const kv4_attn_cfg* cfg, const Cache& c) {
  if (!cfg || cfg->T < 0 || cfg->n_q_heads < 1 || cfg->max_q < 1) return MOE_ERR_ARG;
  if (cfg->n_q_heads % c.Hkv) return MOE_ERR_ARG;
  if (!(cfg->scale == cfg->scale) || cfg->scale - cfg->scale != 0.f) return MOE_ERR_ARG;
  if (cfg->n_q_heads > 4096 || static_cast<long long>(cfg->T) * cfg->n_q_heads > (1ll << 30)) return MOE_ERR_UNSUPPORTED;
  if (!stride_ok(cfg->q_token_stride, cfg->T, 8) || !stride_ok(cfg->q_head_stride, cfg->n_q_heads, 8))
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
  const int stall = test_stall_mask();
  const int withhold = stall & MOE_TEST_STALL_KV4_ATTEND ? kWithholdLast : stall & MOE_TEST_STALL_KV4_FIRST ? kWithholdFirst : 0;
  AttendArgs a{c, static_cast<const uint16_t*>(q), cfg->q_token_stride, cfg->q_head_stride, q_start, base, visible,
               static_cast<uint16_t*>(out), lse, cfg->T, cfg->n_q_heads, cfg->n_q_heads / c.Hkv, cfg->scale * kLog2e,
               static_cast<float*>(workspace),
               reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + part_bytes(p, c)), dev_err, withhold};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.rb == kWideRows) return wide_launch(a, p.grid, s);
  return c.D == 128 ? launch_attend<128>(a, p, s) : launch_attend<64>(a, p, s);
}
