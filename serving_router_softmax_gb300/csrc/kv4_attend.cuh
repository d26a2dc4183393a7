// What the two kv4_attend kernels share: arguments, the tile producer, the
// visibility of a tile's slots, the partial sums of items cut between CTAs.
#pragma once

#include "kv4.cuh"
#include "kv4_sched.cuh"

namespace moe {
namespace kv4 {

constexpr uint64_t kWaitBudgetNs = 2000000000ull;  // 2 s
constexpr float kLazy = 8.f;  // the running maximum may lag by this much (log2) before sums are rescaled

struct AttendArgs {
  Cache c;
  const uint16_t* q;
  long long q_ts, q_hs;
  const int32_t* q_start;
  const int32_t* base;
  const uint64_t* visible;
  uint16_t* out;
  float* lse;
  int32_t T, Hq, G;
  float scale_log2;
  float* part;     // [CTAs][2] partial sums of row blocks, see part_floats
  int32_t* meta;   // [CTAs][8]: a cut item that starts in this CTA
  int32_t* dev_err;
  int32_t withhold;  // test hook: each CTA's last or first tile does not come, so that the wait for it runs out
};
constexpr int kWithholdLast = 1, kWithholdFirst = 2;

// One row block's partial sums: outputs [RB][D] (the wide kernel: [D][RB], columns as they lie in TMEM), running
// maxima [RB], sums [RB].
template <int D, int RB>
constexpr size_t part_floats() { return static_cast<size_t>(RB) * (D + 2); }

// Query row r of an item's sequence and head.
__device__ __forceinline__ const uint16_t* q_row(const AttendArgs& a, const SeqShape& q, int h, int r) {
  const int i = r / a.G, g = r - i * a.G;
  return a.q + (q.q0 + i) * a.q_ts + static_cast<long long>(h * a.G + g) * a.q_hs;
}

__device__ __forceinline__ uint64_t low_ones(long long n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; }

// Which of the 64 slots from j0 on new token i (mask bits `bits`, if there
// are masks) sees, as far as lengths and masks go.
__device__ __forceinline__ uint64_t sees(const SeqShape& q, bool masks, uint64_t bits, int i, int j0) {
  uint64_t v;
  if (masks) {
    const int d = j0 - q.base;  // new slot of the first one
    v = d >= 64 ? 0 : d >= 0 ? bits >> d : d <= -64 ? ~0ull : low_ones(-d) | (bits << -d);
  } else {
    v = low_ones(static_cast<long long>(q.base) + i + 1 - j0);
  }
  return v & low_ones(static_cast<long long>(q.total) - j0);
}

// Bit 16 g + x of the result: slot group g of the tile lies in a valid page.
__device__ __forceinline__ uint64_t group_mask(uint32_t groups) {
  uint64_t m = 0;
#pragma unroll
  for (int g = 0; g < 4; ++g) m |= (groups >> g & 1) ? 0xFFFFull << (16 * g) : 0ull;
  return m;
}

// A tile in shared memory: one segment per page (64 slots of it at most),
// laid out as a page block is: K codes, V codes, parameters.  So a page of up
// to 64 slots comes in one copy.
template <int D>
struct Tile {
  alignas(128) uint8_t b[kTile * (D + 8)];
};

// Where a tile's rows lie.
template <int D>
struct TileMap {
  int seg_log2, seg;
  __device__ __forceinline__ explicit TileMap(const Cache& c) : seg_log2(min(c.page_log2, 6)), seg(1 << seg_log2) {}
  __device__ __forceinline__ int base(int r) const { return (r >> seg_log2) * (seg * (D + 8)); }
  __device__ __forceinline__ int k(int r) const { return base(r) + (r & (seg - 1)) * (D / 2); }
  __device__ __forceinline__ int v(int r) const { return base(r) + (seg + (r & (seg - 1))) * (D / 2); }
  __device__ __forceinline__ int p(int r) const { return base(r) + seg * D + (r & (seg - 1)) * 8; }
};

// CTAs that share `total` units: at least kMinUnits each, so that the sums they
// leave to be joined stay small beside their work, and at most all.
__device__ __forceinline__ int used_ctas(long long total, int min_units) {
  const long long n = total / min_units;
  return static_cast<int>(n < 1 ? (total > 0) : n < gridDim.x ? n : gridDim.x);
}

// Units that an item costs beyond its tiles (query rows in, sums out).  With 1, 2, 3 and 4, on the device: 4 trees of up to 7
// tokens on up to 8192 slots 38.4, 35.2, 34.9 and 35.0 us, 48 tokens on up to 32,768 each 206.4, 202.4, 199.1 and 198.6.
constexpr int kItemUnits = 3;

// Page lookup and copies of tiles, one warp.  A lone warp's instructions wait
// for each other, so what does not change from tile to tile is kept.
template <int D>
struct TileLoader {
  int seg_log2, nseg, lane;
  int s = -1, h = -1, cached_at = 0, cached = -1;
  const uint8_t* head;     // block of page 0, head h
  size_t stride;           // bytes from page to page

  __device__ __forceinline__ explicit TileLoader(const Cache& c) {
    seg_log2 = min(c.page_log2, 6);
    nseg = kTile >> seg_log2;
    lane = threadIdx.x & 31;
    stride = static_cast<size_t>(c.Hkv) * c.block_bytes();
  }

  // Starts the copies of the cursor's tile into st; *groups gets the valid
  // slot groups before `full` completes.  Whole warp.
  __device__ __forceinline__ void load(const AttendArgs& a, const Cursor& k, Tile<D>& st, uint32_t* groups, uint64_t* full) {
    const int p0 = (k.tile * kTile) >> a.c.page_log2;
    if (k.s != s || k.h != h || p0 < cached_at || p0 + nseg > cached_at + 32) {
      // One table entry per lane, 32 pages ahead.
      s = k.s;
      h = k.h;
      cached_at = p0;
      cached = page_of(a.c, k.s, (p0 + lane) << a.c.page_log2);
      head = a.c.pages + static_cast<size_t>(k.h) * a.c.block_bytes();
    }
    const int i = lane & (nseg - 1);
    int page = __shfl_sync(0xFFFFFFFFu, cached, p0 + i - cached_at);
    const bool want = lane < nseg && k.tile * kTile + (i << seg_log2) < k.q.total;
    const bool have = want && page >= 0;
    const uint32_t hv = __ballot_sync(0xFFFFFFFFu, have);
    const uint32_t bytes = (D + 8) << seg_log2;
    if (lane == 0) {
      uint32_t gr = 15;
      if (__popc(hv) < nseg) gr = 0;
      for (uint32_t x = gr ? 0 : hv; x; x &= x - 1) gr |= ((1u << (1 << (seg_log2 - 4))) - 1u) << ((__ffs(x) - 1) << (seg_log2 - 4));
      *groups = gr;
      tc::mbar_arrive_expect_tx(full, __popc(hv) * bytes);
    }
    if (want && page < 0) flag_error(a.dev_err, MOE_DEV_BAD_ID);
    __syncwarp();
    if (!have) return;
    const uint8_t* b = head + page * stride;
    uint8_t* dst = st.b + lane * bytes;
    if (a.c.page_log2 <= 6) {
      bulk_copy(dst, b, bytes, full);
    } else {
      const int r0 = (k.tile * kTile) & (a.c.page_size - 1);
      bulk_copy(dst, b + r0 * (D / 2), kTile * (D / 2), full);
      bulk_copy(dst + kTile * (D / 2), b + (a.c.page_size + r0) * (D / 2), kTile * (D / 2), full);
      bulk_copy(dst + kTile * D, b + a.c.page_size * D + r0 * 8, kTile * 8, full);
    }
  }
};

// The part of the unit order that a CTA does in one item.
struct Span {
  int row0, rows;    // the block's query rows
  int need;          // tiles that one of its rows can see
  int n, tiles;      // units of the item that are this CTA's, tiles among them
  bool first, whole; // it has the item's first tile; all of them
};
template <int RB>
__device__ __forceinline__ Span span_of(const AttendArgs& a, const Cursor& k, long long u, long long u1) {
  Span s;
  s.n = static_cast<int>(u1 - u < k.nt - k.tile ? u1 - u : k.nt - k.tile);
  s.row0 = k.rb * RB;
  s.rows = min(RB, k.q.nq * a.G - s.row0);
  const int seen = a.visible ? k.q.total : min(k.q.total, k.q.base + (s.row0 + s.rows - 1) / a.G + 1);
  s.need = (seen + kTile - 1) / kTile;
  s.tiles = max(0, min(s.n, s.need - k.tile));
  s.first = k.tile == 0;
  s.whole = s.first && s.tiles == s.need;
  return s;
}

// Arrivals that fill stage i of the tile ring; with the test hook on the first tile its stage never looks full.
__device__ __forceinline__ uint32_t arrivals_of_stage(const AttendArgs& a, int i) {
  return a.withhold == kWithholdFirst && i == 0 ? 2 : 1;
}

// Tiles of a span to copy; the test hook keeps back the last one of the CTA's last span (`last`).
__device__ __forceinline__ int copied_tiles(const AttendArgs& a, const Span& s, bool last) {
  return s.tiles - (a.withhold == kWithholdLast && last && s.tiles > 0 ? 1 : 0);
}

// Notes an item that starts in this CTA and ends in a later one; u is the item's first unit.
__device__ __forceinline__ void note_cut(const AttendArgs& a, int cta, const Shares& shares, const Cursor& k, const Span& s,
                                         long long u, int slot) {
  int32_t* M = a.meta + static_cast<size_t>(cta) * 8;
  M[1] = k.s;
  M[2] = k.h;
  M[3] = s.row0;
  M[4] = s.rows;
  M[5] = shares.of(u + s.need - 1);  // the CTA that owns the item's last tile
  M[6] = slot;
  M[0] = 1;
}

// Joins the partial sums of the item that starts in CTA blockIdx.x and ends
// in a later one: rows 8 * blockIdx.y to + 7 of it, eight dimensions a thread,
// the contributors dealt out to kShare threads whose sums are added in order, so
// results do not depend on timing.  The maximum comes first, so that the loads
// of the second loop do not wait for each other.
// kCols: outputs lie as [D][RB], column n * (D / 8) + w being dimension 8 w + n.
template <int D, int RB, bool kCols, int kShare>
__global__ void __launch_bounds__(D * kShare) combine_kernel(const AttendArgs a) {
  constexpr int W = D / 8;
  constexpr size_t PF = part_floats<D, RB>();
  __shared__ float part[kShare - 1][9][D];
  pdl_wait();
  pdl_trigger();
  const int c0 = blockIdx.x, tid = threadIdx.x % D, share = threadIdx.x / D;
  const int4 M = *reinterpret_cast<const int4*>(a.meta + static_cast<size_t>(c0) * 8);
  const int4 M2 = *reinterpret_cast<const int4*>(a.meta + static_cast<size_t>(c0) * 8 + 4);
  if (M.x == 0 || blockIdx.y * 8 >= M2.x) return;
  const int r = blockIdx.y * 8 + (kCols ? tid & 7 : tid / W), w = kCols ? tid >> 3 : tid % W;
  // Contributor 0 left its sums in place M2.z of CTA c0, contributor i > 0 in place 0 of CTA c0 + i.
  const int n = M2.y - c0 + 1;
  const float* P = a.part + static_cast<size_t>(c0) * 2 * PF;
  const float* P0 = P + M2.z * PF;
  const float* ms = P + RB * D + r;
  float m = P0[RB * D + r];
#pragma unroll 4
  for (int i = 1; i < n; ++i) m = fmaxf(m, ms[2 * PF * i]);
  float l = 0.f, v[8] = {};
#pragma unroll 2
  for (int i = share; i < n; i += kShare) {
    const float* Q = i ? P + 2 * PF * i : P0;
    const float f = ex2(Q[RB * D + r] - m);
    l = fmaf(Q[RB * D + RB + r], f, l);
    float q[8];
    if (kCols) {
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = Q[(j * W + w) * RB + r];
    } else {
      const float4 x = *reinterpret_cast<const float4*>(Q + r * D + 8 * w), y = *reinterpret_cast<const float4*>(Q + r * D + 8 * w + 4);
      q[0] = x.x, q[1] = x.y, q[2] = x.z, q[3] = x.w, q[4] = y.x, q[5] = y.y, q[6] = y.z, q[7] = y.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fmaf(q[j], f, v[j]);
  }
  if (share > 0) {
    part[share - 1][8][tid] = l;
#pragma unroll
    for (int j = 0; j < 8; ++j) part[share - 1][j][tid] = v[j];
  }
  __syncthreads();
  if (share > 0 || r >= M2.x) return;
#pragma unroll
  for (int x = 0; x < kShare - 1; ++x) {
    l += part[x][8][tid];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += part[x][j][tid];
  }
  const int ri = M.w + r, tok = ri / a.G, hd = M.z * a.G + ri - tok * a.G;
  const size_t at = (static_cast<size_t>(a.q_start[M.y]) + tok) * a.Hq + hd;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b[j]) : "f"(v[2 * j + 1] * inv), "f"(v[2 * j] * inv));
  *reinterpret_cast<uint4*>(a.out + at * D + 8 * w) = make_uint4(b[0], b[1], b[2], b[3]);
  if (w == 0 && a.lse) a.lse[at] = l == 0.f ? -INFINITY : (m + lg2(l)) * kLn2;
}

template <int D, int RB, bool kCols>
int launch_combine(const AttendArgs& a, int grid, cudaStream_t s) {
  // A chain of loads per share: four shares read a long list sooner than two (one decoded token over 777 slots: 10.4 us
  // on the device against 11.4, 4 trees on up to 8192 34.8 against 38.9), eight cost more in idle CTAs than they save
  // (10.4 and 37.3; 48 sequences: 204.8 us against 199.1).
  constexpr int kShare = 4;
  LaunchScope ls(kProfKv4Attend, s);
  return launch_k(combine_kernel<D, RB, kCols, kShare>, dim3(grid, RB / 8), dim3(D * kShare), 0, s, true, a);
}

constexpr int kWideRows = 128;
// The tensor-core kernel (tcgen05) for row blocks of 128.
int wide_grid();
int wide_launch(const AttendArgs& a, int grid, cudaStream_t s);  // with its combine kernel

}  // namespace kv4
}  // namespace moe
