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
};

// One row block's partial sums: outputs [RB][D], running maxima [RB], sums [RB].
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

__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   tc::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}

// A tile as it lies in the cache: codes and parameters of 64 slots.
template <int D>
struct Tile {
  alignas(128) uint8_t k[kTile * D / 2];
  uint8_t v[kTile * D / 2];
  uint8_t p[kTile * 8];
};

// Page lookup and copies of tiles, one warp.
template <int D>
struct TileLoader {
  int cached_s = -1, cached_at = 0, cached = -1;

  // Starts the copies of the cursor's tile into st; *groups gets the valid
  // slot groups before `full` completes.  Whole warp.
  __device__ __forceinline__ void load(const AttendArgs& a, const Cursor& k, Tile<D>& st, uint32_t* groups, uint64_t* full) {
    const int lane = threadIdx.x & 31;
    const int seg_rows = a.c.page_size < kTile ? a.c.page_size : kTile;
    const int nseg = kTile / seg_rows;
    // One table entry per lane, 32 pages ahead.
    const int p0 = (k.tile * kTile) >> a.c.page_log2;
    if (k.s != cached_s || p0 < cached_at || p0 + nseg > cached_at + 32) {
      cached_s = k.s;
      cached_at = p0;
      cached = page_of(a.c, k.s, (p0 + lane) << a.c.page_log2);
    }
    int page = __shfl_sync(0xFFFFFFFFu, cached, (p0 + lane % nseg - cached_at) & 31);
    const int j0 = k.tile * kTile + (lane % nseg) * seg_rows;  // first slot of this lane's segment
    if (j0 >= k.q.total) page = -1;
    const uint32_t have = __ballot_sync(0xFFFFFFFFu, lane < nseg && page >= 0);
    const bool broken = __any_sync(0xFFFFFFFFu, lane < nseg && page < 0 && j0 < k.q.total);
    if (lane == 0) {
      uint32_t gr = 0;
      for (int i = 0; i < nseg; ++i)
        if ((have >> i) & 1) gr |= ((1u << (seg_rows / 16)) - 1u) << (i * (seg_rows / 16));
      *groups = gr;
      if (broken) flag_error(a.dev_err, MOE_DEV_BAD_ID);
      tc::mbar_arrive_expect_tx(full, __popc(have) * seg_rows * (D + 8));
    }
    __syncwarp();
    if (lane < nseg && page >= 0) {
      const uint8_t* b = page_block(a.c, page, k.h);
      const int r0 = j0 & (a.c.page_size - 1);
      bulk_copy(st.k + lane * seg_rows * (D / 2), b + static_cast<size_t>(r0) * (D / 2), seg_rows * (D / 2), full);
      bulk_copy(st.v + lane * seg_rows * (D / 2), b + static_cast<size_t>(a.c.page_size + r0) * (D / 2), seg_rows * (D / 2), full);
      bulk_copy(st.p + lane * seg_rows * 8, b + static_cast<size_t>(a.c.page_size) * D + r0 * 8, seg_rows * 8, full);
    }
  }
};

// Notes an item that starts in this CTA and ends in a later one.
__device__ __forceinline__ void note_cut(const AttendArgs& a, int cta, int ncta, long long total, const Cursor& k, int row0,
                                         int rows, long long item_end, int slot) {
  int32_t* M = a.meta + static_cast<size_t>(cta) * 8;
  M[1] = k.s;
  M[2] = k.h;
  M[3] = row0;
  M[4] = rows;
  M[5] = static_cast<int>((item_end * ncta - 1) / total);  // the CTA that owns the item's last unit
  M[6] = slot;
  M[0] = 1;
}

constexpr int kWideRows = 128;
// The tensor-core kernel (tcgen05) for row blocks of 128.
int wide_grid();
int wide_launch(const AttendArgs& a, int grid, cudaStream_t s);

}  // namespace kv4
}  // namespace moe
