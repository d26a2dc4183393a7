// moe_group_gate_up, moe_group_down: the experts' products of a prompt's
// tokens, grouped by expert, on pairs of CTAs.
//
// A tile is 256 weight rows of one expert times up to 256 rows of its group
// (N, a multiple of 32): a group of any size pads by 31 rows at most, whereas
// tokens as the product's M would pad to 128 or 256.  gate/up takes 128 gate and
// the same 128 up rows, half of each in either CTA: gate in the CTA's TMEM lanes
// 0-63, up in 64-127.  K goes through a ring of stages of 64 columns, 16 KB of
// weights and up to 16 KB of rows each; the sums are kept twice, so that a
// tile's epilogue runs beside the next one's products.
//
// The rows come by TMA where they lie: down's in one box a stage (a map for each
// number of rows), gate/up's, the tokens' rows of x through perm_token, by its
// gather of four rows a copy.  What a bulk copy costs is its thread's time, 65 cycles
// and more, so eight warps share the gather's copies of a stage.  (One warp: 3.63 ms
// for 65,536 rows of 4096 x 1536 matrices; four warps: 1.31; rows copied side by side
// first: 0.1 ms for that alone.)
//
// What bounds full tiles is loading, 32 KB a stage and CTA from L2.  (Rows loaded once for
// two pairs and sent to both took gate/up from 1.11 to 1.01 ms; a copy to several CTAs must
// not read another GPU's memory, which a caller's pointers may be.)
//
// Persistent: pair i takes tiles i, i + pairs, ..., in an order that has a
// matrix's rows go over all of their group's chunks before the next rows come,
// and an expert's before the next expert's: what runs at the same time shares
// weights and rows in L2.
//
// Roles of a CTA: warp 0 loads weights, warp 1 owns TMEM and (in the pair's first
// CTA) issues the products, warps 2-5 take the sums out, the warps from 6 on load
// rows.  Every wait is bounded.
//
// 8192 tokens of 8 of 128 experts, 4096 x 1536, on the device: gate/up 1.11 ms, 1480
// TFLOP/s; down 0.54 ms, 1520, and 0.09 for the sum.  (Tensor pipe 66% and 70% busy with
// 4096 tokens of 2 of 16.)  300 tokens: gate/up 0.465 ms, the weights' bytes at 6.9 TB/s.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "apart.cuh"
#include "common.cuh"
#include "smem_limit.cuh"
#include "tc_pair.cuh"

namespace moe {
namespace {

template <bool kGateUp>
constexpr int kThreads = 192 + (kGateUp ? 256 : 32);
constexpr int kStages = 6;
constexpr int kABytes = 128 * 128, kBBytes = 128 * 128;
constexpr int kMaxU = 1024;
constexpr uint64_t kWaitNs = 2000000000ull;

struct GroupArgs {
  const int32_t *n_unique, *unique, *offsets, *perm, *slot_of;
  uint16_t* out;              // [rows][N]
  int32_t* dev_err;
  int T, rows, E, cap, n_slots;
  int N, K;                   // rows of a matrix (gate/up: of one of its halves), reduction length
  int tiled, MT, stall;
};

// Maps of the rows with boxes of a CTA's part of 32, 64, ... 256 of them (gate/up: the first, of one row).
struct RowMaps {
  CUtensorMap m[8];
};

struct Smem {
  alignas(1024) uint8_t a[kStages][kABytes];
  alignas(1024) uint8_t b[kStages][kBBytes];
  alignas(16) uint16_t turn[4][32][32];
  float swap[2][4][16][32];   // gate/up: what a warp hands to its partner, twice
  int cum[kMaxU + 1];         // chunks before each expert of the union
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int abort;
  int part[14];
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// Chunks of a group of n rows, and rows of a chunk (all but the last).
__host__ __device__ __forceinline__ int chunks_of(int n) { return (n + 255) / 256; }
__device__ __forceinline__ int chunk_rows(int n) {
  const int c = chunks_of(n);
  return ((n + c - 1) / c + 31) & ~31;
}

struct Tile {
  int u, slot, m, p, n, N;  // expert's place in the union, its weights, row tile, first row of the chunk, its rows, padded
};

// Group u's expert slot and rows, or n = 0 if any of it is out of range.
__device__ __forceinline__ void group_of(const GroupArgs& a, int u, int* slot, int* p0, int* n) {
  const int e = a.unique[u], b = a.offsets[u], q = a.offsets[u + 1];
  const bool ok = e >= 0 && e < a.E && b >= 0 && b <= q && q <= a.rows;
  *slot = ok ? weight_slot(a.slot_of, a.n_slots, e) : -1;
  *p0 = b;
  *n = *slot >= 0 ? q - b : -1;
}

// Walks the tiles of one pair.
struct Walk {
  const GroupArgs& a;
  const int* cum;
  int U, u = 0, first = -1, slot, p0, n, rows, nc;
  __device__ __forceinline__ Walk(const GroupArgs& args, const int* c, int us) : a(args), cum(c), U(us) {}
  __device__ __forceinline__ bool at(long long t, Tile* x) {
    while (u < U && static_cast<long long>(cum[u + 1]) * a.MT <= t) ++u;
    if (u >= U) return false;
    if (first != u) {
      group_of(a, u, &slot, &p0, &n);
      first = u;
      nc = cum[u + 1] - cum[u];
      rows = chunk_rows(n);
    }
    const int r = static_cast<int>(t - static_cast<long long>(cum[u]) * a.MT), c = r % nc;
    x->u = u, x->slot = slot, x->m = r / nc;
    x->p = p0 + c * rows;
    x->n = min(rows, n - c * rows);
    x->N = (x->n + 31) & ~31;
    return true;
  }
};

// A loading warp's way out.  Copies in flight land in microseconds; nothing tells this CTA of those that report to the other one.
__device__ __noinline__ void give_up_loading(Smem& sm, const GroupArgs& a, int lane) {
  if (lane == 0) {
    *static_cast<volatile int*>(&sm.abort) = 1;
    flag_error(a.dev_err, MOE_DEV_TIMEOUT);
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 5000000ull) __nanosleep(1000);
  }
  __syncwarp();
}

template <bool kGateUp>
__global__ void __launch_bounds__(kThreads<kGateUp>, 1)
    group_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ RowMaps xmap, const GroupArgs a) {
  extern __shared__ uint8_t raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = tc::cluster_rank();  // in the pair
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) tc::mbar_init(&sm.full[i], 1), tc::mbar_init(&sm.empty[i], 1);
    for (int i = 0; i < 2; ++i) tc::mbar_init(&sm.acc_full[i], 1), tc::mbar_init(&sm.acc_empty[i], 8);
    tc::mbar_init(&sm.drain, 1);
    sm.abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc_pair(&sm.tmem, 512);
    tc::tmem_relinquish_pair();
  }
  // The union's chunks, added up.
  const int U0 = *a.n_unique;
  const bool counted = U0 >= 0 && U0 <= a.cap;
  const int U = counted ? U0 : 0;
  if (!counted && blockIdx.x == 0 && tid == 0) flag_error(a.dev_err, MOE_DEV_CAPACITY);
  int before = 0;
  for (int base = 0; base < U; base += kThreads<kGateUp>) {
    const int u = base + tid;
    int c = 0;
    if (u < U) {
      int slot, p0, n;
      group_of(a, u, &slot, &p0, &n);
      if (n < 0 && blockIdx.x == 0) flag_error(a.dev_err, MOE_DEV_BAD_ID);
      c = n > 0 ? chunks_of(n) : 0;
    }
    const int inc = warp_inclusive_sum(c, lane);
    if (lane == 31) sm.part[warp] = inc;
    __syncthreads();
    int sum = before;
    for (int w = 0; w < kThreads<kGateUp> / 32; ++w) {
      if (w < warp) sum += sm.part[w];
      before += sm.part[w];
    }
    if (u < U) sm.cum[u + 1] = sum + inc;
    __syncthreads();
  }
  if (tid == 0) sm.cum[0] = 0;
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const long long total = static_cast<long long>(before) * a.MT;
  const int KB = a.K / 64;
  volatile int* gave_up = &sm.abort;
  Walk walk(a, sm.cum, U);
  Tile x;

  if (warp == 0) {
    // ---------------------------------------------------------- weights
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (long long t = pair; t < total && ok; t += pairs) {
      walk.at(t, &x);
      const uint32_t bytes = 2u * (kABytes + x.N / 2 * 128);
      // Where the tile's rows begin in the map, and its steps from one block of columns to the next.
      int wx = 0, wy, wz = 0, dx = 0, dy = 0, dz = 0;
      const int r = static_cast<int>(rank);
      if (kGateUp) {
        wy = r * 64 + (a.tiled ? 0 : x.m * 128);
        wz = 2 * (a.tiled ? (x.slot * a.MT + x.m) * KB : x.slot);
        (a.tiled ? dz : dx) = a.tiled ? 2 : 64;
      } else {
        wy = a.tiled ? (x.slot * ((a.N + 127) / 128) + 2 * x.m + r) * KB * 128 : x.slot * a.N + x.m * 256 + r * 128;
        (a.tiled ? dy : dx) = a.tiled ? 128 : 64;
      }
      for (int kb = 0; kb < KB; ++kb) {
        ok = tc::mbar_sleep<true>(&sm.empty[s], ph ^ 1, gave_up, kWaitNs);
        if (!ok) break;
        if (tc::elect_one()) {
          if (rank == 0) tc::mbar_arrive_expect_tx(&sm.full[s], bytes);
          const uint32_t bar = tc::smem_of(&sm.full[s], 0);
          if (!a.stall) {
            if (kGateUp)
              tc::tma_load_3d_pair(sm.a[s], &wmap, wx, wy, wz, bar);
            else
              tc::tma_load_2d_pair(sm.a[s], &wmap, wx, wy, bar);
          }
        }
        __syncwarp();
        wx += dx, wy += dy, wz += dz;
        if (++s == kStages) s = 0, ph ^= 1;
      }
    }
    // The last products' arrivals, which come from the pair's first CTA, are seen before this CTA may leave.
    for (int i = 0; i < kStages && ok; ++i) {
      ok = tc::mbar_sleep<true>(&sm.empty[s], ph ^ 1, gave_up, kWaitNs);
      if (++s == kStages) s = 0, ph ^= 1;
    }
    if (!ok) give_up_loading(sm, a, lane);
  } else if (warp == 1) {
    // ---------------------------------------------------------- products
    // The whole warp goes through the loop and one thread of it issues: where the compiler sees one lane's branch instead, a
    // product's operands reach its registers one by one, 710 cycles a stage whatever its size.
    if (rank == 0) {
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true, there = false;
      const uint64_t ad0 = tc::smem_desc_sw128(tc::smem_u32(sm.a[0])), bd0 = tc::smem_desc_sw128(tc::smem_u32(sm.b[0]));
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      for (long long t = pair; t < total && ok; t += pairs) {
        walk.at(t, &x);
        const uint32_t idesc = tc::idesc_bf16_f32(256, __shfl_sync(0xFFFFFFFFu, x.N, 0)), d = tm + acc * 256;
        ok = tc::mbar_sleep<true, true>(&sm.acc_empty[acc], aph ^ 1, gave_up, kWaitNs);
        tc::tc_fence_after();
        for (int kb = 0; kb < KB; ++kb) {
          if (!there && ok) ok = tc::mbar_sleep<true>(&sm.full[s], ph, gave_up, kWaitNs);
          if (!ok) break;
          tc::tc_fence_after();
          const uint64_t ad = ad0 + s * (kABytes >> 4), bd = bd0 + s * (kBBytes >> 4);
          uint64_t* done = &sm.empty[s];
          if (++s == kStages) s = 0, ph ^= 1;
          if (tc::elect_one()) {
            tc::mma_bf16_pair(d, ad, bd, idesc, kb);
            tc::mma_bf16_pair(d, ad + 2, bd + 2, idesc, 1);
            tc::mma_bf16_pair(d, ad + 4, bd + 4, idesc, 1);
            tc::mma_bf16_pair(d, ad + 6, bd + 6, idesc, 1);
            tc::mma_commit_pair(done);
          }
          __syncwarp();
          // The look at the next stage's barrier (100 cycles) runs beside the products.
          there = __all_sync(0xFFFFFFFFu, tc::mbar_test(&sm.full[s], ph));
        }
        if (ok && tc::elect_one()) tc::mma_commit_pair(&sm.acc_full[acc]);
        __syncwarp();
        if (++acc == 2) acc = 0, aph ^= 1;
      }
      if (!ok && lane == 0) flag_error(a.dev_err, MOE_DEV_TIMEOUT);
      if (!ok && tc::elect_one()) {
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(tc::smem_u32(&sm.drain)) : "memory");
        int never = 0;
        tc::mbar_wait_bounded(&sm.drain, 0, &never, kWaitNs / 100);
      }
    }
    __syncwarp();
  } else if (warp >= 6) {
    // ---------------------------------------------------------- rows
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (long long t = pair; t < total && ok; t += pairs) {
      walk.at(t, &x);
      const int half = x.N / 2, first = static_cast<int>(rank) * half;  // this CTA's rows
      const int four = (warp - 6) * 4 + lane;  // gate/up: rows 4 four .. 4 four + 3, by the first lanes
      const bool mine = kGateUp ? lane < 4 && 4 * four < half : lane == 0;
      int row[4] = {x.p + first, 0, 0, 0};
      if (kGateUp && mine) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          row[i] = a.perm[x.p + min(first + 4 * four + i, x.n - 1)];  // the last row stands in for those behind it
          if (row[i] < 0 || row[i] >= a.T) flag_error(a.dev_err, MOE_DEV_BAD_ID), row[i] = 0;
        }
      }
      const CUtensorMap* map = &xmap.m[kGateUp ? 0 : half / 16 - 1];
      for (int kb = 0; kb < KB; ++kb) {
        ok = tc::mbar_sleep<true>(&sm.empty[s], ph ^ 1, gave_up, kWaitNs);
        if (!ok) break;
        if (mine && !a.stall) {
          const uint32_t bar = tc::smem_of(&sm.full[s], 0);
          if (kGateUp)
            tc::tma_gather4_pair(sm.b[s] + four * 512, map, kb * 64, row, bar);
          else
            tc::tma_load_2d_pair(sm.b[s], map, kb * 64, row[0], bar);
        }
        __syncwarp();
        if (++s == kStages) s = 0, ph ^= 1;
      }
    }
    if (!ok) give_up_loading(sm, a, lane);
  } else {
    // ---------------------------------------------------------- sums out
    const int q = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    int acc = 0, flip = 0;
    uint32_t aph = 0;
    bool ok = true;
    for (long long t = pair; t < total && ok; t += pairs) {
      walk.at(t, &x);
      ok = tc::mbar_sleep<true>(&sm.acc_full[acc], aph, gave_up, kWaitNs);
      // (Partners give up together: a barrier is between them.)
      if (kGateUp) {
        int both;
        asm volatile("{\n\t.reg .pred p, r;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.red.and.pred r, %2, 64, p;\n\tselp.b32 %0, 1, 0, r;\n\t}"
                     : "=r"(both) : "r"(static_cast<int>(ok)), "r"(1 + (q & 1)) : "memory");
        ok = both != 0;
      }
      if (!ok) break;
      tc::tc_fence_after();
      const uint32_t src = tmem + acc * 256 + lanes;
      // 32 output columns of this warp, for all of the chunk's rows.
      const int i0 = kGateUp ? x.m * 128 + static_cast<int>(rank) * 64 + (q & 1) * 32 : x.m * 256 + static_cast<int>(rank) * 128 + q * 32;
      uint16_t* out = a.out + static_cast<size_t>(x.p) * a.N + i0;
      uint16_t(&turn)[32][32] = sm.turn[warp - 2];
      for (int c = 0; c < x.N; c += 32) {
        float v0[16], v1[16];
        tc::tmem_ld16(src + c, v0);
        tc::tmem_ld16(src + c + 16, v1);
        tc::tmem_ld_wait();
        // A lane has one output column and the chunk's rows side by side: through shared memory, so that a store takes 16
        // bytes of a row (two-byte stores took 68 cycles each, as long as a tile's products).
        __syncwarp();
        if (kGateUp) {
#pragma unroll
          for (int j = 0; j < 16; ++j) sm.swap[flip][q][j][lane] = q < 2 ? v1[j] : v0[j];
          tc::named_bar_sync(1 + (q & 1), 64);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float other = sm.swap[flip][q ^ 2][j][lane];
            const float g = q < 2 ? v0[j] : other, w = q < 2 ? other : v1[j];
            turn[j][lane] = __bfloat16_as_ushort(__float2bfloat16_rn(__fdividef(g, 1.f + __expf(-g)) * w));
          }
          flip ^= 1;
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            turn[j][lane] = __bfloat16_as_ushort(__float2bfloat16_rn(v0[j]));
            turn[16 + j][lane] = __bfloat16_as_ushort(__float2bfloat16_rn(v1[j]));
          }
        }
        __syncwarp();
        const int c0 = c + (kGateUp && q >= 2 ? 16 : 0), part = (lane & 3) * 8;
        if (i0 + part < a.N) {
#pragma unroll
          for (int j = 0; j < (kGateUp ? 16 : 32); j += 8) {
            const int r = j + (lane >> 2);
            if (c0 + r < x.n)
              *reinterpret_cast<uint4*>(out + static_cast<size_t>(c0 + r) * a.N + part) = *reinterpret_cast<const uint4*>(&turn[r][part]);
          }
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_at(tc::smem_of(&sm.acc_empty[acc], 0));
      if (++acc == 2) acc = 0, aph ^= 1;
    }
    if (!ok && lane == 0) {
      *gave_up = 1;
      flag_error(a.dev_err, MOE_DEV_TIMEOUT);
    }
    __syncwarp();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();
  if (warp == 1) tc::tmem_dealloc_pair(tmem, 512);
}

// y_t = sum_j w_tj o[inv_tj] in slot order in fp32, eight values a thread.
//
// The products o lie between the two kernels in bf16: off by 2^-8 of each term at most,
// so y by 2^-8 sum_j |w_tj o_j| and 2^-8 |y_t| of its own rounding.  Where terms cancel
// that is more than 2^-8 of y, by any factor; with weights that are all positive it is
// 2.3e-3 of y's norm in all, 1.7e-3 with the result's rounding alone.  (moe_verify_ffn
// keeps its terms in fp32.)  Bound by their bytes: 91 us for 65,536 rows of 4096, 6.6
// TB/s, behind the product; fp32 would double them, and what the product writes.
__global__ void __launch_bounds__(256) group_sum_kernel(const uint16_t* __restrict__ o, const int32_t* __restrict__ inv,
                                                        const float* __restrict__ w, const int32_t* __restrict__ n_unique,
                                                        uint16_t* __restrict__ y, int T, int k, int H, int cap, int32_t* dev_err) {
  const long long i = blockIdx.x * 256ll + threadIdx.x;
  const int per = H / 8;
  if (i >= static_cast<long long>(T) * per) return;
  const int t = static_cast<int>(i / per), c = static_cast<int>(i % per) * 8;
  const int U = *n_unique;
  float acc[8] = {};
  if (U > 0 && U <= cap) {
    // Four terms' rows are asked for before the first is used.
    for (int j0 = 0; j0 < k; j0 += 4) {
      uint4 v[4];
      float f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[j] = 0.f, v[j] = make_uint4(0, 0, 0, 0);
        if (j0 + j >= k) continue;
        const long long p = inv[static_cast<long long>(t) * k + j0 + j];
        if (p < 0 || p >= static_cast<long long>(T) * k) {
          if (c == 0) flag_error(dev_err, MOE_DEV_BAD_ID);
          continue;
        }
        f[j] = w[static_cast<long long>(t) * k + j0 + j];
        v[j] = __ldg(reinterpret_cast<const uint4*>(o + p * H + c));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t vw[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          acc[2 * q] += f[j] * __uint_as_float(vw[q] << 16);
          acc[2 * q + 1] += f[j] * __uint_as_float(vw[q] & 0xFFFF0000u);
        }
      }
    }
  }
  uint32_t r[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * q], acc[2 * q + 1]);
    r[q] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(y + static_cast<size_t>(t) * H + c) = make_uint4(r[0], r[1], r[2], r[3]);
}

int group_validate(const moe_layer_weights& lw, int T, int k, const void* w) {
  if (T < 0 || k < 1) return MOE_ERR_ARG;
  if (lw.dtype != MOE_DTYPE_BF16 || k > 16 || T > (1 << 22) || static_cast<long long>(T) * k > (1 << 22)) return MOE_ERR_UNSUPPORTED;
  if (lw.E < 1 || lw.E > 1024 || lw.H < 64 || lw.I < 64 || lw.H % 64 || lw.I % 64 || lw.H > (1 << 20) || lw.I > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (lw.layout != MOE_LAYOUT_ROWMAJOR && lw.layout != MOE_LAYOUT_TILED) return MOE_ERR_ARG;
  if (!w || reinterpret_cast<uintptr_t>(w) & 15) return MOE_ERR_ARG;
  if (lw.pool && (lw.pool->n_slots < 1 || lw.pool->n_slots > 65536 || !lw.pool->slot_of)) return MOE_ERR_ARG;
  // A tensor map's rows are counted in 32 bits.
  const long long mg = (lw.I + 127) / 128, md = (lw.H + 127) / 128;
  const long long per = lw.layout == MOE_LAYOUT_TILED ? (mg * (lw.H / 64) > md * (lw.I / 64) ? mg * (lw.H / 64) : md * (lw.I / 64)) * 256
                                                      : (2ll * lw.I > lw.H ? 2ll * lw.I : lw.H);
  if (weight_slots(lw) * per >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The maps of the weights and of the rows they multiply, and the launch.
template <bool kGateUp>
int group_launch(const moe_layer_weights& lw, const void* rows, int n_rows, const void* w, GroupArgs a, cudaStream_t s) {
  a.MT = kGateUp ? (a.N + 127) / 128 : (a.N + 255) / 256;
  a.tiled = lw.layout == MOE_LAYOUT_TILED;
  a.stall = (test_stall_mask() & MOE_TEST_STALL_GROUP) != 0;
  CUtensorMap wmap;
  RowMaps xmap = {};
  const uint64_t K = a.K, slots = a.n_slots;
  // gate/up: rows of a half, then the halves (of every slot, or of every block of a slot): a box takes 64 of both.
  const uint64_t blocks = slots * ((a.N + 127) / 128) * (K / 64);
  const uint64_t N = a.N, wide = a.tiled ? 64 : K, high = kGateUp ? (a.tiled ? 128 : N) : a.tiled ? blocks * 128 : slots * N;
  const uint64_t wd[3] = {wide, high, 2 * (a.tiled ? blocks : slots)}, ws[2] = {wide * 2, wide * high * 2};
  const uint64_t xd[2] = {K, static_cast<uint64_t>(n_rows)}, xs[1] = {K * 2};
  const uint32_t wb[3] = {64, kGateUp ? 64u : 128u, 2};
  if (!tc::make_bf16_map(&wmap, w, kGateUp ? 3 : 2, wd, ws, wb)) return MOE_ERR_CUDA;
  for (uint32_t i = 0; i < (kGateUp ? 1 : 8); ++i) {
    const uint32_t xb[2] = {64, kGateUp ? 1 : 16 * (i + 1)};
    if (!tc::make_bf16_map(&xmap.m[i], rows, 2, xd, xs, xb)) return MOE_ERR_CUDA;
  }
  const int e = allow_smem<group_kernel<kGateUp>>(kSmemBytes);
  if (e != MOE_OK) return e;
  // At most this many tiles (a chunk a full 256 rows, and one more for each expert).
  const long long most = (a.rows / 256 + static_cast<long long>(a.cap)) * a.MT;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr, cfg.numAttrs = 1, cfg.stream = s;
  cfg.blockDim = dim3(kThreads<kGateUp>), cfg.dynamicSmemBytes = kSmemBytes;
  cfg.gridDim = dim3(2);
  static std::atomic<int> found[64];  // pairs that a device holds at once
  int dev = 0, fits = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (dev >= 0 && dev < 64) fits = found[dev].load(std::memory_order_relaxed);
  if (!fits) {
    if (cudaOccupancyMaxActiveClusters(&fits, group_kernel<kGateUp>, &cfg) != cudaSuccess || fits < 1) return MOE_ERR_CUDA;
    if (dev >= 0 && dev < 64) found[dev].store(fits, std::memory_order_relaxed);
  }
  cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<long long>(fits, most)));
  LaunchScope ls(kGateUp ? kProfGroupGateUp : kProfGroupDown, s);
  return cudaLaunchKernelEx(&cfg, group_kernel<kGateUp>, wmap, xmap, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

bool misaligned(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) & (n - 1); }

}  // namespace
}  // namespace moe

extern "C" int moe_group_gate_up(const void* x, int32_t T, int32_t k, const moe_layer_weights* lw, const int32_t* n_unique,
                                 const int32_t* unique, const int32_t* offsets, const int32_t* perm_token, void* h,
                                 int32_t* dev_err, void* stream) {
  using namespace moe;
  if (!lw) return MOE_ERR_ARG;
  const int st = group_validate(*lw, T, k, lw->w_gate_up);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!x || !n_unique || !unique || !offsets || !perm_token || !h) return MOE_ERR_ARG;
  if (misaligned(x, 16) || misaligned(h, 16) || misaligned(n_unique, 4) || misaligned(unique, 4) || misaligned(offsets, 4) ||
      misaligned(perm_token, 4) || misaligned(dev_err, 4))
    return MOE_ERR_ARG;
  const int rows = T * k, cap = lw->E < rows ? lw->E : rows;
  if (!rows_apart(whole(x, 2ll * T * lw->H), whole(h, 2ll * rows * lw->I))) return MOE_ERR_ARG;
  GroupArgs a = {};
  a.n_unique = n_unique, a.unique = unique, a.offsets = offsets, a.perm = perm_token, a.slot_of = slot_table(*lw);
  a.out = static_cast<uint16_t*>(h), a.dev_err = dev_err;
  a.T = T, a.rows = rows, a.E = lw->E, a.cap = cap, a.n_slots = weight_slots(*lw), a.N = lw->I, a.K = lw->H;
  return group_launch<true>(*lw, x, T, lw->w_gate_up, a, static_cast<cudaStream_t>(stream));
}

extern "C" size_t moe_group_down_workspace(const moe_layer_weights* lw, int32_t T, int32_t k) {
  using namespace moe;
  if (!lw || group_validate(*lw, T, k, lw->w_down) != MOE_OK) return 0;
  return align_up(static_cast<size_t>(T) * k * lw->H * 2, 256) + 256;
}

extern "C" int moe_group_down(const void* h, int32_t T, int32_t k, const moe_layer_weights* lw, const int32_t* n_unique,
                              const int32_t* unique, const int32_t* offsets, const int32_t* inv, const float* w, void* y,
                              void* workspace, size_t ws_bytes, int32_t* dev_err, void* stream) {
  using namespace moe;
  if (!lw) return MOE_ERR_ARG;
  const int st = group_validate(*lw, T, k, lw->w_down);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!h || !n_unique || !unique || !offsets || !inv || !w || !y) return MOE_ERR_ARG;
  if (misaligned(h, 16) || misaligned(y, 16) || misaligned(n_unique, 4) || misaligned(unique, 4) || misaligned(offsets, 4) ||
      misaligned(inv, 4) || misaligned(w, 4) || misaligned(dev_err, 4))
    return MOE_ERR_ARG;
  if (!workspace || ws_bytes < moe_group_down_workspace(lw, T, k)) return MOE_ERR_WORKSPACE;
  if (misaligned(workspace, 256)) return MOE_ERR_ARG;
  const int rows = T * k, cap = lw->E < rows ? lw->E : rows;
  const Rows rh = whole(h, 2ll * rows * lw->I), ry = whole(y, 2ll * T * lw->H);
  const Rows rws = whole(workspace, static_cast<long long>(moe_group_down_workspace(lw, T, k)));
  if (!rows_apart(rh, ry) || !rows_apart(rh, rws) || !rows_apart(ry, rws)) return MOE_ERR_ARG;
  uint16_t* o = static_cast<uint16_t*>(workspace);
  GroupArgs a = {};
  a.n_unique = n_unique, a.unique = unique, a.offsets = offsets, a.slot_of = slot_table(*lw), a.out = o, a.dev_err = dev_err;
  a.T = T, a.rows = rows, a.E = lw->E, a.cap = cap, a.n_slots = weight_slots(*lw), a.N = lw->H, a.K = lw->I;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int e = group_launch<false>(*lw, h, rows, lw->w_down, a, s);
  if (e != MOE_OK) return e;
  LaunchScope ls(kProfGroupDown, s);
  const long long n = static_cast<long long>(T) * (lw->H / 8);
  group_sum_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(o, inv, w, n_unique, static_cast<uint16_t*>(y), T, k, lw->H, cap,
                                                                       dev_err);
  return check_launch();
}
