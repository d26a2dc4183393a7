// kv4_weigh: adds to every slot the softmax weight that the new tokens gave it.
//
//   mass[s, h, j] += sum over the query rows i of kv head h: exp(S_ij - lse_i)
//
// with the lse of kv4_attend, so one pass over the keys alone (half the
// cache).  Slots are the rows of the product on the 5th-generation tensor cores,
// S^T [128 slots x query rows] = C_k Q^T: a thread owns a slot, unpacks its key
// into TMEM (the nibbles are fp16 numbers already, see kv4.cuh), keeps its scale and zero in
// registers, and sums its own columns' exponentials in fp32 in a fixed order: no
// atomics, no exchange between threads.
//
// Four warps and 128 TMEM columns (keys, 64 columns of scores) a CTA, three CTAs
// an SM (four at D = 64 and for few rows), so that one's products and loads run while the others' exponentials do.
// The floor is memory's (D / 2 + 4 bytes of keys, 8 of mass a slot) up to about 100 query rows a kv head (60 at D = 64),
// the exponentials' (32 a clock and SM) beyond; 16 trees of up to 5 tokens, 64 query heads on 8 and up to 16k slots take
// 50 us, 30% of the copy rate, in the chain of a unit: keys to TMEM, product, exponentials (issue slots 49% busy,
// the exponentials' unit 12%).
//
// More than 128 query rows (a prompt's chunk) are shared by the CTAs of a cluster, which take the same
// slots and add up their sums in the order of their ranks: a slot's row blocks one after the
// other in one CTA take 621 us for 6400 rows and 405 slots, with clusters of 8 85 us.
#include <cooperative_groups.h>

#include "kv4.cuh"
#include "kv4_sched.cuh"
#include "tc_f16.cuh"

namespace moe {
namespace kv4 {

int attn_validate(const kv4_attn_cfg* cfg, const Cache& c);

namespace {

namespace cg = cooperative_groups;

using tc::add2;
using tc::fma2;
using tc::mul2;

constexpr int kThreads = 128;
constexpr int kSlots = 128;          // slots of a unit, one a thread
constexpr int kCols = 64;            // columns of a product
constexpr int kAllRows = 1 << 30;    // one row block per kv head
constexpr int kStages = 3;           // key rows on their way
// What beginning an item costs, in units: a CTA with two units whose second begins another item took the longest (on
// the device, 4 trees on up to 4000 slots 14.6 us with 0, 11.4 with 1, 12.5 with 2; 16 on up to 16k 47.4, 46.8, 45.5).
constexpr int kItemUnits = 1;
constexpr int kNoToken = -(1 << 30) - 1;  // of a row that has seen nothing: below every slot's distance from the new ones
constexpr int kGroup = 8;            // units whose sums wait in shared memory where rows come in several blocks
constexpr uint32_t kTmemCols = 128;
constexpr uint64_t kWaitBudgetNs = 2000000000ull;  // 2 s

struct WeighArgs {
  Cache c;
  const uint16_t* q;
  long long q_ts, q_hs;
  const int32_t* q_start;
  const int32_t* base;
  const uint64_t* visible;
  const float* lse;
  float* mass;
  int32_t T, Hq, G;
  float scale_log2;
  int32_t* dev_err;
  bool withhold;   // test hook: the first stage of a CTA's first warp never looks full, so that the wait for it runs out
};

template <int D, int kRows>  // kRows: query rows held at a time
struct Smem {
  alignas(1024) uint8_t q[kRows * D * 2];                    // panels of 64 dimensions: [kRows][128 B], 128-byte swizzle
  alignas(16) uint8_t k[4][kStages][32 * (D / 2)];           // per warp: key rows of its 32 slots
  alignas(16) uint8_t par[4][kStages][32 * 8];               // their parameters
  alignas(16) float cq[kRows];
  alignas(16) float cqs[kRows];
  alignas(16) float nl[kRows];                               // -lse, in log2; -inf: no weight
  uint64_t mask[kRows];
  long long at[kRows];                                       // where in q
  int token[kRows];
  float acc[kGroup][kSlots];
  uint64_t done, full[4][kStages];
  uint32_t groups[4][kStages];                               // bit x: slots 16 x .. of the warp's lie in a valid page
  long long scratch[32];
  uint32_t tmem;
  int abort, never;
  long long cum[1];
};

// Rows row0 .. of the item's queries into shared memory as the product's
// second operand, in the order of the key words' pairs (see prep_q of kv4.cuh).
// A thread a row finds its place, lse and mask; W lanes a row convert it.
// Returns whether the thread's row has seen nothing (an lse of -inf).
template <int D, int kRows>
__device__ __forceinline__ bool load_queries(const WeighArgs& a, const Cursor& k, int row0, int rows, Smem<D, kRows>& sm) {
  constexpr int W = D / 8;  // a row's code words, one a lane
  const int padded = (rows + 15) & ~15;
  const int mine = threadIdx.x, tok = (row0 + min(mine, rows - 1)) / a.G;
  float lse = -INFINITY;
  uint64_t mask = 0;
  if (mine < rows) {
    const int hd = k.h * a.G + (row0 + mine) - tok * a.G;
    sm.at[mine] = (k.q.q0 + tok) * a.q_ts + hd * a.q_hs;
    lse = a.lse[(static_cast<size_t>(k.q.q0) + tok) * a.Hq + hd];  // (used below the loop, whose loads go out meanwhile)
    if (a.visible) mask = a.visible[k.q.q0 + tok];
  }
  __syncthreads();
  const int x = threadIdx.x % W;
  constexpr int kStep = kThreads / W, kBeside = 4;  // rows of a pass; passes beside each other, step by step
#pragma unroll 1
  for (int r0 = threadIdx.x / W; r0 < padded; r0 += kBeside * kStep) {
    uint4 raw[kBeside];
    float sum[kBeside];
    uint32_t top[kBeside];  // largest magnitude, as bf16
#pragma unroll
    for (int y = 0; y < kBeside; ++y) {
      const int r = r0 + y * kStep;
      raw[y] = make_uint4(0, 0, 0, 0);
      if (r < rows) raw[y] = *reinterpret_cast<const uint4*>(a.q + sm.at[r] + 8 * x);
    }
#pragma unroll
    for (int y = 0; y < kBeside; ++y) {
      const uint32_t u[4] = {raw[y].x, raw[y].y, raw[y].z, raw[y].w};
      uint32_t t = 0;
      sum[y] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        t = __vmaxu2(t, u[j] & 0x7FFF7FFFu);
        sum[y] += __uint_as_float(u[j] << 16) + __uint_as_float(u[j] & 0xFFFF0000u);
      }
      top[y] = max(t >> 16, t & 0xFFFFu);
    }
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
      for (int y = 0; y < kBeside; ++y) {
        top[y] = max(top[y], __shfl_xor_sync(0xFFFFFFFFu, top[y], o));
        sum[y] += __shfl_xor_sync(0xFFFFFFFFu, sum[y], o);
      }
#pragma unroll
    for (int y = 0; y < kBeside; ++y) {
      const int r = r0 + y * kStep;
      if (r >= padded) continue;
      // (Below 2^-113 a row's largest magnitude lands below 2^14; its scores are zero all the same.)
      const int ex = static_cast<int>(top[y] >> 7);
      const int e = ex > 0 && ex < 255 ? min(14 + 127 - ex, 127) : 0;
      const float f = __uint_as_float(static_cast<uint32_t>(127 + e) << 23), f16 = f * 0.0625f;
      auto pair = [&](uint32_t lo, uint32_t hi, float by) {
        const float2 v = mul2(make_float2(__uint_as_float(lo), __uint_as_float(hi)), make_float2(by, by));
        return pack_h2(v.x, v.y);
      };
      const uint4 u = raw[y];
      *reinterpret_cast<uint4*>(sm.q + (x >> 3) * (kRows * 128) + (r >> 3) * 1024 + (r & 7) * 128 + (((x & 7) ^ (r & 7)) << 4)) =
          make_uint4(pair(u.x << 16, u.z << 16, f), pair(u.x & 0xFFFF0000u, u.z & 0xFFFF0000u, f16),
                     pair(u.y << 16, u.w << 16, f), pair(u.y & 0xFFFF0000u, u.w & 0xFFFF0000u, f16));
      if (x == 0) {
        const int up = 24 - e;  // the codes carry 2^-24
        sm.cq[r] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + (up >> 1)) << 23) *
                   __uint_as_float(static_cast<uint32_t>(127 + up - (up >> 1)) << 23);
        sm.cqs[r] = a.scale_log2 * sum[y];
      }
    }
  }
  if (mine < padded) {
    const bool none = lse == -INFINITY;  // a row that saw nothing sees no slot, whatever those hold
    sm.nl[mine] = none ? -INFINITY : -lse * kLog2e;
    sm.token[mine] = none ? kNoToken : tok;
    sm.mask[mine] = none ? 0 : mask;
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  return mine < rows && lse == -INFINITY;
}

// kShared: the CTAs of a cluster take the same units, each with its share of the query rows.
template <int D, int kRows, bool kShared>
__global__ void __launch_bounds__(kThreads, 4) weigh_kernel(const WeighArgs a) {
  constexpr int P = D / 32;   // 16-byte pieces of a key row
  constexpr uint32_t kACol = 0, kSCol = D / 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<D, kRows>& sm = *reinterpret_cast<Smem<D, kRows>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tc::mbar_init(&sm.done, 1);
    for (int w = 0; w < 4; ++w)
      for (int i = 0; i < kStages; ++i) tc::mbar_init(&sm.full[w][i], a.withhold && w + i == 0 ? 2 : 1);
    sm.abort = sm.never = 0;
    tc::fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(&sm.tmem, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  pdl_wait();
  pdl_trigger();
  build_units(a.c, a.q_start, a.base, a.T, a.G, kAllRows, kSlots, kItemUnits, sm.cum, sm.scratch, a.dev_err, blockIdx.x == 0);
  tc::tc_fence_after();
  const uint32_t tmem = sm.tmem, mine = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  const uint64_t qd = tc::smem_desc_sw128(tc::smem_u32(sm.q));
  volatile int* abort_flag = &sm.abort;
  const long long total = sm.cum[a.c.S];
  const cg::cluster_group cluster = cg::this_cluster();
  const int cs = kShared ? static_cast<int>(cluster.num_blocks()) : 1;
  const int rank = kShared ? static_cast<int>(cluster.block_rank()) : 0;
  const int team = blockIdx.x / cs;
  const Shares shares(total, gridDim.x / cs);
  const long long u0 = shares.begin(team), u1 = shares.begin(team + 1);
  const size_t width = static_cast<size_t>(a.c.width) << a.c.page_log2;
  const size_t stride = static_cast<size_t>(a.c.Hkv) * a.c.block_bytes();
  const int last_row = a.c.page_size - 1;
  // A warp's 32 slots lie in one page, or in two of 16.
  const int seg_log2 = min(a.c.page_log2, 5), nseg = 32 >> seg_log2;
  int st = 0, st_next = 0;       // stages of the copies: read next, started next
  uint32_t phase = 0;
  uint32_t parity = 0;
  bool dead = false;
  int told = 0;  // first slot that not all rows held see: the context's end, or 0 where a row has seen nothing
  Cursor k;
  if (u0 < u1) cursor_at(k, a.c, a.q_start, a.base, a.T, a.G, kAllRows, kSlots, kItemUnits, sm.cum, u0);
  for (long long u = u0; u < u1 && (kShared || !dead);) {  // (to its end in any case: a cluster's CTAs meet in it)
    const int span = static_cast<int>(u1 - u < k.nt - k.tile ? u1 - u : k.nt - k.tile);
    const int units = max(0, min(span, k.nt - kItemUnits - k.tile));  // those with slots
    const int of_all = k.q.nq * a.G, share = kShared ? ((of_all + cs - 1) / cs + 15) & ~15 : of_all;
    const int row_at = rank * share, all = min(share, of_all - row_at);  // (none: negative)
    const int blocks = all > 0 ? (all + kRows - 1) / kRows : 0;
    if (a.visible && k.q.nq > kMaxTree && tid == 0) flag_error(a.dev_err, MOE_DEV_CAPACITY);
    float* mass = a.mass + (static_cast<size_t>(k.s) * a.c.Hkv + k.h) * width;
    const int group = kShared || blocks > 1 ? kGroup : units;
    const uint8_t* from = a.c.pages + static_cast<size_t>(k.h) * a.c.block_bytes();
    const int32_t* table = a.c.table + static_cast<size_t>(k.s) * a.c.width;
    for (int g0 = 0; g0 < units && (kShared || !dead); g0 += group) {
      const int n = min(group, units - g0), t0 = k.tile + g0;
      for (int block = 0; block < blocks && !dead; ++block) {
        const int row0 = row_at + block * kRows, rows = min(kRows, all - block * kRows), padded = (rows + 15) & ~15;
        // Key rows: the lane of each page segment looks its page up, one unit ahead, and copies it.
        // (What it finds is not looked at before it is needed: a use would wait for the load.)
        int page = 0;
        bool wanted = false;
        auto look = [&](int i) {
          const int j = (t0 + i) * kSlots + warp * 32 + (lane << seg_log2);
          wanted = lane < nseg && i < n && j < k.q.total;
          if (wanted) page = table[j >> a.c.page_log2];
        };
        auto start = [&](int i) {
          const bool found = wanted && page >= 0 && page < a.c.n_pages;
          if (wanted && !found) flag_error(a.dev_err, MOE_DEV_BAD_ID);
          const uint32_t have = __ballot_sync(0xFFFFFFFFu, found);
          uint64_t* bar = &sm.full[warp][st_next];
          if (lane == 0) {
            sm.groups[warp][st_next] = nseg == 1 ? have * 3 : have;
            tc::mbar_arrive_expect_tx(bar, (__popc(have) * (D / 2 + 8)) << seg_log2);
          }
          __syncwarp();
          if (found) {
            const int r = ((t0 + i) * kSlots + warp * 32 + (lane << seg_log2)) & last_row;
            const uint8_t* b = from + page * stride;
            bulk_copy(sm.k[warp][st_next] + (lane << seg_log2) * (D / 2), b + r * (D / 2), (D / 2) << seg_log2, bar);
            bulk_copy(sm.par[warp][st_next] + (lane << seg_log2) * 8, b + a.c.page_size * D + r * 8, 8u << seg_log2, bar);
          }
          st_next = st_next + 1 == kStages ? 0 : st_next + 1;
        };
        // Another role's giving up does not end the copies of this warp's stage, which is filled again before long.
        auto give_up = [&] {
          *abort_flag = 1;
          tc::mbar_wait_bounded(&sm.full[warp][st], phase, &sm.never, 100000000ull);
        };
        look(0);
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i) {
          start(i);
          look(i + 1);
        }
        __syncthreads();  // the rows before have been read
        if (!kShared || g0 == 0 || blocks > 1)
          told = __syncthreads_or(load_queries<D, kRows>(a, k, row0, rows, sm)) ? 0 : k.q.base;
        else
          __syncthreads();
        const bool last = !kShared && block == blocks - 1;
        // The mass of this unit's slot, loaded one unit ahead.
        auto mass_of = [&](int i) {
          const int j = (t0 + i) * kSlots + tid;
          return last && i < n && j < k.q.total ? mass[j] : 0.f;
        };
        float next_mass = mass_of(0);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          if (!tc::mbar_wait_bounded(&sm.full[warp][st], phase, abort_flag, kWaitBudgetNs)) give_up();
          __syncwarp();
          const int j0 = (t0 + i) * kSlots, j = j0 + tid;
          const bool valid = j < k.q.total && ((sm.groups[warp][st] >> (lane >> 4)) & 1);
          uint32_t o[16];
          const uint8_t* row = sm.k[warp][st] + lane * (D / 2);
          const float2 kp = __half22float2(*reinterpret_cast<const __half2*>(sm.par[warp][st] + lane * 8));
#pragma unroll
          for (int x = 0; x < P; ++x) {
            const uint4 w = *reinterpret_cast<const uint4*>(row + 16 * x);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              o[4 * y] = nibbles<0>(ww[y]);
              o[4 * y + 1] = nibbles<1>(ww[y]);
              o[4 * y + 2] = nibbles<2>(ww[y]);
              o[4 * y + 3] = nibbles<3>(ww[y]);
            }
            tc::tmem_st16(mine + kACol + 16 * x, o);
          }
          if (++st == kStages) st = 0, phase ^= 1;
          __syncwarp();
          start(i + kStages - 1);  // (an empty phase where there is no such unit)
          look(i + kStages);
          float before = next_mass;
          next_mass = mass_of(i + 1);
          if (block > 0) before += sm.acc[i][tid];
          tc::tmem_st_wait();
          const float2 ks = make_float2(kp.x, kp.x), kz = make_float2(kp.y, kp.y);
          float2 w0 = make_float2(0.f, 0.f), w1 = w0;
          for (int c0 = 0; c0 < padded; c0 += kCols) {
            const int cols = min(kCols, padded - c0);
            tc::tc_fence_before();
            __syncthreads();  // keys in place, the scores before have been read
            if (tid == 0) {
              tc::tc_fence_after();
              const uint32_t id = tc::idesc_f16(kSlots, cols);
              const uint64_t b = qd + c0 * 8;  // 128-byte rows
#pragma unroll
              for (int t = 0; t < D / 16; ++t)
                tc::mma_f16_ts(tmem + kSCol, tmem + kACol + 8 * t, b + (t >> 2) * (kRows * 128 >> 4) + (t & 3) * 2, id, t > 0);
              tc::mma_commit(&sm.done);
            }
            if (!tc::mbar_wait_bounded(&sm.done, parity, abort_flag, kWaitBudgetNs)) *abort_flag = 1;
            __syncwarp();
            parity ^= 1;
            tc::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < cols; c += 16) {
              float v[16];
              tc::tmem_ld16(mine + kSCol + c, v);
              const float4* cq = reinterpret_cast<const float4*>(sm.cq + c0 + c);
              const float4* cqs = reinterpret_cast<const float4*>(sm.cqs + c0 + c);
              const float4* nl = reinterpret_cast<const float4*>(sm.nl + c0 + c);
              tc::tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const float4 f = cq[x], z = cqs[x], l = nl[x];
                float2 t = fma2(ks, mul2(make_float2(v[4 * x], v[4 * x + 1]), make_float2(f.x, f.y)),
                                fma2(kz, make_float2(z.x, z.y), make_float2(l.x, l.y)));
                float2 y = fma2(ks, mul2(make_float2(v[4 * x + 2], v[4 * x + 3]), make_float2(f.z, f.w)),
                                fma2(kz, make_float2(z.z, z.w), make_float2(l.z, l.w)));
                t = make_float2(ex2(t.x), ex2(t.y));
                y = make_float2(ex2(y.x), ex2(y.y));
                if (j0 + kSlots > told && j >= told) {
                  const int d = j - k.q.base, r = c0 + c + 4 * x;
                  auto see = [&](int e) {
                    if (!a.visible || d < 0) return d <= sm.token[r + e];
                    return d < kMaxTree && ((sm.mask[r + e] >> d) & 1);
                  };
                  t.x = see(0) ? t.x : 0.f;
                  t.y = see(1) ? t.y : 0.f;
                  y.x = see(2) ? y.x : 0.f;
                  y.y = see(3) ? y.y : 0.f;
                }
                w0 = add2(w0, t);
                w1 = add2(w1, y);
              }
            }
          }
          w0 = add2(w0, w1);
          const float sum = before + (w0.x + w0.y);
          if (!last) sm.acc[i][tid] = sum;
          else if (valid) mass[j] = sum;
          if (*abort_flag) dead = true;
        }
        // The two empty phases beyond the last unit; nothing is in flight after them.
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i) {
          if (!tc::mbar_wait_bounded(&sm.full[warp][st], phase, abort_flag, kWaitBudgetNs)) give_up();
          __syncwarp();
          if (++st == kStages) st = 0, phase ^= 1;
        }
        dead = __syncthreads_or(dead);
      }
      if constexpr (kShared) {
        // The shares' sums in the order of the ranks; each rank writes its part of the units.
        cluster.sync();
        const int shares = (of_all + share - 1) / share;
        for (int i = rank; i < n; i += cs) {
          const int j = (t0 + i) * kSlots + tid;
          const int page = j < k.q.total ? table[j >> a.c.page_log2] : -1;
          if (page < 0 || page >= a.c.n_pages) continue;
          const float before = mass[j];
          float sum = 0.f;
          for (int r = 0; r < shares; ++r) sum += cluster.map_shared_rank(sm.acc[i], r)[tid];
          mass[j] = before + sum;
        }
        cluster.sync();
      }
    }
    u += span;
    if (u < u1) cursor_next(k, a.c, a.q_start, a.base, a.T, a.G, kAllRows, kSlots, kItemUnits, sm.cum);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) {
    // Products and copies in flight end before TMEM and shared memory go.
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 1000000ull) {}
    flag_error(a.dev_err, MOE_DEV_TIMEOUT);
  }
  __syncthreads();
  if (warp == 0) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// ctas: what fits an SM (TMEM: four); cluster: CTAs that share an item's query rows.  Clusters above 2 do not
// fill every SM, and a grid that does not fit at once takes twice the time (16 sequences of 8k slots,
// 512 rows, clusters of 4: 291 us with a full grid, 237 with nine tenths).
template <int D, int kRows, bool kShared>
int launch_weigh(const WeighArgs& a, int ctas, int cluster, cudaStream_t s) {
  constexpr auto kernel = weigh_kernel<D, kRows, kShared>;
  const size_t smem = sizeof(Smem<D, kRows>) + static_cast<size_t>(a.c.S) * 8;
  const int st = allow_smem<kernel>(smem);
  if (st != MOE_OK) return st;
  LaunchScope ls(kProfKv4Weigh, s);
  if constexpr (kShared)
    return launch_clusters(kernel, sm_count() * ctas * (cluster > 2 ? 9 : 10) / (10 * cluster), cluster, kThreads, smem, s, a);
  return launch_k(kernel, dim3(sm_count() * ctas), dim3(kThreads), smem, s, false, a);
}

}  // namespace
}  // namespace kv4
}  // namespace moe

extern "C" int kv4_weigh(const kv4_cache* cache, const void* q, const int32_t* q_start, const int32_t* base,
                         const uint64_t* visible, const float* lse, const kv4_attn_cfg* cfg, float* mass,
                         int32_t* dev_err, void* stream) {
  using namespace moe;
  using namespace moe::kv4;
  Cache c;
  int st = cache_validate(cache, &c);
  if (st != MOE_OK || (st = attn_validate(cfg, c)) != MOE_OK) return st;
  if (cfg->T == 0 || c.S == 0) return MOE_OK;
  if (!q || !q_start || !base || !lse || !mass) return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(q) & 15) || (reinterpret_cast<uintptr_t>(visible) & 7) ||
      ((reinterpret_cast<uintptr_t>(q_start) | reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(lse) |
        reinterpret_cast<uintptr_t>(mass)) & 3))
    return MOE_ERR_ARG;
  WeighArgs a{c, static_cast<const uint16_t*>(q), cfg->q_token_stride, cfg->q_head_stride, q_start, base, visible, lse,
              mass, cfg->T, cfg->n_q_heads, cfg->n_q_heads / c.Hkv, cfg->scale * kLog2e, dev_err,
              (test_stall_mask() & MOE_TEST_STALL_KV4_WEIGH) != 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long rows = static_cast<long long>(cfg->max_q) * a.G;
  // Clusters of 1 / 2 / 4 / 8 take, on the device, at 136 rows (2 sequences of 3k slots) 24 / 18 / 18 / 22 us, at 224 (16
  // of 8k) 114 / 128 / 157 / 241, at 320 (4 of 4k) 45 / 37 / 33 / 41, at 512 (16 of 8k) 241 / 249 / 237 / 274, at 2400 (4 of
  // 2k) 275 / 186 / 152 / 132.
  int cluster = 1;
  while (cluster < 8 && rows > 128 * cluster) cluster *= 2;
  if (cluster > 1) return c.D == 128 ? launch_weigh<128, 128, true>(a, 3, cluster, s) : launch_weigh<64, 128, true>(a, 4, cluster, s);
  if (c.D == 64) return launch_weigh<64, 128, false>(a, 4, 1, s);
  // 64 rows in shared memory leave room for a fourth CTA.
  return rows <= 64 ? launch_weigh<128, 64, false>(a, 4, 1, s) : launch_weigh<128, 128, false>(a, 3, 1, s);
}
