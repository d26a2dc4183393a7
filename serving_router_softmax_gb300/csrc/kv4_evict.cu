// kv4_evict: brings a cache down to its budget by accumulated attention weight.
//
// Per sequence and kv head, of n slots: the last `recent` stay, and of the
// others those with the largest mass (equal ones: the lower slot) until
// `keep` are kept; they move to slots 0..keep-1 in their old order, codes and
// parameters together, so slots stay in the order in which tokens came.
//
// A cluster of CTAs per (sequence, head), each with its share of the slots,
// their masses in shared memory as ordered bits: the smallest kept mass by a
// radix select (11, 11 and 10 bits; the CTAs add up each other's histograms),
// the kept slots in order by running counts, then the moves.  Moves go in
// rounds in ascending order, each read whole by the cluster before any of it is
// written: a slot never moves up, so a round writes nothing that a later
// one reads.  What it moves is far below the memory's rate; the time is in the
// chain of phases, which is why few rows get clusters of up to 8 CTAs.  On the device 17 us for 32 rows of
// 2304 slots to 2048 (9.4 MB, 1.4 us at the copy rate), 35 us for 32 of up to 40k to 4096 (35 MB, 5.2 us).
#include <cooperative_groups.h>

#include "kv4.cuh"

namespace moe {
namespace kv4 {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kBins = 2048;
constexpr int kHeld = 18432;  // masses that a CTA holds in shared memory; more are read again each time
constexpr int kRound = 4;     // pieces of 16 bytes that a thread moves in a round

struct EvictArgs {
  Cache c;
  const float* mass;
  const int32_t* lens;
  int32_t keep, recent;
  int32_t* new_len;
  int32_t* origin;
  float* mass_out;
  int32_t* dev_err;
};

struct Smem {
  int hist[3][kBins];
  int warp_a[kThreads / 32], warp_b[kThreads / 32];
  int count[2];              // the CTA's kept and tied slots
  int bin, left;
  uint32_t key[kHeld];
};

// Bits whose unsigned order is the masses' order; a NaN is below everything, -0 equals +0.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

// Sums of a and b over the threads before this one; *all_a, *all_b over the block.
__device__ __forceinline__ void block_scan2(Smem& sm, int& a, int& b, int& all_a, int& all_b) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int ia = a, ib = b;
  warp_inclusive_sum2(ia, ib, lane);
  if (lane == 31) {
    sm.warp_a[wid] = ia;
    sm.warp_b[wid] = ib;
  }
  __syncthreads();
  all_a = all_b = 0;
  int before_a = ia - a, before_b = ib - b;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int x = sm.warp_a[w], y = sm.warp_b[w];
    before_a += w < wid ? x : 0;
    before_b += w < wid ? y : 0;
    all_a += x;
    all_b += y;
  }
  a = before_a;
  b = before_b;
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const cg::cluster_group cluster = cg::this_cluster();
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int row_i = blockIdx.x / C;
  const int s = row_i / a.c.Hkv, h = row_i - s * a.c.Hkv;
  const size_t width = static_cast<size_t>(a.c.width) << a.c.page_log2;
  const float* mass = a.mass + static_cast<size_t>(row_i) * width;
  float* mass_out = a.mass_out + static_cast<size_t>(row_i) * width;
  int32_t* origin = a.origin + static_cast<size_t>(row_i) * a.keep;
  int n = a.lens[s];
  if (n < 0 || static_cast<size_t>(n) > width) {
    if (tid == 0 && rank == 0) flag_error(a.dev_err, MOE_DEV_CAPACITY);
    n = 0;
  }
  const int kept = min(n, a.keep);
  const int all_threads = C * kThreads, all_tid = rank * kThreads + tid;
  if (h == 0 && all_tid == 0) a.new_len[s] = kept;
  for (int i = kept + all_tid; i < a.keep; i += all_threads) origin[i] = -1;
  if (n <= a.keep) {
    for (int i = all_tid; i < n; i += all_threads) {
      origin[i] = i;
      mass_out[i] = mass[i];
    }
    return;
  }
  const int free_n = n - a.recent;      // slots that may go
  const int want = a.keep - a.recent;   // of them, how many stay
  // This CTA's slots: [lo, lo + mine), `per` of them a thread, side by side.
  const int per = (n + all_threads - 1) / all_threads;
  const int lo = min(n, rank * per * kThreads), mine = min(n - lo, per * kThreads);
  for (int i = tid; i < 3 * kBins; i += kThreads) (&sm.hist[0][0])[i] = 0;
  bool nan = false;
  const int held = min(mine, kHeld);
  for (int i = tid; i < held; i += 8 * kThreads) {
    float m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = i + j * kThreads < held ? mass[lo + i + j * kThreads] : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      nan |= m[j] != m[j] && lo + i + j * kThreads < free_n;
      if (i + j * kThreads < held) sm.key[i + j * kThreads] = ordered(m[j]);
    }
  }
  auto key_of = [&](int i) { return i < kHeld ? sm.key[i] : ordered(mass[lo + i]); };
  for (int i = kHeld + tid; i < mine; i += kThreads) nan |= mass[lo + i] != mass[lo + i] && lo + i < free_n;
  if (nan) flag_error(a.dev_err, MOE_DEV_BAD_PROB);
  __syncthreads();
  // Radix select: the want-th largest key among the first free_n slots.
  uint32_t prefix = 0;
  int left = want;
  if (want > 0) {
    const int mine_free = max(0, min(mine, free_n - lo));
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      int* hist = sm.hist[pass];
      for (int i = tid; i < mine_free; i += kThreads) {
        const uint32_t k = key_of(i);
        if (pass == 0 || (k >> (shift + bits)) == (prefix >> (shift + bits))) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
      }
      cluster.sync();
      // Thread t adds up bins 4 t' .. 4 t' + 3, t' counting from the top.
      const int b0 = kBins - 4 - 4 * tid;
      int4 sum = make_int4(0, 0, 0, 0);
      for (int r = 0; r < C; ++r) {
        const int4 x = *reinterpret_cast<const int4*>(cluster.map_shared_rank(hist, r) + b0);
        sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
      }
      int above = sum.x + sum.y + sum.z + sum.w, zero = 0, all, all_zero;
      const int in4 = above;
      block_scan2(sm, above, zero, all, all_zero);  // above: keys in higher bins than these four
      if (above < left && above + in4 >= left) {
        int b = b0 + 3, rest = left - above;
        const int c4[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int j = 3; j > 0; --j)
          if (b == b0 + j && rest > c4[j]) {
            rest -= c4[j];
            --b;
          }
        sm.bin = b;
        sm.left = rest;
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(sm.bin) << shift;
      left = sm.left;
    }
  }
  // Kept: keys above `prefix`, the first `left` slots whose key equals it, and the recent ones.
  int above = 0, tie = 0;
  const int i0 = tid * per, i1 = min(mine, i0 + per);
  for (int i = i0; i < i1; ++i) {
    if (lo + i >= free_n) {
      ++above;
    } else if (want > 0) {
      const uint32_t k = key_of(i);
      above += k > prefix;
      tie += k == prefix;
    }
  }
  int all_above, all_tie;
  block_scan2(sm, above, tie, all_above, all_tie);
  if (tid == 0) {
    sm.count[0] = all_above;
    sm.count[1] = all_tie;
  }
  cluster.sync();
  for (int r = 0; r < rank; ++r) {
    const int* count = cluster.map_shared_rank(sm.count, r);
    above += count[0];
    tie += count[1];
  }
  for (int i = i0; i < i1; ++i) {
    bool stay = lo + i >= free_n;
    if (!stay && want > 0) {
      const uint32_t k = key_of(i);
      if (k == prefix) {
        if (tie < left) origin[above + tie] = lo + i;
        ++tie;
      }
      stay = k > prefix;
    }
    if (stay) origin[above++ + min(tie, left)] = lo + i;
  }
  cluster.sync();
  // Moves: D / 16 16-byte pieces of codes (K, then V) and one of 8 bytes of parameters per slot.
  constexpr int P = D / 16, kSlots = kThreads / P;
  const int x = tid % P, part = x / (P / 2), off = (x % (P / 2)) * 16;
  for (int r0 = 0; r0 < kept; r0 += C * kRound * kSlots) {
    int src[kRound], ps[kRound], pd[kRound];
    uint4 codes[kRound];
    uint2 par[kRound];
    float m[kRound];
    const int at = r0 + rank * kRound * kSlots + tid / P;
#pragma unroll
    for (int q = 0; q < kRound; ++q) src[q] = at + q * kSlots < kept ? origin[at + q * kSlots] : -1;
#pragma unroll
    for (int q = 0; q < kRound; ++q) {
      const int i = at + q * kSlots;
      ps[q] = pd[q] = -1;
      if (src[q] >= 0 && src[q] != i) {
        ps[q] = page_of(a.c, s, src[q]);
        pd[q] = page_of(a.c, s, i);
        if (x == 0 && (ps[q] < 0 || pd[q] < 0)) flag_error(a.dev_err, MOE_DEV_BAD_ID);
        if (ps[q] < 0) pd[q] = -1;
      }
    }
#pragma unroll
    for (int q = 0; q < kRound; ++q) {
      if (pd[q] >= 0) {
        const uint8_t* b = page_block(a.c, ps[q], h);
        const int r = src[q] & (a.c.page_size - 1);
        codes[q] = *reinterpret_cast<const uint4*>(b + (part * a.c.page_size + r) * (D / 2) + off);
        if (x == 0) par[q] = *reinterpret_cast<const uint2*>(b + a.c.page_size * D + r * 8);
      }
      if (x == 0 && src[q] >= 0) m[q] = mass[src[q]];
    }
    cluster.sync();
#pragma unroll
    for (int q = 0; q < kRound; ++q) {
      const int i = at + q * kSlots, r = i & (a.c.page_size - 1);
      if (pd[q] >= 0) {
        uint8_t* b = page_block(a.c, pd[q], h);
        *reinterpret_cast<uint4*>(b + (part * a.c.page_size + r) * (D / 2) + off) = codes[q];
        if (x == 0) *reinterpret_cast<uint2*>(b + a.c.page_size * D + r * 8) = par[q];
      }
      if (x == 0 && src[q] >= 0) mass_out[i] = m[q];
    }
  }
  for (int i = kept + all_tid; i < n; i += all_threads) mass_out[i] = 0.f;
}

// CTAs of a row: as many as keep the GPU's two places an SM filled, but no
// fewer than 512 slots each.  On the device, with 2, 4 and 8 CTAs a row: 32 rows of 2304
// slots 21.8, 16.6 and 22.6 us, 32 of up to 40k 59.8, 32.4 and 35.2.  The lengths
// are device data, so it goes by the slots that the table can hold: the former in
// a table of 36,864 slots take 22.9 us.
int cluster_size(const Cache& c) {
  const long long rows = static_cast<long long>(c.S) * c.Hkv, slots = static_cast<long long>(c.width) << c.page_log2;
  int n = 8;
  while (n > 1 && (rows * n > 2 * sm_count() || slots < 512ll * n)) n >>= 1;
  return n;
}

template <int D>
int launch_evict(const EvictArgs& a, cudaStream_t s) {
  const int st = allow_smem<evict_kernel<D>>(sizeof(Smem));
  if (st != MOE_OK) return st;
  const int n = cluster_size(a.c);
  LaunchScope ls(kProfKv4Evict, s);
  return launch_clusters(evict_kernel<D>, a.c.S * a.c.Hkv, n, kThreads, sizeof(Smem), s, a);
}

}  // namespace
}  // namespace kv4
}  // namespace moe

extern "C" int kv4_evict(const kv4_cache* cache, const float* mass, const int32_t* lens, const kv4_evict_cfg* cfg,
                         int32_t* new_len, int32_t* origin, float* mass_out, int32_t* dev_err, void* stream) {
  using namespace moe;
  using namespace moe::kv4;
  Cache c;
  int st = cache_validate(cache, &c);
  if (st != MOE_OK) return st;
  if (!cfg || cfg->keep < 1 || cfg->recent < 0 || cfg->recent > cfg->keep) return MOE_ERR_ARG;
  if (cfg->keep > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if (c.S == 0) return MOE_OK;
  if (!mass || !lens || !new_len || !origin || !mass_out) return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(mass) | reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(new_len) |
       reinterpret_cast<uintptr_t>(origin) | reinterpret_cast<uintptr_t>(mass_out)) & 3)
    return MOE_ERR_ARG;
  EvictArgs a{c, mass, lens, cfg->keep, cfg->recent, new_len, origin, mass_out, dev_err};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return c.D == 128 ? launch_evict<128>(a, s) : launch_evict<64>(a, s);
}
