// kv4_evict: brings a cache down to its budget by accumulated attention weight.
//
// Per sequence and kv head, of n slots: the last `recent` stay, and of the
// others those with the largest mass (equal ones: the lower slot) until
// `keep` are kept; they move to slots 0..keep-1 in their old order, codes and
// parameters together, so slots stay in the order in which tokens came.
//
// One CTA per (sequence, head): the smallest kept mass by a radix select on
// the masses' ordered bits (8 bits a pass), the kept slots in order by a
// running count, then the moves.  Moves go in chunks in ascending order, each
// read whole before it is written; a slot never moves up, so a chunk writes
// nothing that a later one reads.
#include "kv4.cuh"

namespace moe {
namespace kv4 {
namespace {

constexpr int kThreads = 1024;

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

// Bits whose unsigned order is the masses' order; a NaN is below everything, -0 equals +0.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

template <int D>
__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_a[32], warp_b[32];
  __shared__ int s_bin, s_left;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int s = blockIdx.x / a.c.Hkv, h = blockIdx.x % a.c.Hkv;
  const size_t width = static_cast<size_t>(a.c.width) << a.c.page_log2;
  const size_t row = static_cast<size_t>(s) * a.c.Hkv + h;
  const float* mass = a.mass + row * width;
  float* mass_out = a.mass_out + row * width;
  int32_t* origin = a.origin + row * a.keep;
  int n = a.lens[s];
  if (n < 0 || static_cast<size_t>(n) > width) {
    if (tid == 0) flag_error(a.dev_err, MOE_DEV_CAPACITY);
    n = 0;
  }
  const int kept = min(n, a.keep);
  if (h == 0 && tid == 0) a.new_len[s] = kept;
  for (int i = kept + tid; i < a.keep; i += kThreads) origin[i] = -1;
  if (n <= a.keep) {
    for (int i = tid; i < n; i += kThreads) {
      origin[i] = i;
      mass_out[i] = mass[i];
    }
    return;
  }
  const int free_n = n - a.recent;    // slots that may go
  int want = a.keep - a.recent;       // of them, how many stay
  // Radix select: the want-th largest key among the first free_n.
  uint32_t prefix = 0;
  bool nan = false;
  int left = want;
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < free_n; i += kThreads) {
        const float m = mass[i];
        nan |= m != m;
        const uint32_t key = ordered(m);
        if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int b = 255, rest = left;
        while (b > 0 && hist[b] < rest) rest -= hist[b--];
        s_bin = b;
        s_left = rest;
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(s_bin) << shift;
      left = s_left;
      __syncthreads();
    }
  }
  if (nan) flag_error(a.dev_err, MOE_DEV_BAD_PROB);
  // Kept: keys above `prefix`, the first `left` slots whose key equals it, and
  // the recent ones; positions in slot order.
  int kept_before = 0, ties_before = 0;
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + tid;
    bool above = false, tie = false;
    if (i < n) {
      if (i >= free_n) above = true;
      else if (want > 0) {
        const uint32_t key = ordered(mass[i]);
        above = key > prefix;
        tie = key == prefix;
      }
    }
    const uint32_t tb = __ballot_sync(0xFFFFFFFFu, tie);
    if (lane == 0) warp_a[wid] = __popc(tb);
    __syncthreads();
    int ties = ties_before + __popc(tb & ((1u << lane) - 1u)), ties_all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      ties += w < wid ? warp_a[w] : 0;
      ties_all += warp_a[w];
    }
    const bool stay = above || (tie && ties < left);
    const uint32_t sb = __ballot_sync(0xFFFFFFFFu, stay);
    if (lane == 0) warp_b[wid] = __popc(sb);
    __syncthreads();
    int pos = kept_before + __popc(sb & ((1u << lane) - 1u)), all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      pos += w < wid ? warp_b[w] : 0;
      all += warp_b[w];
    }
    if (stay) origin[pos] = i;
    kept_before += all;
    ties_before += ties_all;
  }
  __syncthreads();
  // Moves: D / 16 16-byte pieces of codes (K, then V) and one of 8 bytes of parameters per slot.
  constexpr int P = D / 16;
  constexpr int kChunk = kThreads / P;
  const int x = tid % P, part = x / (P / 2), off = (x % (P / 2)) * 16;
  for (int i0 = 0; i0 < kept; i0 += kChunk) {
    const int i = i0 + tid / P;
    const int src = i < kept ? origin[i] : i;
    const bool move = i < kept && src != i;
    int ps = -1, pd = -1;
    uint4 codes = make_uint4(0, 0, 0, 0);
    uint2 par = make_uint2(0, 0);
    float m = 0.f;
    const int rs = src & (a.c.page_size - 1), rd = i & (a.c.page_size - 1);
    if (move) {
      ps = page_of(a.c, s, src);
      pd = page_of(a.c, s, i);
      if (x == 0 && (ps < 0 || pd < 0)) flag_error(a.dev_err, MOE_DEV_BAD_ID);
      if (ps >= 0 && pd >= 0) {
        const uint8_t* b = page_block(a.c, ps, h);
        codes = *reinterpret_cast<const uint4*>(b + (static_cast<size_t>(part) * a.c.page_size + rs) * (D / 2) + off);
        if (x == 0) par = *reinterpret_cast<const uint2*>(b + static_cast<size_t>(a.c.page_size) * D + rs * 8);
      }
    }
    if (x == 0 && i < kept) m = mass[src];
    __syncthreads();
    if (move && ps >= 0 && pd >= 0) {
      uint8_t* b = page_block(a.c, pd, h);
      *reinterpret_cast<uint4*>(b + (static_cast<size_t>(part) * a.c.page_size + rd) * (D / 2) + off) = codes;
      if (x == 0) *reinterpret_cast<uint2*>(b + static_cast<size_t>(a.c.page_size) * D + rd * 8) = par;
    }
    if (x == 0 && i < kept) mass_out[i] = m;
    __syncthreads();
  }
  for (int i = kept + tid; i < n; i += kThreads) mass_out[i] = 0.f;
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
  if (static_cast<long long>(c.S) * c.Hkv * cfg->keep > (1ll << 40)) return MOE_ERR_UNSUPPORTED;
  if (c.S == 0) return MOE_OK;
  if (!mass || !lens || !new_len || !origin || !mass_out) return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(mass) | reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(new_len) |
       reinterpret_cast<uintptr_t>(origin) | reinterpret_cast<uintptr_t>(mass_out)) & 3)
    return MOE_ERR_ARG;
  EvictArgs a{c, mass, lens, cfg->keep, cfg->recent, new_len, origin, mass_out, dev_err};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  LaunchScope ls(kProfKv4Evict, s);
  return launch_k(c.D == 128 ? evict_kernel<128> : evict_kernel<64>, dim3(static_cast<unsigned>(c.S) * c.Hkv),
                  dim3(kThreads), 0, s, false, a);
}
