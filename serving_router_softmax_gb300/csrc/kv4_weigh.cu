// kv4_weigh: adds to every slot the softmax weight that the new tokens gave it.
//
//   mass[s, h, j] += sum over the query rows i of kv head h: exp(S_ij - lse_i)
//
// with the lse of kv4_attend, so one pass over the keys alone (half the
// cache): a warp holds the codes of 16 slots in registers as the matrix row
// operand, goes through all query rows in steps of 8 and sums its slots'
// weights in fp32 in a fixed order; no atomics.
#include "kv4.cuh"
#include "kv4_sched.cuh"

namespace moe {
namespace kv4 {

int attn_validate(const kv4_attn_cfg* cfg, const Cache& c);

namespace {

constexpr int kWarps = 8;
constexpr int kSlots = 16 * kWarps;  // slots of a unit
constexpr int kRows = 128;           // query rows held at a time
constexpr int kAllRows = 1 << 30;    // one row block per kv head

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
};

template <int D>
struct Smem {
  uint2 frag[kRows / 8 * (D / 16) * 32];
  float cq[kRows], cqs[kRows], lse2[kRows];
  uint64_t mask[kRows];
  int token[kRows];
  long long scratch[32];
  long long cum[1];
};

template <int D>
__global__ void __launch_bounds__(32 * kWarps) weigh_kernel(const WeighArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  pdl_wait();
  pdl_trigger();
  build_units(a.c, a.q_start, a.base, a.T, a.G, kAllRows, kSlots, 0, sm.cum, sm.scratch, a.dev_err, blockIdx.x == 0);
  const long long total = sm.cum[a.c.S];
  const long long u0 = total * blockIdx.x / gridDim.x, u1 = total * (blockIdx.x + 1) / gridDim.x;
  const size_t width = static_cast<size_t>(a.c.width) << a.c.page_log2;
  Cursor k;
  if (u0 < u1) cursor_at(k, a.c, a.q_start, a.base, a.T, a.G, kAllRows, kSlots, 0, sm.cum, u0);
  int held_s = -1, held_h = -1, held_row = -1;  // query rows in shared memory
  for (long long u = u0; u < u1; ++u) {
    if (k.tile == k.nt) cursor_next(k, a.c, a.q_start, a.base, a.T, a.G, kAllRows, kSlots, 0, sm.cum);
    const int j0 = k.tile * kSlots + 16 * warp;
    const int page = j0 < k.q.total ? page_of(a.c, k.s, j0) : -1;
    if (page < 0 && j0 < k.q.total && lane == 0) flag_error(a.dev_err, MOE_DEV_BAD_ID);
    uint32_t ka[D / 32] = {}, kb[D / 32] = {};
    float2 pa = make_float2(0.f, 0.f), pb = pa;
    const int sa = slot_of_row(g), sb = slot_of_row(g + 8);
    float* mass = a.mass + (static_cast<size_t>(k.s) * a.c.Hkv + k.h) * width;
    if (page >= 0) {
      const uint8_t* b = page_block(a.c, page, k.h);
      const int r0 = j0 & (a.c.page_size - 1);
      load_k_words<D>(b + static_cast<size_t>(r0 + sa) * (D / 2), c, ka);
      load_k_words<D>(b + static_cast<size_t>(r0 + sb) * (D / 2), c, kb);
      const uint8_t* p = b + static_cast<size_t>(a.c.page_size) * D;
      pa = __half22float2(*reinterpret_cast<const __half2*>(p + (r0 + sa) * 8));
      pb = __half22float2(*reinterpret_cast<const __half2*>(p + (r0 + sb) * 8));
    }
    const bool edge = j0 + 16 > k.q.base;
    float wa = 0.f, wb = 0.f;
    const int all = k.q.nq * a.G;
    if (a.visible && k.q.nq > kMaxTree && tid == 0) flag_error(a.dev_err, MOE_DEV_CAPACITY);
    for (int row0 = 0; row0 < all; row0 += kRows) {
      const int rows = min(kRows, all - row0), padded = (rows + 7) & ~7;
      if (k.s != held_s || k.h != held_h || row0 != held_row) {
        __syncthreads();
        prep_q<D>(
            [&](int r) -> const uint16_t* {
              if (r >= rows) return nullptr;
              const int i = (row0 + r) / a.G, x = (row0 + r) - i * a.G;
              return a.q + (k.q.q0 + i) * a.q_ts + static_cast<long long>(k.h * a.G + x) * a.q_hs;
            },
            padded, a.scale_log2, sm.frag, sm.cq, sm.cqs, tid, 32 * kWarps);
        for (int r = tid; r < padded; r += 32 * kWarps) {
          const int i = (row0 + min(r, rows - 1)) / a.G, x = (row0 + r) - i * a.G;
          float v = INFINITY;
          if (r < rows) {
            v = a.lse[(static_cast<size_t>(k.q.q0) + i) * a.Hq + k.h * a.G + x] * kLog2e;
            if (v == -INFINITY) v = INFINITY;  // a row that saw nothing gives no weight
          }
          sm.lse2[r] = v;
          // such a row sees no new slot either, whatever those hold
          sm.token[r] = v == INFINITY ? -1 : i;
          sm.mask[r] = a.visible && v != INFINITY ? a.visible[k.q.q0 + i] : 0;
        }
        held_s = k.s, held_h = k.h, held_row = row0;
        __syncthreads();
      }
      if (page < 0) continue;
      for (int t = 0; t < padded / 8; ++t) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        qk_16x8<D>(acc, ka, kb, [&](int i) { return sm.frag[(t * (D / 16) + i) * 32 + lane]; });
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 8 * t + 2 * c + (e & 1);
          const float2 p = e < 2 ? pa : pb;
          float w = ex2(fmaf(p.x, acc[e] * sm.cq[r], fmaf(p.y, sm.cqs[r], -sm.lse2[r])));
          if (edge) {
            const int j = j0 + (e < 2 ? sa : sb), d = j - k.q.base;
            bool see = d < 0;
            if (!see && j < k.q.total) see = a.visible ? d < kMaxTree && ((sm.mask[r] >> d) & 1) : d <= sm.token[r];
            w = see ? w : 0.f;
          }
          if (e < 2) wa += w;
          else wb += w;
        }
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      wa += __shfl_xor_sync(0xFFFFFFFFu, wa, o);
      wb += __shfl_xor_sync(0xFFFFFFFFu, wb, o);
    }
    if (page >= 0 && c == 0) {
      if (j0 + sa < k.q.total) mass[j0 + sa] += wa;
      if (j0 + sb < k.q.total) mass[j0 + sb] += wb;
    }
    ++k.tile;
  }
}

template <int D>
int launch_weigh(const WeighArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(Smem<D>) + static_cast<size_t>(a.c.S) * 8;
  const int st = allow_smem<weigh_kernel<D>>(smem);
  if (st != MOE_OK) return st;
  LaunchScope ls(kProfKv4Weigh, s);
  return launch_k(weigh_kernel<D>, dim3(sm_count() * 3), dim3(32 * kWarps), smem, s, false, a);
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
              mass, cfg->T, cfg->n_q_heads, cfg->n_q_heads / c.Hkv, cfg->scale * kLog2e, dev_err};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return c.D == 128 ? launch_weigh<128>(a, s) : launch_weigh<64>(a, s);
}
