// moe_prompt_attend: causal attention of packed prompts.
//
// First form: a warp per row of a query head walks its keys, the running
// maximum and sum beside the output in registers.
#include <cmath>

#include "common.cuh"

namespace moe {
namespace {

struct PromptArgs {
  const uint16_t *q, *k, *v;
  const int32_t* start;
  uint16_t* out;
  float* lse;
  int32_t* dev_err;
  long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;
  int T, S, Hq, G;
  float scale;
};

template <int D>
__global__ void __launch_bounds__(256) attend_rows_kernel(const PromptArgs a) {
  constexpr int W = D / 32;
  const int lane = threadIdx.x & 31;
  const long long item = blockIdx.x * 8ll + (threadIdx.x >> 5);
  if (item >= static_cast<long long>(a.T) * a.Hq) return;
  const int t = static_cast<int>(item / a.Hq), h = static_cast<int>(item % a.Hq), kh = h / a.G;
  int first = -1;
  for (int s = 0; s < a.S; ++s) {
    const int b = a.start[s], e = a.start[s + 1];
    if (b < 0 || e > a.T || b > e) {
      if (lane == 0) flag_error(a.dev_err, MOE_DEV_CAPACITY);
      return;
    }
    if (t >= b && t < e) first = b;
  }
  if (first < 0) return;
  float q[W], o[W];
  for (int i = 0; i < W; ++i) q[i] = bf16_bits_to_float(a.q[t * a.q_ts + h * a.q_hs + lane + 32 * i]), o[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int j = first; j <= t; ++j) {
    float s = 0.f;
    for (int i = 0; i < W; ++i) s += q[i] * bf16_bits_to_float(a.k[j * a.k_ts + kh * a.k_hs + lane + 32 * i]);
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    s *= a.scale;
    if (s == -INFINITY) continue;
    const float top = fmaxf(m, s), f = m == -INFINITY ? 0.f : __expf(m - top), p = __expf(s - top);
    l = l * f + p;
    for (int i = 0; i < W; ++i) o[i] = o[i] * f + p * bf16_bits_to_float(a.v[j * a.v_ts + kh * a.v_hs + lane + 32 * i]);
    m = top;
  }
  const float r = l == 0.f ? 0.f : 1.f / l;
  for (int i = 0; i < W; ++i) {
    const float x = o[i] * r;
    a.out[item * D + lane + 32 * i] = x == x ? float_to_bf16_bits_rn(x) : 0x7FFF;
  }
  if (a.lse && lane == 0) a.lse[item] = l == 0.f ? -INFINITY : m + logf(l);
}

bool stride_ok(long long st, int n) { return n <= 1 || (st >= 0 && st % 8 == 0 && st < (1ll << 38)); }

}  // namespace
}  // namespace moe

extern "C" int moe_prompt_attend(const void* q, const void* k, const void* v, const int32_t* start,
                                 const moe_prompt_cfg* cfg, void* out, float* lse, int32_t* dev_err, void* stream) {
  using namespace moe;
  if (!cfg) return MOE_ERR_ARG;
  const moe_prompt_cfg& c = *cfg;
  if (c.T < 0 || c.n_seq < 0 || c.n_q_heads < 1 || c.n_kv_heads < 1 || !std::isfinite(c.scale)) return MOE_ERR_ARG;
  if (c.n_q_heads % c.n_kv_heads) return MOE_ERR_ARG;
  if (c.head_dim != 64 && c.head_dim != 128) return MOE_ERR_UNSUPPORTED;
  if (c.T > (1 << 24) || c.n_seq > 4096 || c.n_q_heads > 1024 || c.n_q_heads / c.n_kv_heads > 128) return MOE_ERR_UNSUPPORTED;
  if (!stride_ok(c.q_token_stride, c.T) || !stride_ok(c.q_head_stride, c.n_q_heads) || !stride_ok(c.k_token_stride, c.T) ||
      !stride_ok(c.k_head_stride, c.n_kv_heads) || !stride_ok(c.v_token_stride, c.T) || !stride_ok(c.v_head_stride, c.n_kv_heads))
    return MOE_ERR_UNSUPPORTED;
  if (c.T == 0 || c.n_seq == 0) return MOE_OK;
  if (!q || !k || !v || !start || !out) return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
       reinterpret_cast<uintptr_t>(out)) & 15 ||
      (reinterpret_cast<uintptr_t>(start) | reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(dev_err)) & 3)
    return MOE_ERR_ARG;
  auto st = [](long long x, int n) { return n <= 1 ? 0 : x; };
  const PromptArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), start,
                     static_cast<uint16_t*>(out), lse, dev_err, st(c.q_token_stride, c.T), st(c.q_head_stride, c.n_q_heads),
                     st(c.k_token_stride, c.T), st(c.k_head_stride, c.n_kv_heads), st(c.v_token_stride, c.T),
                     st(c.v_head_stride, c.n_kv_heads), c.T, c.n_seq, c.n_q_heads, c.n_q_heads / c.n_kv_heads, c.scale};
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(c.T) * c.n_q_heads + 7) / 8);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  LaunchScope ls(kProfPrompt, s);
  if (c.head_dim == 64)
    attend_rows_kernel<64><<<blocks, 256, 0, s>>>(a);
  else
    attend_rows_kernel<128><<<blocks, 256, 0, s>>>(a);
  return check_launch();
}
