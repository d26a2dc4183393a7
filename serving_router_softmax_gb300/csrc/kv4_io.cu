// kv4_append / kv4_read: rows of keys and values into and out of the 4-bit
// paged cache.
//
// Both are bound by memory: a row of D values is read once and its D / 2
// bytes of codes and 4 bytes of parameters are written once (or the other
// way round).  D / 8 lanes take one row of K or V of one token and head, 8
// values each: one or two 16-byte accesses on the value side, 4 bytes a lane
// on the code side (a row's 32 or 64 bytes side by side).
#include "kv4.cuh"

namespace moe {
namespace kv4 {

int cache_validate(const kv4_cache* c, Cache* out) {
  if (!c) return MOE_ERR_ARG;
  if (c->n_pages < 0 || c->n_seq < 0 || c->max_pages < 1 || c->n_kv_heads < 1) return MOE_ERR_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return MOE_ERR_UNSUPPORTED;
  int lg = 4;
  while (lg < 8 && (1 << lg) != c->page_size) ++lg;
  if ((1 << lg) != c->page_size) return MOE_ERR_UNSUPPORTED;
  if (c->n_kv_heads > 1024 || c->n_seq > kMaxSeq) return MOE_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->max_pages) * c->page_size > (1ll << 30)) return MOE_ERR_UNSUPPORTED;
  if (!c->table || (c->n_pages > 0 && !c->pages)) return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(c->pages) & 15) || (reinterpret_cast<uintptr_t>(c->table) & 3)) return MOE_ERR_ARG;
  *out = Cache{static_cast<uint8_t*>(c->pages), c->table, c->n_pages, c->page_size, lg,
               c->n_kv_heads, c->head_dim, c->n_seq, c->max_pages};
  return MOE_OK;
}

namespace {

constexpr int kIoThreads = 256;

struct IoArgs {
  Cache c;
  const void* x[2];         // k, v
  long long ts[2], hs[2];   // their token and head strides, in elements
  const int32_t* seq;
  const int32_t* slot;
  int32_t T;
  void* y[2];               // append: held values (or NULL); read: outputs; [T, Hkv, D]
  int32_t* dev_err;
};

template <bool F32>
__device__ __forceinline__ void load8(const void* p, long long i, float (&v)[8]) {
  if constexpr (F32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(u[j] << 16);
      v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, long long i, const float (&v)[8]) {
  if constexpr (F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
  }
}

// (hi - lo) / 15 rounded to fp32: the difference as an unrounded sum of two
// numbers, the quotient corrected by its remainder.
__device__ __forceinline__ float fifteenth(float hi, float lo) {
  const float d = hi - lo, b = d - hi;
  const float tail = (hi - (d - b)) + (-lo - b);
  const float q = d / 15.f;
  return fmaf(fmaf(-q, 15.f, d) + tail, 1.f / 15.f, q);
}

// The code of x: the whole number nearest to the real quotient (x - zero) /
// scale, ties to even, within 0..15.  The fp32 quotient is within 3e-6 of the
// real one (three roundings of a number below 16); where that leaves the nearest code open it is taken in 64 bits.
__device__ __forceinline__ uint32_t code_of(float x, float zero, float scale, float inv) {
  const float q = (x - zero) * inv;
  float r = rintf(q);
  if (fabsf(q - r) > 0.49999f && q < 16.f)
    r = static_cast<float>(rint((static_cast<double>(x) - static_cast<double>(zero)) / static_cast<double>(scale)));
  return static_cast<uint32_t>(fminf(fmaxf(r, 0.f), 15.f));
}

template <int D, bool F32>
__global__ void __launch_bounds__(kIoThreads) append_kernel(const IoArgs a) {
  constexpr int LPR = D / 8;
  pdl_wait();
  pdl_trigger();
  const long long i = static_cast<long long>(blockIdx.x) * (kIoThreads / LPR) + threadIdx.x / LPR;
  const int x = threadIdx.x % LPR;
  // row i = (token, head, K or V), K and V of a head side by side
  const int part = static_cast<int>(i & 1);
  const int h = static_cast<int>((i >> 1) % a.c.Hkv);
  const long long t = (i >> 1) / a.c.Hkv;
  if (t >= a.T) return;
  const int s = a.seq[t], j = a.slot[t];
  float v[8];
  load8<F32>(a.x[part], t * a.ts[part] + h * a.hs[part] + 8 * x, v);
  float lo = v[0], hi = v[0], sum = 0.f;
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    lo = fminf(lo, v[d]);
    hi = fmaxf(hi, v[d]);
    sum += fabsf(v[d]) * 0.0078125f;  // not finite (or far out of range) when a value is not: min and max drop a NaN
  }
  const uint32_t mask = ((LPR == 32 ? 0u : (1u << LPR)) - 1u) << ((threadIdx.x & 31) / LPR * LPR);
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(mask, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(mask, hi, o));
    sum += __shfl_xor_sync(mask, sum, o);
  }
  const bool ok_value = sum - sum == 0.f && lo >= -65504.f && hi <= 65504.f;
  const int page = j >= 0 && s >= 0 && s < a.c.S ? page_of(a.c, s, j) : -1;
  if (x == 0 && ((j != -1 && page < 0) || (j >= 0 && !ok_value)))
    flag_error(a.dev_err, (page < 0 ? MOE_DEV_BAD_ID : 0) | (ok_value ? 0 : MOE_DEV_BAD_KV));
  __half scale = __float2half_rn(fifteenth(hi, lo));
  __half zero = __float2half_rn(lo);
  if (!ok_value) {
    scale = __float2half_rn(0.f);
    zero = __ushort_as_half(0x7E00);
  }
  const float sf = __half2float(scale), zf = __half2float(zero);
  const float inv = sf > 0.f ? 1.f / sf : 0.f;
  uint32_t codes = 0;
  float held[8];
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    const uint32_t q = ok_value && sf > 0.f ? code_of(v[d], zf, sf, inv) : 0u;
    codes |= q << (4 * d);
    held[d] = fmaf(sf, static_cast<float>(q), zf);
  }
  if (a.y[part]) {
    if (page < 0) {
#pragma unroll
      for (int d = 0; d < 8; ++d) held[d] = 0.f;
    }
    store8<F32>(a.y[part], (t * a.c.Hkv + h) * D + 8 * x, held);
  }
  if (page < 0) return;
  const int r = j & (a.c.page_size - 1);
  uint8_t* b = page_block(a.c, page, h);
  *reinterpret_cast<uint32_t*>(b + (static_cast<size_t>(part) * a.c.page_size + r) * (D / 2) + 4 * x) = codes;
  if (x == 0)
    *reinterpret_cast<__half2*>(b + static_cast<size_t>(a.c.page_size) * D + r * 8 + part * 4) = __halves2half2(scale, zero);
}

template <int D, bool F32>
__global__ void __launch_bounds__(kIoThreads) read_kernel(const IoArgs a) {
  constexpr int LPR = D / 8;
  pdl_wait();
  pdl_trigger();
  const long long i = static_cast<long long>(blockIdx.x) * (kIoThreads / LPR) + threadIdx.x / LPR;
  const int x = threadIdx.x % LPR;
  const int part = static_cast<int>(i & 1);
  const int h = static_cast<int>((i >> 1) % a.c.Hkv);
  const long long t = (i >> 1) / a.c.Hkv;
  if (t >= a.T) return;
  const int s = a.seq[t], j = a.slot[t];
  const int page = j >= 0 && s >= 0 && s < a.c.S ? page_of(a.c, s, j) : -1;
  if (x == 0 && j != -1 && page < 0) flag_error(a.dev_err, MOE_DEV_BAD_ID);
  float v[8];
#pragma unroll
  for (int d = 0; d < 8; ++d) v[d] = 0.f;
  if (page >= 0) {
    const int r = j & (a.c.page_size - 1);
    const uint8_t* b = page_block(a.c, page, h);
    const uint32_t codes = *reinterpret_cast<const uint32_t*>(b + (static_cast<size_t>(part) * a.c.page_size + r) * (D / 2) + 4 * x);
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(b + static_cast<size_t>(a.c.page_size) * D + r * 8 + part * 4));
#pragma unroll
    for (int d = 0; d < 8; ++d) v[d] = fmaf(p.x, static_cast<float>((codes >> (4 * d)) & 15u), p.y);
  }
  store8<F32>(a.y[part], (t * a.c.Hkv + h) * D + 8 * x, v);
}

template <bool Append>
int launch_io(const IoArgs& a, bool f32, cudaStream_t s) {
  const long long rows = 2ll * a.T * a.c.Hkv;
  const int per = kIoThreads / (a.c.D / 8);
  const dim3 grid(static_cast<unsigned>((rows + per - 1) / per));
  void (*k)(IoArgs);
  if (Append)
    k = a.c.D == 128 ? (f32 ? append_kernel<128, true> : append_kernel<128, false>)
                     : (f32 ? append_kernel<64, true> : append_kernel<64, false>);
  else
    k = a.c.D == 128 ? (f32 ? read_kernel<128, true> : read_kernel<128, false>)
                     : (f32 ? read_kernel<64, true> : read_kernel<64, false>);
  LaunchScope ls(Append ? kProfKv4Append : kProfKv4Read, s);
  return launch_k(k, grid, dim3(kIoThreads), 0, s, false, a);
}

// The row count must fit the grid, and 16-byte accesses the rows.
int rows_validate(const kv4_rows_cfg* cfg, const Cache& c) {
  if (!cfg || cfg->T < 0) return MOE_ERR_ARG;
  if (cfg->dtype != MOE_DTYPE_F32 && cfg->dtype != MOE_DTYPE_BF16) return MOE_ERR_UNSUPPORTED;
  if (static_cast<long long>(cfg->T) * c.Hkv > (1ll << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

}  // namespace
}  // namespace kv4
}  // namespace moe

extern "C" int kv4_append(const kv4_cache* cache, const void* k, const void* v, const kv4_rows_cfg* cfg,
                          const int32_t* seq, const int32_t* slot, void* k_held, void* v_held, int32_t* dev_err,
                          void* stream) {
  using namespace moe;
  using namespace moe::kv4;
  Cache c;
  int st = cache_validate(cache, &c);
  if (st != MOE_OK || (st = rows_validate(cfg, c)) != MOE_OK) return st;
  if (cfg->T == 0) return MOE_OK;
  if (!k || !v || !seq || !slot || (!k_held != !v_held)) return MOE_ERR_ARG;
  const int per = cfg->dtype == MOE_DTYPE_F32 ? 4 : 8;  // elements of 16 bytes
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(k_held, 16) || misaligned(v_held, 16) ||
      misaligned(seq, 4) || misaligned(slot, 4))
    return MOE_ERR_ARG;
  for (long long x : {cfg->k_token_stride, cfg->k_head_stride, cfg->v_token_stride, cfg->v_head_stride})
    if (x < 0 || x % per) return MOE_ERR_UNSUPPORTED;
  IoArgs a{c, {k, v}, {cfg->k_token_stride, cfg->v_token_stride}, {cfg->k_head_stride, cfg->v_head_stride},
           seq, slot, cfg->T, {k_held, v_held}, dev_err};
  return launch_io<true>(a, cfg->dtype == MOE_DTYPE_F32, static_cast<cudaStream_t>(stream));
}

extern "C" int kv4_read(const kv4_cache* cache, const int32_t* seq, const int32_t* slot, const kv4_rows_cfg* cfg,
                        void* k, void* v, int32_t* dev_err, void* stream) {
  using namespace moe;
  using namespace moe::kv4;
  Cache c;
  int st = cache_validate(cache, &c);
  if (st != MOE_OK || (st = rows_validate(cfg, c)) != MOE_OK) return st;
  if (cfg->T == 0) return MOE_OK;
  if (!k || !v || !seq || !slot) return MOE_ERR_ARG;
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(seq, 4) || misaligned(slot, 4)) return MOE_ERR_ARG;
  IoArgs a{c, {nullptr, nullptr}, {0, 0}, {0, 0}, seq, slot, cfg->T, {k, v}, dev_err};
  return launch_io<false>(a, cfg->dtype == MOE_DTYPE_F32, static_cast<cudaStream_t>(stream));
}
