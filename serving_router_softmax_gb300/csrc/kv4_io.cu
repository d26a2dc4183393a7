// kv4_append / kv4_read: rows of keys and values into and out of the 4-bit
// paged cache.
//
// Both are bound by memory: a row of D values is read once and its D / 2
// bytes of codes and 4 bytes of parameters are written once (or the other
// way round).  The lanes of a row of K or V of one token and head take 16 bytes
// of values each, side by side, 4 (fp32) or 8 (bf16) of them, and the 2 or 4
// bytes of their codes.  A warp's rows share their token's look-up
// (with one a row the first below took 147 us, the second 72).  Append of 32,768 bf16 tokens of 8 heads of 128 with the
// held values out: 72 us, 62% of the copy rate (82 before the quotients and held values went two to an
// instruction).  What is left of the conversion and the two reductions a row keep it from more: issue slots 72% busy,
// the ALU pipe 70%.  On the device four CTAs an SM take 70 us, three 79, five 73, six 75.  Read of as many to fp32: 55 us,
// 81%.  7 tokens appended 2.3 us, 333 read 2.0, under the host's 12 to 16 a call.
#include "kv4.cuh"
#include "tc_f16.cuh"

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
  if ((c->n_seq > 0 && !c->table) || (c->n_pages > 0 && !c->pages)) return MOE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(c->pages) & 15) || (reinterpret_cast<uintptr_t>(c->table) & 3)) return MOE_ERR_ARG;
  *out = Cache{static_cast<uint8_t*>(c->pages), c->table, c->n_pages, c->page_size, lg,
               c->n_kv_heads, c->head_dim, c->n_seq, c->max_pages};
  return MOE_OK;
}

namespace {

using tc::add2;
using tc::fma2;

constexpr int kIoThreads = 256;

struct IoArgs {
  Cache c;
  const void* x[2];         // k, v
  long long ts[2], hs[2];   // their token and head strides, in elements
  const int32_t* seq;
  const int32_t* slot;
  int32_t T;
  int32_t groups;           // warps of a token
  void* y[2];               // append: held values (or NULL); read: outputs; [T, Hkv, D]
  int32_t* dev_err;
};

// 16 bytes of values: 4 fp32 or 8 bf16.
template <int E>
__device__ __forceinline__ void values_of(const uint4& r, float (&v)[E]) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (E == 4) {
      v[j] = __uint_as_float(u[j]);
    } else {
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

template <int E>
__device__ __forceinline__ void store_values(void* p, long long i, const float (&v)[E]) {
  if constexpr (E == 4)
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
}

// The larger; NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}

__device__ __forceinline__ uint32_t max2_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Smallest and largest value of a row (the latter NaN if one value is), in all its lanes.
template <int E, int LPR>
__device__ __forceinline__ void extremes(const uint4& r, const float (&v)[E], float& lo, float& hi) {
  if constexpr (E == 4) {
    lo = min3(fminf(v[0], v[1]), v[2], v[3]);
    hi = max_nan(max_nan(v[0], v[1]), v[2], v[3]);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
    }
  } else {
    // Two bf16 at a time: the largest of the values and of their opposites.
    constexpr uint32_t kSigns = 0x80008000u;
    const uint32_t p = max2_bf16(max2_bf16(r.x, r.y), max2_bf16(r.z, r.w));
    const uint32_t n = max2_bf16(max2_bf16(r.x ^ kSigns, r.y ^ kSigns), max2_bf16(r.z ^ kSigns, r.w ^ kSigns));
    uint32_t m = max2_bf16(__byte_perm(p, n, 0x5410), __byte_perm(p, n, 0x7632));  // (largest, largest opposite)
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = max2_bf16(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    hi = __uint_as_float(m << 16);
    lo = -__uint_as_float(m & 0xFFFF0000u);
  }
}

// (hi - lo) / 15 rounded to fp32: the difference as an unrounded sum of two
// numbers (Knuth's TwoSum, The Art of Computer Programming vol. 2, 4.2.2), the
// quotient corrected by its remainder (Markstein 1990).
__device__ __forceinline__ float fifteenth(float hi, float lo) {
  const float d = hi - lo, b = d - hi;
  const float tail = (hi - (d - b)) + (-lo - b);
  const float q = d * (1.f / 15.f);
  return fmaf(fmaf(-q, 15.f, d) + tail, 1.f / 15.f, q);
}

// Which of k and k + 1 is the whole number nearest to the real quotient
// (x - zero) / scale, known to lie within 1e-5 of k + 1/2; ties to even.  Exact
// in fp32: (k + 1/2) scale has 16 bits, x - zero is an unrounded sum of two
// numbers (TwoSum), and the larger of them is so near to the former that their
// difference has no rounding.
__device__ __forceinline__ float nearer(float x, float zero, float scale, float k) {
  const float d = x - zero, b = d - x;
  const float tail = (x - (d - b)) + (-zero - b);
  const float t = fmaf(-(k + 0.5f), scale, d) + tail;
  return t > 0.f || (t == 0.f && (static_cast<int>(k) & 1)) ? k + 1.f : k;
}

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: a sum with it is rounded to a whole number (ties to even)

// A warp's rows: U passes of 32 / LPR rows of one token (first all K heads,
// then all V heads).  The token's place is looked up once for all of them and
// their loads are on their way together, which is what keeps memory busy: the
// look-up is a chain of three loads.
struct TokenRows {
  int t, first, s, j, page;
};
template <int U, int LPR>
__device__ __forceinline__ bool token_rows(const IoArgs& a, TokenRows& r) {
  const uint32_t w = blockIdx.x * (kIoThreads / 32) + (threadIdx.x >> 5);
  const uint32_t t = w / static_cast<uint32_t>(a.groups);
  if (t >= static_cast<uint32_t>(a.T)) return false;
  r.t = static_cast<int>(t);
  r.first = static_cast<int>(w - t * static_cast<uint32_t>(a.groups)) * (U * (32 / LPR)) + (threadIdx.x & 31) / LPR;
  r.s = a.seq[t];
  r.j = a.slot[t];
  r.page = r.j >= 0 && r.s >= 0 && r.s < a.c.S ? page_of(a.c, r.s, r.j) : -1;
  return true;
}

// Quotients are within 5e-6 of the real ones (five roundings of a number of at
// most 15); where one is nearer than that to a half, `nearer` decides.
template <int D, int E, int U>
__global__ void __launch_bounds__(kIoThreads, 4) append_kernel(const IoArgs a) {
  constexpr int LPR = D / E, RPW = 32 / LPR;
  pdl_wait();
  pdl_trigger();
  const int x = threadIdx.x % LPR;
  TokenRows r;
  if (!token_rows<U, LPR>(a, r)) return;
  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = r.first + u * RPW, part = row >= a.c.Hkv, h = row - part * a.c.Hkv;
    raw[u] = make_uint4(0, 0, 0, 0);
    if (h < a.c.Hkv)
      raw[u] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.x[part]) +
                                               (r.t * a.ts[part] + h * a.hs[part] + E * x) * (16 / E));
  }
  if (x == 0 && r.j != -1 && r.page < 0) flag_error(a.dev_err, MOE_DEV_BAD_ID);
  const int at = r.j & (a.c.page_size - 1);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = r.first + u * RPW, part = row >= a.c.Hkv, h = row - part * a.c.Hkv;
    float v[E], lo, hi;
    values_of<E>(raw[u], v);
    extremes<E, LPR>(raw[u], v, lo, hi);
    const bool ok = lo >= -65504.f && hi <= 65504.f;  // false for a NaN
    const __half scale = ok ? __float2half_rn(fifteenth(hi, lo)) : __float2half_rn(0.f);
    const __half zero = ok ? __float2half_rn(lo) : __ushort_as_half(0x7E00);
    const float sf = __half2float(scale), zf = __half2float(zero);
    // An fp16 above zero has a reciprocal of at most 2^24.  No scale (or no zero): all codes 0.
    const float inv = sf > 0.f ? rcp(sf) * (1.f / 15.f) : 0.f;
    float code[E], off = 0.f;
    const float2 fifteen = make_float2(15.f, 15.f), magic = make_float2(kMagic, kMagic);
#pragma unroll
    for (int d = 0; d < E; d += 2) {
      const float2 above = add2(make_float2(v[d], v[d + 1]), make_float2(-zf, -zf));
      const float2 q = make_float2(__saturatef(above.x * inv), __saturatef(above.y * inv));  // quotient / 15; NaN becomes 0
      const float2 k = add2(fma2(q, fifteen, magic), make_float2(-kMagic, -kMagic));
      const float2 e = fma2(q, fifteen, make_float2(-k.x, -k.y));
      code[d] = k.x;
      code[d + 1] = k.y;
      off = max3_abs(off, e.x, e.y);
    }
    if (off > 0.49999f) {
#pragma unroll
      for (int d = 0; d < E; ++d) {
        const float e = fmaf(__saturatef((v[d] - zf) * inv), 15.f, -code[d]);
        if (fabsf(e) > 0.49999f) code[d] = nearer(v[d], zf, sf, e > 0.f ? code[d] : code[d] - 1.f);
      }
    }
    if (h >= a.c.Hkv) continue;
    if (x == 0 && r.j >= 0 && !ok) flag_error(a.dev_err, MOE_DEV_BAD_KV);
    // Four codes side by side are a whole number below 2^16: they join as one, behind 2^23's exponent.
    uint32_t four[E / 4];
#pragma unroll
    for (int g = 0; g < E / 4; ++g)
      four[g] = __float_as_uint(fmaf(code[4 * g + 3], 4096.f, fmaf(code[4 * g + 2], 256.f, fmaf(code[4 * g + 1], 16.f, code[4 * g] + 8388608.f))));
    if (a.y[part]) {
      const float hs = r.page < 0 ? 0.f : sf, hz = r.page < 0 ? 0.f : zf;
      float held[E];
#pragma unroll
      for (int d = 0; d < E; d += 2) {
        const float2 y = fma2(make_float2(hs, hs), make_float2(code[d], code[d + 1]), make_float2(hz, hz));
        held[d] = y.x;
        held[d + 1] = y.y;
      }
      store_values<E>(a.y[part], (static_cast<long long>(r.t) * a.c.Hkv + h) * D + E * x, held);
    }
    if (r.page < 0) continue;
    uint8_t* b = page_block(a.c, r.page, h);
    uint8_t* cp = b + (part * a.c.page_size + at) * (D / 2) + (E / 2) * x;
    if constexpr (E == 8) *reinterpret_cast<uint32_t*>(cp) = __byte_perm(four[0], four[E / 4 - 1], 0x5410);
    else *reinterpret_cast<uint16_t*>(cp) = static_cast<uint16_t>(four[0]);
    if (x == 0) *reinterpret_cast<__half2*>(b + a.c.page_size * D + at * 8 + part * 4) = __halves2half2(scale, zero);
  }
}

template <int D, int E, int U>
__global__ void __launch_bounds__(kIoThreads) read_kernel(const IoArgs a) {
  constexpr int LPR = D / E, RPW = 32 / LPR;
  pdl_wait();
  pdl_trigger();
  const int x = threadIdx.x % LPR;
  TokenRows r;
  if (!token_rows<U, LPR>(a, r)) return;
  if (x == 0 && r.j != -1 && r.page < 0) flag_error(a.dev_err, MOE_DEV_BAD_ID);
  const int at = r.j & (a.c.page_size - 1);
  uint32_t codes[U];
  __half2 par[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = r.first + u * RPW, part = row >= a.c.Hkv, h = row - part * a.c.Hkv;
    codes[u] = 0;
    par[u] = __float2half2_rn(0.f);
    if (r.page >= 0 && h < a.c.Hkv) {
      const uint8_t* b = page_block(a.c, r.page, h);
      const uint8_t* cp = b + (part * a.c.page_size + at) * (D / 2) + (E / 2) * x;
      codes[u] = E == 8 ? *reinterpret_cast<const uint32_t*>(cp) : *reinterpret_cast<const uint16_t*>(cp);
      par[u] = *reinterpret_cast<const __half2*>(b + a.c.page_size * D + at * 8 + part * 4);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = r.first + u * RPW, part = row >= a.c.Hkv, h = row - part * a.c.Hkv;
    if (h >= a.c.Hkv) break;
    const float2 p = __half22float2(par[u]);
    float v[E];
#pragma unroll
    for (int d = 0; d < E; ++d) {
      // a nibble behind 2^23's exponent is that number plus the code
      const float c = __uint_as_float(((codes[u] >> (4 * d)) & 15u) | 0x4B000000u) - 8388608.f;
      v[d] = fmaf(p.x, c, p.y);
    }
    store_values<E>(a.y[part], (static_cast<long long>(r.t) * a.c.Hkv + h) * D + E * x, v);
  }
}

// Passes of a warp: four when that still leaves every SM its 32 warps, one
// otherwise (a small call's time is its code's length, from a cold cache).
template <bool Append, int D, int E>
int launch_rows(IoArgs a, cudaStream_t s) {
  constexpr int RPW = 32 / (D / E);
  const int passes = (2 * a.c.Hkv + RPW - 1) / RPW;
  const bool four = static_cast<long long>(a.T) * passes >= 4ll * 32 * sm_count();
  a.groups = four ? (passes + 3) / 4 : passes;
  const long long warps = static_cast<long long>(a.T) * a.groups;
  const dim3 grid(static_cast<unsigned>((warps + kIoThreads / 32 - 1) / (kIoThreads / 32)));
  void (*k)(IoArgs);
  if (Append) k = four ? append_kernel<D, E, 4> : append_kernel<D, E, 1>;
  else k = four ? read_kernel<D, E, 4> : read_kernel<D, E, 1>;
  LaunchScope ls(Append ? kProfKv4Append : kProfKv4Read, s);
  return launch_k(k, grid, dim3(kIoThreads), 0, s, false, a);
}

template <bool Append>
int launch_io(const IoArgs& a, bool f32, cudaStream_t s) {
  if (a.c.D == 128) return f32 ? launch_rows<Append, 128, 4>(a, s) : launch_rows<Append, 128, 8>(a, s);
  return f32 ? launch_rows<Append, 64, 4>(a, s) : launch_rows<Append, 64, 8>(a, s);
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
  if (!stride_ok(cfg->k_token_stride, cfg->T, per) || !stride_ok(cfg->v_token_stride, cfg->T, per) ||
      !stride_ok(cfg->k_head_stride, c.Hkv, per) || !stride_ok(cfg->v_head_stride, c.Hkv, per))
    return MOE_ERR_UNSUPPORTED;
  IoArgs a{c, {k, v}, {cfg->k_token_stride, cfg->v_token_stride}, {cfg->k_head_stride, cfg->v_head_stride},
           seq, slot, cfg->T, 0, {k_held, v_held}, dev_err};
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
  IoArgs a{c, {nullptr, nullptr}, {0, 0}, {0, 0}, seq, slot, cfg->T, 0, {k, v}, dev_err};
  return launch_io<false>(a, cfg->dtype == MOE_DTYPE_F32, static_cast<cudaStream_t>(stream));
}
