// moe_rotate: rotary positions of queries and keys, one or several axes.
//
// A pair's angle is pos * f.  As a part of a full turn held in 64 bits,
// pos * turns[i] mod 2^64 is exact integer arithmetic for any position: the
// turns that a far position has made fall out at the top.  What is left is an
// angle within half a turn either way, known to 2^-34 of a turn before it is
// rounded to fp32, so cosine and sine are as good at position 2^31 as at 0.
//
// Bound by memory: every value is read and written once.  A thread keeps the
// cosines and sines of one unit of pairs (16 bytes of first and 16 of second
// halves) of one token in registers and walks the token's heads with them, in
// 16-byte loads and stores.  How many heads it walks is a rule on the work:
// as many as leave the device full, since a walk saves the angles and a thread
// more hides latency.
#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxWalk = 8;

struct RotateArgs {
  const uint8_t *q, *k;
  uint8_t *oq, *ok;
  const int32_t *pos, *axis;
  const uint64_t* turns;
  int32_t* dev_err;
  long long q_ts, q_hs, k_ts, k_hs, oq_ts, oq_hs, ok_ts, ok_hs;  // bytes
  int T, Hq, H, D, R, n_axes, inverse;
  int units, turning;   // units of a row; those that turn come first
  int walk, groups;     // heads of a thread, threads a token and unit
  int copies;           // dimensions past R are copied
};

// V values of 16 bytes as floats and back.
template <typename T>
struct Row;
template <>
struct Row<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void get(uint4 u, float (&v)[V]) {
    v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y), v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&v)[V]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct Row<__nv_bfloat16> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void get(uint4 u, float (&v)[V]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  static __device__ __forceinline__ uint4 put(const float (&v)[V]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const RotateArgs a) {
  constexpr int V = Row<T>::V;
  const long long id = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x;
  const int unit = static_cast<int>(id % a.units);
  const long long rest = id / a.units;
  const int g = static_cast<int>(rest % a.groups);
  const long long t = rest / a.groups;
  if (t >= a.T) return;
  const bool turns = unit < a.turning;
  if (!turns && !a.copies) return;
  // Bytes of the unit's two 16-byte parts in a row (one part where it copies).
  const int first = turns ? (kInterleaved ? unit * 32 : unit * 16) : a.R * static_cast<int>(sizeof(T)) + (unit - a.turning) * 16;
  const int second = kInterleaved ? first + 16 : first + a.R / 2 * static_cast<int>(sizeof(T));
  const int h0 = g * a.walk, h1 = min(a.H, h0 + a.walk);
  float c[V], s[V];
  if (turns) {
    int last = -1;
    uint64_t pos = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int ax = a.axis[unit * V + i];
      const bool ok = ax >= 0 && ax < a.n_axes;
      if (!ok && g == 0 && t == 0) flag_error(a.dev_err, MOE_DEV_BAD_ID);
      if (ok && ax != last) pos = static_cast<uint64_t>(static_cast<int64_t>(a.pos[static_cast<long long>(ax) * a.T + t])), last = ax;
      const uint64_t turn = ok ? pos * a.turns[unit * V + i] : 0;
      // The nearest quarter turn and what is left of it, at most an eighth either way.
      const uint64_t near = turn + (1ull << 61);
      const int quarter = static_cast<int>(near >> 62);
      const int64_t left = static_cast<int64_t>(turn - (static_cast<uint64_t>(quarter) << 62));
      float sn, cs;
      sincospif(static_cast<float>(left) * 0x1p-63f, &sn, &cs);
      const float x = (quarter & 1) ? -sn : cs, y = (quarter & 1) ? cs : sn;
      c[i] = (quarter & 2) ? -x : x;
      s[i] = ((quarter & 2) != 0) != (a.inverse != 0) ? -y : y;
    }
  }
  for (int h = h0; h < h1; ++h) {
    const bool isq = h < a.Hq;
    const uint8_t* in = isq ? a.q + t * a.q_ts + h * a.q_hs : a.k + t * a.k_ts + (h - a.Hq) * a.k_hs;
    uint8_t* out = isq ? a.oq + t * a.oq_ts + h * a.oq_hs : a.ok + t * a.ok_ts + (h - a.Hq) * a.ok_hs;
    uint4 u = *reinterpret_cast<const uint4*>(in + first);
    if (turns) {
      uint4 w = *reinterpret_cast<const uint4*>(in + second);
      float x[V], y[V];
      Row<T>::get(u, x);
      Row<T>::get(w, y);
      if (kInterleaved) {  // pairs side by side: the first part holds the unit's first V / 2 pairs
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float a0 = x[i], b0 = x[i + 1], a1 = y[i], b1 = y[i + 1];
          x[i] = a0 * c[i / 2] - b0 * s[i / 2], x[i + 1] = a0 * s[i / 2] + b0 * c[i / 2];
          y[i] = a1 * c[V / 2 + i / 2] - b1 * s[V / 2 + i / 2], y[i + 1] = a1 * s[V / 2 + i / 2] + b1 * c[V / 2 + i / 2];
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float a0 = x[i], b0 = y[i];
          x[i] = a0 * c[i] - b0 * s[i], y[i] = a0 * s[i] + b0 * c[i];
        }
      }
      u = Row<T>::put(x);
      *reinterpret_cast<uint4*>(out + second) = Row<T>::put(y);
    }
    *reinterpret_cast<uint4*>(out + first) = u;
  }
}

// A stride of n tokens or heads.
bool stride_ok(long long st, int n, int per16) { return n <= 1 || (st >= 0 && st % per16 == 0 && st < (1ll << 40)); }
// No two of an output's rows share a value: one stride steps over a row, the other over all rows of the first.
bool apart(long long ts, int T, long long hs, int H, long long D) {
  if (T <= 1 && H <= 1) return true;
  if (T <= 1) return hs >= D;
  if (H <= 1) return ts >= D;
  return (hs >= D && ts >= hs * (H - 1) + D) || (ts >= D && hs >= ts * (T - 1) + D);
}

template <typename T>
int launch(const moe_rotate_cfg& c, RotateArgs a, cudaStream_t s) {
  constexpr int V = Row<T>::V;
  a.turning = a.R / (2 * V);
  a.units = a.turning + (a.D - a.R) / V;
  const long long threads = static_cast<long long>(a.T) * a.units * a.H, full = sm_count() * 2048ll;
  a.walk = static_cast<int>(threads / full);
  a.walk = a.walk < 1 ? 1 : a.walk > kMaxWalk ? kMaxWalk : a.walk;
  a.groups = (a.H + a.walk - 1) / a.walk;
  const long long blocks = (static_cast<long long>(a.T) * a.units * a.groups + kThreads - 1) / kThreads;
  if (blocks > 0x7FFFFFFFll) return MOE_ERR_UNSUPPORTED;
  LaunchScope ls(kProfRotate, s);
  if (c.interleaved)
    rotate_kernel<T, true><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
  else
    rotate_kernel<T, false><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
  return check_launch();
}

}  // namespace
}  // namespace moe

extern "C" int moe_rotate(const void* q, const void* k, const int32_t* pos, const uint64_t* turns, const int32_t* axis,
                          const moe_rotate_cfg* cfg, void* out_q, void* out_k, int32_t* dev_err, void* stream) {
  using namespace moe;
  if (!cfg) return MOE_ERR_ARG;
  const moe_rotate_cfg& c = *cfg;
  if (c.T < 0 || c.n_q_heads < 1 || c.n_k_heads < 0 || c.n_axes < 1) return MOE_ERR_ARG;
  if ((c.interleaved | c.inverse) & ~1) return MOE_ERR_ARG;
  if (c.dtype != MOE_DTYPE_BF16 && c.dtype != MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
  if (c.T > (1 << 24) || c.n_q_heads > 4096 || c.n_k_heads > 4096 - c.n_q_heads || c.n_axes > 4) return MOE_ERR_UNSUPPORTED;
  if (c.head_dim < 16 || c.head_dim > 512 || c.head_dim % 8 || c.rotary_dim < 16 || c.rotary_dim > c.head_dim || c.rotary_dim % 16)
    return MOE_ERR_UNSUPPORTED;
  const int size = c.dtype == MOE_DTYPE_F32 ? 4 : 2, per16 = 16 / size;
  const long long D = c.head_dim;
  const int Tk = c.n_k_heads ? c.T : 0;
  if (!stride_ok(c.q_token_stride, c.T, per16) || !stride_ok(c.q_head_stride, c.n_q_heads, per16) ||
      !stride_ok(c.k_token_stride, Tk, per16) || !stride_ok(c.k_head_stride, c.n_k_heads, per16) ||
      !stride_ok(c.oq_token_stride, c.T, per16) || !stride_ok(c.oq_head_stride, c.n_q_heads, per16) ||
      !stride_ok(c.ok_token_stride, Tk, per16) || !stride_ok(c.ok_head_stride, c.n_k_heads, per16) ||
      !apart(c.oq_token_stride, c.T, c.oq_head_stride, c.n_q_heads, D) ||
      (c.n_k_heads && !apart(c.ok_token_stride, c.T, c.ok_head_stride, c.n_k_heads, D)))
    return MOE_ERR_UNSUPPORTED;
  if (c.T == 0) return MOE_OK;
  if (!q || !out_q || !pos || !turns || !axis || (c.n_k_heads && (!k || !out_k))) return MOE_ERR_ARG;
  const uintptr_t rows = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out_q) |
                         (c.n_k_heads ? reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(out_k) : 0);
  if (rows & 15 || (reinterpret_cast<uintptr_t>(pos) | reinterpret_cast<uintptr_t>(axis) | reinterpret_cast<uintptr_t>(dev_err)) & 3 ||
      reinterpret_cast<uintptr_t>(turns) & 7)
    return MOE_ERR_ARG;
  RotateArgs a = {};
  a.q = static_cast<const uint8_t*>(q), a.k = static_cast<const uint8_t*>(k);
  a.oq = static_cast<uint8_t*>(out_q), a.ok = static_cast<uint8_t*>(out_k);
  a.pos = pos, a.axis = axis, a.turns = turns, a.dev_err = dev_err;
  auto bytes = [&](long long st, int n) { return n <= 1 ? 0 : st * size; };
  a.q_ts = bytes(c.q_token_stride, c.T), a.q_hs = bytes(c.q_head_stride, c.n_q_heads);
  a.k_ts = bytes(c.k_token_stride, c.T), a.k_hs = bytes(c.k_head_stride, c.n_k_heads);
  a.oq_ts = bytes(c.oq_token_stride, c.T), a.oq_hs = bytes(c.oq_head_stride, c.n_q_heads);
  a.ok_ts = bytes(c.ok_token_stride, c.T), a.ok_hs = bytes(c.ok_head_stride, c.n_k_heads);
  a.T = c.T, a.Hq = c.n_q_heads, a.H = c.n_q_heads + c.n_k_heads, a.D = c.head_dim, a.R = c.rotary_dim;
  a.n_axes = c.n_axes, a.inverse = c.inverse;
  a.copies = a.R < a.D && (q != out_q || (c.n_k_heads && k != out_k));
  return c.dtype == MOE_DTYPE_F32 ? launch<float>(c, a, static_cast<cudaStream_t>(stream))
                                  : launch<__nv_bfloat16>(c, a, static_cast<cudaStream_t>(stream));
}
