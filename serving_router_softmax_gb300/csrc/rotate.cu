// moe_rotate: rotary positions of queries and keys, one or several axes.
//
// A pair's angle is pos * f.  As a part of a full turn held in 64 bits,
// pos * turns[i] mod 2^64 is exact integer arithmetic for any position: the
// turns that a far position has made fall out at the top.  What is left is an
// angle within half a turn either way, known to 2^-34 of a turn before it is
// rounded to fp32, so cosine and sine are as good at position 2^31 as at 0.
//
// Bound by memory: every value is read and written once (8192 tokens of 40 heads
// of 128 in bf16: 29 us, 5.8 TB/s).  A block takes a few tokens, as many as give each
// of its threads one cosine and sine to make, and these go to shared memory for all
// of the tokens' heads (each thread making its own for up to 8 heads: 40 us).  A
// thread keeps its 16 bytes' place in a row and steps through rows, two units' loads
// (halves; four where a unit is one load) asked for before the first is used, the
// first of them before the cosines; 48 registers a thread leave five blocks an SM
// (twice as many loads in 97 registers: 40 us; an item's place worked out by division:
// 32 us, and 30 instead of 19 for 3001 tokens of 72 fp32 heads).  With few tokens the
// heads are split over blocks.
#include <cuda_bf16.h>

#include <algorithm>

#include "apart.cuh"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;
constexpr int kMaxAngles = 512;

struct RotateArgs {
  const uint8_t *q, *k;
  uint8_t *oq, *ok;
  const int32_t *pos, *axis;
  const uint64_t* turns;
  int32_t* dev_err;
  long long q_ts, q_hs, k_ts, k_hs, oq_ts, oq_hs, ok_ts, ok_hs;  // bytes
  int T, Hq, H, D, R, n_axes, inverse;
  int units, turning;   // units of a row that is read; those that turn come first
  int lanes_log2;       // threads a row: the units, rounded up to a power of two
  int tokens, heads;    // of a block
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

// Cosine and sine (of minus the angle: `inverse`) of position pos and pair i.
__device__ __forceinline__ float2 turn_of(const RotateArgs& a, long long t, int i, bool report) {
  const int ax = a.axis[i];
  if (ax < 0 || ax >= a.n_axes) {
    if (report) flag_error(a.dev_err, MOE_DEV_BAD_ID);
    return make_float2(1.f, 0.f);
  }
  const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(a.pos[static_cast<long long>(ax) * a.T + t])) * a.turns[i];
  // The nearest quarter turn and what is left of it, at most an eighth either way.
  const int quarter = static_cast<int>((turn + (1ull << 61)) >> 62);
  const int64_t left = static_cast<int64_t>(turn - (static_cast<uint64_t>(quarter) << 62));
  float sn, cs;
  sincospif(static_cast<float>(static_cast<int32_t>(left >> 30)) * 0x1p-33f, &sn, &cs);
  const float x = (quarter & 1) ? -sn : cs, y = (quarter & 1) ? cs : sn;
  return make_float2((quarter & 2) ? -x : x, ((quarter & 2) != 0) != (a.inverse != 0) ? -y : y);
}

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 5) rotate_kernel(const RotateArgs a) {
  constexpr int V = Row<T>::V, kAt = kInterleaved ? 2 * kAhead : kAhead, kPairs = kInterleaved ? V / 2 : V;  // pairs of a unit
  // A unit's first four and last four (of 8) lie apart, so that neighbouring units' 16 bytes lie side by side.
  __shared__ alignas(16) float cs[kMaxAngles], sn[kMaxAngles];
  auto slot = [](int i) { return kPairs == 8 ? ((i >> 2) & 1) * (kMaxAngles / 2) + (i >> 3) * 4 + (i & 3) : i; };
  const int half = a.R / 2, h0 = blockIdx.y * a.heads, heads = min(a.heads, a.H - h0);
  const long long t0 = static_cast<long long>(blockIdx.x) * a.tokens;
  const int tokens = static_cast<int>(min(static_cast<long long>(a.tokens), a.T - t0)), rows = tokens * heads;
  // A thread has one unit of every step-th row (a head of a token); its place in them stays.
  const int unit = threadIdx.x & ((1 << a.lanes_log2) - 1), step = kThreads >> a.lanes_log2;
  const bool turns = unit < a.turning, idle = unit >= a.units;
  const int first = turns ? unit * 16 : a.R * static_cast<int>(sizeof(T)) + (unit - a.turning) * 16;
  const int second = first + half * static_cast<int>(sizeof(T));
  const int step_tok = step / heads, step_h = step % heads;
  int row = threadIdx.x >> a.lanes_log2, tok = row / heads, h = row - tok * heads;
  bool ready = false;
  while (row < rows || !ready) {
    uint4 u[kAt], w[kInterleaved ? 1 : kAt];
    uint8_t* out[kAt];
    int angle[kAt];
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      out[j] = nullptr;
      if (row < rows && !idle) {
        const long long t = t0 + tok;
        const int head = h0 + h;
        const uint8_t* in = (head < a.Hq ? a.q + t * a.q_ts + head * a.q_hs : a.k + t * a.k_ts + (head - a.Hq) * a.k_hs) + first;
        out[j] = (head < a.Hq ? a.oq + t * a.oq_ts + head * a.oq_hs : a.ok + t * a.ok_ts + (head - a.Hq) * a.ok_hs) + first;
        angle[j] = tok * half + unit * kPairs;
        u[j] = *reinterpret_cast<const uint4*>(in);
        if (!kInterleaved && turns) w[j] = *reinterpret_cast<const uint4*>(in + (second - first));
      }
      row += step, tok += step_tok, h += step_h;
      if (h >= heads) h -= heads, ++tok;
    }
    if (!ready) {
      for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const float2 c = turn_of(a, t0 + i / half, i % half, blockIdx.x == 0 && blockIdx.y == 0);
        cs[slot(i)] = c.x, sn[slot(i)] = c.y;
      }
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      if (!out[j]) continue;
      if (turns) {
        float x[V], c[kPairs], s[kPairs];
        Row<T>::get(u[j], x);
        if (kPairs == 2) {
          *reinterpret_cast<float2*>(c) = *reinterpret_cast<const float2*>(cs + angle[j]);
          *reinterpret_cast<float2*>(s) = *reinterpret_cast<const float2*>(sn + angle[j]);
        } else {
#pragma unroll
          for (int i = 0; i < kPairs; i += 4) {
            *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + slot(angle[j] + i));
            *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(sn + slot(angle[j] + i));
          }
        }
        if (kInterleaved) {  // pairs side by side
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const float a0 = x[i], b0 = x[i + 1];
            x[i] = a0 * c[i / 2] - b0 * s[i / 2], x[i + 1] = a0 * s[i / 2] + b0 * c[i / 2];
          }
        } else {
          float y[V];
          Row<T>::get(w[j], y);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float a0 = x[i], b0 = y[i];
            x[i] = a0 * c[i] - b0 * s[i], y[i] = a0 * s[i] + b0 * c[i];
          }
          *reinterpret_cast<uint4*>(out[j] + (second - first)) = Row<T>::put(y);
        }
        u[j] = Row<T>::put(x);
      }
      *reinterpret_cast<uint4*>(out[j]) = u[j];
    }
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
int launch(const moe_rotate_cfg& c, RotateArgs a, bool copies, cudaStream_t s) {
  constexpr int V = Row<T>::V;
  a.turning = a.R / (c.interleaved ? V : 2 * V);
  a.units = a.turning + (copies ? (a.D - a.R) / V : 0);
  a.lanes_log2 = 0;
  while ((1 << a.lanes_log2) < a.units) ++a.lanes_log2;
  a.tokens = std::max(1, kMaxAngles / a.R);  // a cosine and a sine a thread
  const long long across = (a.T + a.tokens - 1) / a.tokens;
  // Twice what the SMs hold, but an item a thread at least where the heads are split.
  const long long want = 10ll * sm_count();
  const int most = std::max(1, a.tokens * a.H * a.units / kThreads);
  const int split = static_cast<int>(std::min<long long>(most, std::max(1ll, want / across)));
  a.heads = (a.H + split - 1) / split;
  const dim3 blocks(static_cast<unsigned>(across), (a.H + a.heads - 1) / a.heads);
  LaunchScope ls(kProfRotate, s);
  if (c.interleaved)
    rotate_kernel<T, true><<<blocks, kThreads, 0, s>>>(a);
  else
    rotate_kernel<T, false><<<blocks, kThreads, 0, s>>>(a);
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
  const uintptr_t at = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out_q) |
                         (c.n_k_heads ? reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(out_k) : 0);
  if (at & 15 || (reinterpret_cast<uintptr_t>(pos) | reinterpret_cast<uintptr_t>(axis) | reinterpret_cast<uintptr_t>(dev_err)) & 3 ||
      reinterpret_cast<uintptr_t>(turns) & 7)
    return MOE_ERR_ARG;
  // In place: row on row.
  auto astray = [&](const void* in, const void* out, long long it, long long ot, int H, long long ih, long long oh) {
    return in == out && ((c.T > 1 && it != ot) || (H > 1 && ih != oh));
  };
  if (astray(q, out_q, c.q_token_stride, c.oq_token_stride, c.n_q_heads, c.q_head_stride, c.oq_head_stride) ||
      (c.n_k_heads && astray(k, out_k, c.k_token_stride, c.ok_token_stride, c.n_k_heads, c.k_head_stride, c.ok_head_stride)))
    return MOE_ERR_ARG;
  auto rows = [&](const void* p, int H, long long ts, long long hs) {
    return Rows{reinterpret_cast<uintptr_t>(p), c.T, ts * size, H, hs * size, D * size};
  };
  const Rows rq = rows(q, c.n_q_heads, c.q_token_stride, c.q_head_stride), rk = rows(k, c.n_k_heads, c.k_token_stride, c.k_head_stride);
  const Rows roq = rows(out_q, c.n_q_heads, c.oq_token_stride, c.oq_head_stride), rok = rows(out_k, c.n_k_heads, c.ok_token_stride, c.ok_head_stride);
  if ((q != out_q && !rows_apart(rq, roq)) || (k != out_k && !rows_apart(rk, rok)) || !rows_apart(rq, rok) || !rows_apart(rk, roq) ||
      !rows_apart(roq, rok))
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
  const bool copies = q != out_q || (c.n_k_heads && k != out_k);  // dimensions past R
  return c.dtype == MOE_DTYPE_F32 ? launch<float>(c, a, copies, static_cast<cudaStream_t>(stream))
                                  : launch<__nv_bfloat16>(c, a, copies, static_cast<cudaStream_t>(stream));
}
