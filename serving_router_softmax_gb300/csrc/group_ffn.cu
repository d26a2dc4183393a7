// moe_group_gate_up, moe_group_down: the experts' products of a prompt's
// tokens, grouped by expert.
//
// First form: 64 x 64 tiles of a group's rows and a matrix's rows on the CUDA
// cores.
#include "common.cuh"

namespace moe {
namespace {

struct GroupArgs {
  const uint16_t* x;          // rows of K values
  const uint16_t* w;
  const int32_t *n_unique, *unique, *offsets, *perm, *slot_of;
  uint16_t* out;              // [rows][N]
  int32_t* dev_err;
  int T, rows, E, cap, n_slots, N, K, tiled;
};

// Weight rows of (slot, row) in either layout: `half` is 0 for a gate row, 1 for an up row.
template <bool kGateUp>
__device__ __forceinline__ const uint16_t* weight(const GroupArgs& a, int slot, int row, int half, int col) {
  if (!a.tiled) return a.w + (static_cast<size_t>(slot) * a.N * (kGateUp ? 2 : 1) + (half ? a.N : 0) + row) * a.K + col;
  const int MT = (a.N + 127) / 128, R = kGateUp ? 256 : 128;
  return a.w + (((static_cast<size_t>(slot) * MT + row / 128) * (a.K / 64) + col / 64) * R + half * 128 + row % 128) * 64 + col % 64;
}

template <bool kGateUp>
__global__ void __launch_bounds__(256) group_tile_kernel(const GroupArgs a) {
  __shared__ float xs[64][17], ws[2][64][17];
  const int U = *a.n_unique;
  if (U < 0 || U > a.cap) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) flag_error(a.dev_err, MOE_DEV_CAPACITY);
    return;
  }
  const int u = blockIdx.y, n0 = blockIdx.x * 64, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  if (u >= U) return;
  const int e = a.unique[u], p0 = a.offsets[u], p1 = a.offsets[u + 1];
  const bool ok = e >= 0 && e < a.E && p0 >= 0 && p0 <= p1 && p1 <= a.rows;
  const int slot = ok ? weight_slot(a.slot_of, a.n_slots, e) : -1;
  if (slot < 0) {
    if (threadIdx.x == 0) flag_error(a.dev_err, MOE_DEV_BAD_ID);
    return;
  }
  for (int p = p0; p < p1; p += 64) {
    float acc[2][4][4] = {};
    for (int k = 0; k < a.K; k += 16) {
      __syncthreads();
      for (int i = threadIdx.x; i < 1024; i += 256) {
        const int r = i / 16, c = i % 16, row = min(p + r, p1 - 1);
        int t = kGateUp ? a.perm[row] : row;
        if (kGateUp && (t < 0 || t >= a.T)) flag_error(a.dev_err, MOE_DEV_BAD_ID), t = 0;
        xs[r][c] = bf16_bits_to_float(a.x[static_cast<size_t>(t) * a.K + k + c]);
        for (int half = 0; half < (kGateUp ? 2 : 1); ++half)
          ws[half][r][c] = n0 + r < a.N ? bf16_bits_to_float(*weight<kGateUp>(a, slot, n0 + r, half, k + c)) : 0.f;
      }
      __syncthreads();
      for (int c = 0; c < 16; ++c)
        for (int half = 0; half < (kGateUp ? 2 : 1); ++half)
          for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) acc[half][i][j] += xs[ty + 16 * i][c] * ws[half][tx + 16 * j][c];
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int row = p + ty + 16 * i, n = n0 + tx + 16 * j;
        if (row >= p1 || n >= a.N) continue;
        float v = acc[0][i][j];
        if (kGateUp) v = v / (1.f + expf(-v)) * acc[1][i][j];
        a.out[static_cast<size_t>(row) * a.N + n] = v == v ? float_to_bf16_bits_rn(v) : 0x7FFF;
      }
  }
}

// y_t = sum_j w_tj o[inv_tj] in slot order, eight values a thread.
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
    for (int j = 0; j < k; ++j) {
      const long long p = inv[static_cast<long long>(t) * k + j];
      const float f = w[static_cast<long long>(t) * k + j];
      if (p < 0 || p >= static_cast<long long>(T) * k) {
        flag_error(dev_err, MOE_DEV_BAD_ID);
        continue;
      }
      const uint4 v = *reinterpret_cast<const uint4*>(o + p * H + c);
      const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
      for (int q = 0; q < 4; ++q) {
        acc[2 * q] += f * __uint_as_float(vw[q] << 16);
        acc[2 * q + 1] += f * __uint_as_float(vw[q] & 0xFFFF0000u);
      }
    }
  }
  for (int q = 0; q < 8; ++q) y[static_cast<size_t>(t) * H + c + q] = acc[q] == acc[q] ? float_to_bf16_bits_rn(acc[q]) : 0x7FFF;
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
  const GroupArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(lw->w_gate_up), n_unique, unique, offsets, perm_token,
                    slot_table(*lw), static_cast<uint16_t*>(h), dev_err, T, rows, lw->E, cap, weight_slots(*lw), lw->I, lw->H,
                    lw->layout == MOE_LAYOUT_TILED};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  LaunchScope ls(kProfGroupGateUp, s);
  group_tile_kernel<true><<<dim3((lw->I + 63) / 64, cap), 256, 0, s>>>(a);
  return check_launch();
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
  uint16_t* o = static_cast<uint16_t*>(workspace);
  const GroupArgs a{static_cast<const uint16_t*>(h), static_cast<const uint16_t*>(lw->w_down), n_unique, unique, offsets, nullptr,
                    slot_table(*lw), o, dev_err, T, rows, lw->E, cap, weight_slots(*lw), lw->H, lw->I, lw->layout == MOE_LAYOUT_TILED};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  {
    LaunchScope ls(kProfGroupDown, s);
    group_tile_kernel<false><<<dim3((lw->H + 63) / 64, cap), 256, 0, s>>>(a);
    const int e = check_launch();
    if (e != MOE_OK) return e;
  }
  LaunchScope ls(kProfGroupDown, s);
  const long long n = static_cast<long long>(T) * (lw->H / 8);
  group_sum_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(o, inv, w, n_unique, static_cast<uint16_t*>(y), T, k, lw->H, cap,
                                                                       dev_err);
  return check_launch();
}
