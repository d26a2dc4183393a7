// 4-bit paged KV cache: layout and device helpers shared by the kv4_* kernels.
//
// A value is zero + scale * code, code in 0..15, with one (scale, zero) pair
// of fp16 per slot, kv head and K or V.  Page p, head h is one block of
// page_size * (D + 8) bytes: K codes [page_size][D/2], V codes
// [page_size][D/2], parameters [page_size][4] (k scale, k zero, v scale, v
// zero).  Byte b of a code row holds dimension 2b in its low nibble.
//
// Attention on the tensor cores works on the bare codes.  A nibble masked
// out of a 32-bit word IS an fp16 number: bits 0-3 of a half are code *
// 2^-24, bits 4-7 are code * 2^-20 (both subnormal or the smallest normals,
// exact), so a pair of codes costs one AND and no conversion; the factors of
// 16 go into the other operand or the accumulator's final scale, the (scale,
// zero) pairs into the softmax:
//   S_ij = scale * (ks_j * (q_i . c_j) + kz_j * sum(q_i))
//   O_i  = sum_j p_ij * vs_j * (c_j + vz_j / vs_j)
// The probabilities go into the second product as p_ij * vs_j, with the
// running maximum taken over S_ij + log2(vs_j): the product's fp16 operand
// is then at most 2^8 whatever the scales are.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "smem_limit.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace kv4 {

constexpr int kTile = 64;          // slots of one pipeline stage
constexpr int kMaxSeq = 4096;
constexpr int kMaxTree = 64;       // new tokens per sequence that a visibility mask can tell apart
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -3.0e38f;  // running maximum of a row that has seen nothing
// The smallest fp16 above zero: stands in for the zero scale of an entry
// whose D values are equal (all its codes are 0, so its value stays `zero`).
constexpr float kMinScale = 5.9604644775390625e-8f;

struct Cache {
  uint8_t* pages;
  const int32_t* table;
  int32_t n_pages, page_size, page_log2, Hkv, D, S, width;
  __host__ __device__ size_t block_bytes() const { return static_cast<size_t>(page_size) * (D + 8); }
};

// Launches `clusters` clusters of `size` CTAs.
template <typename... KArgs, typename... Args>
int launch_clusters(void (*kernel)(KArgs...), int clusters, int size, int threads, size_t smem, cudaStream_t s,
                    Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters) * size);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int cache_validate(const kv4_cache* c, Cache* out);

// A stride over n tokens or heads (of one: never used, so anything goes).
inline bool stride_ok(long long stride, int n, int multiple) { return n <= 1 || (stride >= 0 && stride % multiple == 0); }

// Block of (page id, head).
__device__ __forceinline__ uint8_t* page_block(const Cache& c, int page, int h) {
  return c.pages + (static_cast<size_t>(page) * c.Hkv + h) * c.block_bytes();
}

// Page id of slot j of sequence s, -1 if the slot or the table's entry is out of range.
__device__ __forceinline__ int page_of(const Cache& c, int s, int j) {
  const int k = j >> c.page_log2;
  if (j < 0 || k >= c.width) return -1;
  const int p = c.table[static_cast<size_t>(s) * c.width + k];
  return p >= 0 && p < c.n_pages ? p : -1;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Waits for a phase of an mbarrier.  Gives up, and sets *abort, when 2 s (or `budget_ns`) have passed or another role
// has set *abort.  A try sleeps in hardware for up to 1 us, so that waiting warps leave the issue slots to the
// others, and the clock is read only after many tries, as reading it would lengthen every wait.
// kWarp: all lanes wait, with one answer.
template <bool kWarp>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort,
                                           uint64_t budget_ns = 2000000000ull) {
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity), "r"(1000u)
        : "memory");
    if (kWarp ? __all_sync(0xFFFFFFFFu, ok) : ok) return true;
    if ((n & 31) == 0) {
      const uint64_t now = tc::globaltimer_ns();
      if (t0 == 0) t0 = now;
      const bool stop = *abort || now - t0 > budget_ns;
      if (kWarp ? __any_sync(0xFFFFFFFFu, stop) : stop) {
        *abort = 1;
        return false;
      }
    }
  }
}

__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   tc::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}

// Query rows in the B-operand layout of mma.m16n8k16 (columns = rows of q).
// Key words are split by masks, so the product's k index follows the nibbles:
// lane c of a quad owns the D/4 dimensions from c * D/4 on; word w of them
// (dimensions 8w..8w+7, n = nibble) gives k-step 2w with the pairs (0, 4) and
// (1, 5)/16 and k-step 2w + 1 with (2, 6) and (3, 7)/16.  Each row is scaled
// by the power of two that puts its largest magnitude in [2^14, 2^15), so the
// fp16 copy of a bf16 row is exact down to 2^-27 of that magnitude.
//   frag  [n_rows / 8][D / 32][32] uint4: k-steps 2w (x, y) and 2w + 1 (z, w)
//   cq    factor of the accumulator, cqs factor of kz (both times scale * log2 e)
// `row` gives the source row (NULL: zeros).  Threads 0..nthreads-1 take part.
template <int D, typename RowPtr>
__device__ __forceinline__ void prep_q(RowPtr row, int n_rows, float scale_log2, uint4* frag, float* cq, float* cqs,
                                       int tid, int nthreads) {
  constexpr int LPR = D / 8;   // lanes of a row, 8 dimensions each
  constexpr int WPC = D / 32;  // words of a lane's chunk
  const int x = tid % LPR;
  for (int r = tid / LPR; r < n_rows; r += nthreads / LPR) {
    const uint16_t* p = row(r);
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (p) raw = *reinterpret_cast<const uint4*>(p + 8 * x);
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
    float m = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m = fmaxf(m, fabsf(v[i]));
      sum += v[i];
    }
    const uint32_t mask = LPR == 32 ? 0xFFFFFFFFu : ((1u << LPR) - 1u) << ((threadIdx.x & 31) / LPR * LPR);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(mask, m, o));
      sum += __shfl_xor_sync(mask, sum, o);
    }
    const int ex = static_cast<int>(__float_as_uint(m) >> 23);
    const int e = m > 0.f && ex < 255 ? 14 + 127 - (ex > 0 ? ex : 1) : 0;
    // 2^e in two factors: e may pass the exponent range of one fp32.
    const float f1 = __uint_as_float(static_cast<uint32_t>(127 + e / 2) << 23);
    const float f2 = __uint_as_float(static_cast<uint32_t>(127 + e - e / 2) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * f1 * f2;
    const int c = x / WPC, w = x % WPC;
    frag[((r >> 3) * (D / 32) + w) * 32 + (r & 7) * 4 + c] =
        make_uint4(pack_h2(v[0], v[4]), pack_h2(v[1] * 0.0625f, v[5] * 0.0625f), pack_h2(v[2], v[6]),
                   pack_h2(v[3] * 0.0625f, v[7] * 0.0625f));
    if (x == 0) {
      cq[r] = ldexpf(scale_log2, 24 - e);  // the codes carry 2^-24
      cqs[r] = scale_log2 * sum;
    }
  }
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Row of a 16-slot group that matrix row (or k index) i stands for: even ones
// the first four, odd ones the next four, so that the lanes of one shared
// memory access fall on rows of both parities (64-byte rows: no conflict for
// keys, two-way for values).
__device__ __forceinline__ int slot_of_row(int i) {
  const int c = (i >> 1) & 3;
  return (i & 8) + ((i & 1) ? 4 + (c ^ 1) : c);
}

// Nibble n (0..3) of both halves as a pair of fp16 numbers: codes * 2^-24
// (n even) or * 2^-20 (n odd).
template <int n>
__device__ __forceinline__ uint32_t nibbles(uint32_t w) {
  return (n < 2 ? w : w >> 8) & ((n & 1) ? 0x00F000F0u : 0x000F000Fu);
}

// Scores' accumulator of 16 slots against 8 query rows: acc[0..1] = slot of
// matrix row lane / 4, query columns 2 (lane % 4) and + 1; acc[2..3] = row + 8.
// ka / kb: the lane's code words of those two slots; frag: the 8 rows' (prep_q).
template <int D>
__device__ __forceinline__ void qk_16x8(float (&acc)[4], const uint32_t (&ka)[D / 32], const uint32_t (&kb)[D / 32],
                                        const uint4* frag) {
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    const uint4 q = frag[32 * w + (threadIdx.x & 31)];
    mma_f16(acc, nibbles<0>(ka[w]), nibbles<0>(kb[w]), nibbles<1>(ka[w]), nibbles<1>(kb[w]), make_uint2(q.x, q.y));
    mma_f16(acc, nibbles<2>(ka[w]), nibbles<2>(kb[w]), nibbles<3>(ka[w]), nibbles<3>(kb[w]), make_uint2(q.z, q.w));
  }
}

// A code row's words of lane c of a quad.
template <int D>
__device__ __forceinline__ void load_k_words(const uint8_t* row, int c, uint32_t (&w)[D / 32]) {
  if constexpr (D == 128) {
    const uint4 t = *reinterpret_cast<const uint4*>(row + 16 * c);
    w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
  } else {
    const uint2 t = *reinterpret_cast<const uint2*>(row + 8 * c);
    w[0] = t.x, w[1] = t.y;
  }
}

}  // namespace kv4
}  // namespace moe
