// What stands around the 8-bit projections: the quantiser and the residual norm.  Both read and
// write every element once.
//
// tp_quantize_fp8: a thread holds 16 consecutive elements (two 16-byte loads, one 16-byte store
// of codes).  By token (1 x 128): 8 lanes share a group and join their maxima by three shuffles.
// By weight block (128 x 128): a CTA of 256 threads holds the block in registers, four rows'
// chunks a thread, so the block is read once although its scale needs all of it.  Both are bound by
// HBM: 4608 x 18432 by token 37.5 us (6.8 TB/s, the measured copy rate), 9216 x 6144 by block 25.4 us
// (6.7 TB/s).
//
// tp_residual_norm: one row is held in registers as fp32 by one warp (short rows) or one CTA; the
// statistics are sums over those registers (the variance about the mean, in a second sum), and
// the normed, modulated row leaves as bf16 or as codes with their scales.  4608 x 6144 with two
// norms, gate and modulation, to fp8: 40.6 us (4.9 TB/s); h alone after an RMS norm 25.9 us (25.0 at the
// copy rate); without a branch, RMS to fp8, 24.6 us (12.5).  Neither HBM (44 % of its peak) nor the issue
// slots (65 %, some 130 instructions a thread for each 8 elements) are full in the first: a row is a
// chain of loads and up to three sums, each with a barrier, and with 64 registers a thread an SM
// holds four rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "tp_e4m3.cuh"
#include "tp_internal.h"

namespace tp {
namespace {

// ---------------------------------------------------------------------------
// Quantiser
// ---------------------------------------------------------------------------

struct QuantParams {
  const uint8_t* x;  // bf16 [rows, cols], row stride ldx bytes
  uint8_t* q;        // e4m3 [rows, cols], row stride ldq
  uint8_t* scales;   // e8m0, row stride lds
  int64_t ldx, ldq, lds;
  int64_t rows;
  int cols;
  int col_groups;    // ceil(cols / 128)
};

// The largest |x| of 16 bf16 elements, as bf16 bits (integer maximum: a NaN wins).
__device__ __forceinline__ uint32_t amax16(const uint4& a, const uint4& b) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t v = __vmaxu2(__vmaxu2(__vmaxu2(a.x & m, a.y & m), __vmaxu2(a.z & m, a.w & m)),
                              __vmaxu2(__vmaxu2(b.x & m, b.y & m), __vmaxu2(b.z & m, b.w & m)));
  return max(v & 0xFFFFu, v >> 16);
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ uint4 codes16(const uint4& a, const uint4& b, float inv) {
  auto four = [&](uint32_t u, uint32_t v) {
    return e4m3x4(bf16_lo(u) * inv, bf16_hi(u) * inv, bf16_lo(v) * inv, bf16_hi(v) * inv);
  };
  return make_uint4(four(a.x, a.y), four(a.z, a.w), four(b.x, b.y), four(b.z, b.w));
}

constexpr int kQuantThreads = 256;

__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(const QuantParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t group = static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 8) + (threadIdx.x >> 3);
  const int64_t row = group / p.col_groups;
  const int kg = static_cast<int>(group - row * p.col_groups);
  const int col = kg * kFp8Group + static_cast<int>(threadIdx.x & 7) * 16;
  const bool on = row < p.rows && col < p.cols;  // cols is a multiple of 16: a chunk is whole or absent
  uint4 a = make_uint4(0, 0, 0, 0), b = a;
  if (on) {
    const uint4* src = reinterpret_cast<const uint4*>(p.x + row * p.ldx + static_cast<int64_t>(col) * 2);
    a = src[0];
    b = src[1];
  }
  uint32_t m = amax16(a, b);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const uint32_t byte = e8m0_of_amax(m << 16);
  if (!on) return;
  *reinterpret_cast<uint4*>(p.q + row * p.ldq + col) = codes16(a, b, e8m0_inverse(byte));
  if ((threadIdx.x & 7) == 0) p.scales[row * p.lds + kg] = static_cast<uint8_t>(byte);
}

__global__ void __launch_bounds__(kQuantThreads) quantize_blocks_kernel(const QuantParams p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ uint32_t warp_max[kQuantThreads / 32];
  const int64_t rg = blockIdx.x / p.col_groups;
  const int kg = static_cast<int>(blockIdx.x - rg * p.col_groups);
  const int col = kg * kFp8Group + static_cast<int>(threadIdx.x & 7) * 16;
  const int64_t row0 = rg * kFp8Group + (threadIdx.x >> 3);
  uint4 a[4], b[4];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + 32 * i;
    a[i] = b[i] = make_uint4(0, 0, 0, 0);
    if (row < p.rows && col < p.cols) {
      const uint4* src = reinterpret_cast<const uint4*>(p.x + row * p.ldx + static_cast<int64_t>(col) * 2);
      a[i] = src[0];
      b[i] = src[1];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, amax16(a[i], b[i]));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantThreads / 32; ++w) m = max(m, warp_max[w]);
  const uint32_t byte = e8m0_of_amax(m << 16);
  const float inv = e8m0_inverse(byte);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + 32 * i;
    if (row < p.rows && col < p.cols)
      *reinterpret_cast<uint4*>(p.q + row * p.ldq + col) = codes16(a[i], b[i], inv);
  }
  if (threadIdx.x == 0) p.scales[rg * p.lds + kg] = static_cast<uint8_t>(byte);
}

// ---------------------------------------------------------------------------
// Residual norm
// ---------------------------------------------------------------------------

struct NormParams {
  const __nv_bfloat16 *x, *y;
  const __nv_bfloat16 *post_weight, *post_bias, *weight, *bias;  // [D], nullable
  const __nv_bfloat16 *gate, *scale, *shift;                     // [mod_rows, D], row stride ld_mod, nullable
  __nv_bfloat16 *h, *u;
  uint8_t *u8, *u_scales;
  int64_t ldx, ldy, ldh, ldu, ld_us, ld_mod;
  uint32_t rows_per_mod;
  int T, D;
  int post_norm, norm;
  int sms, ahead;  // ahead: a row asks for the one that many rows on
  float alpha, eps, inv_d;
  bool few_rows;   // fewer than SMs
};

// Two fp32 values in one 64-bit register, for the paired instructions: the row's arithmetic, not
// its bytes, is what a scalar version of this kernel is bound by (51 instructions an element).
using f2 = uint64_t;
__device__ __forceinline__ f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(f2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum2(f2 v) {
  float a, b;
  unpair(v, a, b);
  return a + b;
}
__device__ __forceinline__ void unpack8(const uint4& a, f2 (&v)[4]) {
  v[0] = pair(bf16_lo(a.x), bf16_hi(a.x)), v[1] = pair(bf16_lo(a.y), bf16_hi(a.y));
  v[2] = pair(bf16_lo(a.z), bf16_hi(a.z)), v[3] = pair(bf16_lo(a.w), bf16_hi(a.w));
}
// Eight elements of a vector or table that many rows read: they stay in L1.  (Not a read-only load:
// this CTA may have been resident while the kernel before wrote a table, and only an ordinary load
// is sure to see that after the grid wait.)
__device__ __forceinline__ void load8(const __nv_bfloat16* p, f2 (&v)[4]) {
  unpack8(*reinterpret_cast<const uint4*>(p), v);
}
// Eight elements of a row that is read once: past L1, which keeps the tables.
__device__ __forceinline__ uint4 load_row8(const __nv_bfloat16* p) {
  uint4 a;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w)
               : "l"(p));
  return a;
}
// A whole row of n bytes (a multiple of 16) into L2.
__device__ __forceinline__ void prefetch_row_l2(const __nv_bfloat16* p, uint32_t n) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(n) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const __nv_bfloat16* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const f2 (&v)[4]) {
  auto two = [](f2 v) {
    float a, b;
    unpair(v, a, b);
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
  };
  *reinterpret_cast<uint4*>(p) = make_uint4(two(v[0]), two(v[1]), two(v[2]), two(v[3]));
}
// Sum over the threads that hold one row: a warp, or the CTA (a fixed order either way).  Sums
// alternate between two parts of the scratch, so that one barrier each is enough: a part is
// written again only after the barrier of the sum between, which every reader has passed.
template <int kThreads>
__device__ __forceinline__ float row_sum(f2 v2, float (*scratch)[32], int& part) {
  float v = sum2(v2);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (kThreads > 32) {
    if ((threadIdx.x & 31) == 0) scratch[part][threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w += 4) {
      const float4 f = *reinterpret_cast<const float4*>(&scratch[part][w]);
      v += (f.x + f.y) + (f.z + f.w);
    }
    part ^= 1;
  }
  return v;
}

// v <- norm(v) over one row of D elements; elements past D (zero) are not part of the sums.
template <int kThreads, int kVecs, bool kFull>
__device__ __forceinline__ void normalise(f2 (&v)[kVecs][4], int kind, const NormParams& p, int lane,
                                          float (*scratch)[32], int& part, const __nv_bfloat16* weight,
                                          const __nv_bfloat16* bias) {
  if (kind == TP_NORM_NONE) return;
  if (kind == TP_NORM_LAYER) {
    f2 s = 0;
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) s = add2(s, v[j][i]);
    const float mean = row_sum<kThreads>(s, scratch, part) * p.inv_d;
    const f2 minus = pair(-mean, -mean);
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
      if (kFull || (j * kThreads + lane) * 8 < p.D)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = add2(v[j][i], minus);
  }
  f2 s = 0;
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fma2(v[j][i], v[j][i], s);
  const float r = rsqrtf(row_sum<kThreads>(s, scratch, part) * p.inv_d + p.eps);  // within 2 ulp
  const f2 rr = pair(r, r);
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[j][i] = mul2(v[j][i], rr);
  if (weight == nullptr && bias == nullptr) return;  // uniform, as every optional vector
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int col = (j * kThreads + lane) * 8;
    if (!kFull && col >= p.D) continue;
    f2 w[4];
    if (weight != nullptr) {
      load8(weight + col, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = mul2(v[j][i], w[i]);
    }
    if (bias != nullptr) {
      load8(bias + col, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = add2(v[j][i], w[i]);
    }
  }
}

// kThreads threads hold a row (32: one warp, four rows a CTA), kVecs vectors of 8 elements each;
// kFull: every vector is inside D, so that nothing is tested against it.
template <int kThreads, int kVecs, bool kFull>
__global__ void __launch_bounds__(kThreads > 32 ? kThreads : 128, kThreads > 32 ? 1024 / kThreads : 8)
    residual_norm_kernel(const NormParams p) {
  __shared__ __align__(16) float scratch[2][32];
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kRows = kThreads > 32 ? 1 : 4;
  const int t = static_cast<int>(blockIdx.x) * kRows + (kRows > 1 ? static_cast<int>(threadIdx.x >> 5) : 0);
  if (t >= p.T) return;  // uniform over a row's threads
  const int lane = kRows > 1 ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int64_t row = t;
  const int64_t mod = p.rows_per_mod > 0 ? static_cast<uint32_t>(t) / p.rows_per_mod * p.ld_mod : 0;
  // Both inputs are asked for at once, and with few rows, where the launch is as long as its chain
  // of memory accesses, the vectors and tables as well.
  uint4 xs[kVecs], ys[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int col = (j * kThreads + lane) * 8;
    xs[j] = ys[j] = make_uint4(0, 0, 0, 0);
    if (kFull || col < p.D) {
      if (p.y != nullptr) ys[j] = load_row8(p.y + row * p.ldy + col);
      xs[j] = load_row8(p.x + row * p.ldx + col);
    }
  }
  if (p.few_rows) {
    const __nv_bfloat16* const vectors[4] = {p.post_weight, p.post_bias, p.weight, p.bias};
    const __nv_bfloat16* const tables[3] = {p.gate, p.scale, p.shift};
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int col = (j * kThreads + lane) * 8;
      if (kFull || col < p.D) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (tables[i] != nullptr) prefetch_l2(tables[i] + mod + col);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (vectors[i] != nullptr) prefetch_l2(vectors[i] + col);
      }
    }
  } else if (lane == 0 && t < p.T - p.ahead) {
    // A row's threads wait for it and then work on it with no other row in flight, so each asks for
    // a row that is not far from its turn to be in L2 by then (42.7 -> 40.3 us at 4608 x 6144).
    if (p.y != nullptr) prefetch_row_l2(p.y + (row + p.ahead) * p.ldy, 2 * static_cast<uint32_t>(p.D));
    prefetch_row_l2(p.x + (row + p.ahead) * p.ldx, 2 * static_cast<uint32_t>(p.D));
  }
  f2 v[kVecs][4];  // zero past D
  int part = 0;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) unpack8(ys[j], v[j]);
  if (p.y != nullptr)
    normalise<kThreads, kVecs, kFull>(v, p.post_norm, p, lane, scratch, part, p.post_weight, p.post_bias);
  const f2 alpha = pair(p.alpha, p.alpha);
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int col = (j * kThreads + lane) * 8;
    if (!kFull && col >= p.D) continue;
    f2 x[4];
    unpack8(xs[j], x);
    if (p.gate != nullptr) {
      f2 g[4];
      load8(p.gate + mod + col, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = mul2(v[j][i], g[i]);
    }
    if (p.y != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = fma2(alpha, x[i], v[j][i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = mul2(alpha, x[i]);
    }
    if (p.h != nullptr) store8(p.h + row * p.ldh + col, v[j]);
  }
  if (p.u == nullptr && p.u8 == nullptr) return;  // uniform over the grid
  normalise<kThreads, kVecs, kFull>(v, p.norm, p, lane, scratch, part, p.weight, p.bias);
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int col = (j * kThreads + lane) * 8;
    const bool on = kFull || col < p.D;
    f2 s[4];
    if (on && p.scale != nullptr) {
      load8(p.scale + mod + col, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = fma2(v[j][i], s[i], v[j][i]);
    }
    if (on && p.shift != nullptr) {
      load8(p.shift + mod + col, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = add2(v[j][i], s[i]);
    }
    if (p.u != nullptr) {
      if (on) store8(p.u + row * p.ldu + col, v[j]);
      continue;
    }
    // 16 lanes hold a group of 128.
    float e[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpair(v[j][i], e[2 * i], e[2 * i + 1]);
    float m = max_abs(max_abs(max_abs(e[0], e[1]), max_abs(e[2], e[3])),
                      max_abs(max_abs(e[4], e[5]), max_abs(e[6], e[7])));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t byte = e8m0_of_amax(abs_bits(m));
    const float inv = e8m0_inverse(byte);
    if (on) {
      const f2 ii = pair(inv, inv);
#pragma unroll
      for (int i = 0; i < 4; ++i) unpair(mul2(v[j][i], ii), e[2 * i], e[2 * i + 1]);
      *reinterpret_cast<uint2*>(p.u8 + row * p.ldu + col) =
          make_uint2(e4m3x4(e[0], e[1], e[2], e[3]), e4m3x4(e[4], e[5], e[6], e[7]));
      if ((lane & 15) == 0) p.u_scales[row * p.ld_us + col / kFp8Group] = static_cast<uint8_t>(byte);
    }
  }
}

template <int kThreads, int kVecs>
tp_status launch_norm(NormParams& p, cudaStream_t stream) {
  constexpr int kRows = kThreads > 32 ? 1 : 4;
  // Half of the rows the GPU works on at a time (a quarter to one and a half times them: 44.7 to 46.5 us).
  p.ahead = p.sms * (kThreads > 32 ? 1024 / kThreads : 8) * kRows / 2;
  auto kernel = p.D == kThreads * kVecs * 8 ? residual_norm_kernel<kThreads, kVecs, true>
                                            : residual_norm_kernel<kThreads, kVecs, false>;
  cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>((p.T + kRows - 1) / kRows)),
                             dim3(kThreads > 32 ? kThreads : 128), 0, stream, p);
  if (e != cudaSuccess) return cuda_fail(e, "residual norm launch");
  return TP_OK;
}

// Threads and vectors for a row of D: rows up to 512 wide take a warp, longer ones a CTA whose
// threads hold few vectors (4608 x 1024: 8.3 us with a warp of four vectors, 7.9 with four of
// one; 4608 x 6144: 42.6 us with 192 threads of four, 40.3 with 256 of three, 43.2 with 384 of two,
// 60 with 768 of one).  With fewer rows than SMs a launch is one row's latency, and a thread gets
// one vector where that fits.
tp_status dispatch_norm(NormParams& p, cudaStream_t s) {
  const int vecs = (p.D + 7) / 8;
  if (!p.few_rows && vecs <= 32) return launch_norm<32, 1>(p, s);
  if (!p.few_rows && vecs <= 64) return launch_norm<32, 2>(p, s);
  if (vecs <= 128) return launch_norm<128, 1>(p, s);
  if (vecs <= 256) return launch_norm<256, 1>(p, s);
  if (p.few_rows && vecs <= 512) return launch_norm<512, 1>(p, s);
  if (p.few_rows && vecs <= 1024) return launch_norm<1024, 1>(p, s);
  if (vecs <= 512) return launch_norm<256, 2>(p, s);
  if (vecs <= 768) return launch_norm<256, 3>(p, s);
  if (vecs <= 1024) return launch_norm<256, 4>(p, s);
  if (vecs <= 1536) return launch_norm<512, 3>(p, s);
  if (vecs <= 2048) return launch_norm<512, 4>(p, s);
  return launch_norm<1024, 4>(p, s);
}

}  // namespace
}  // namespace tp

extern "C" {

tp_status tp_quantize_fp8(const void* x, int64_t ldx, int64_t rows, int64_t cols, int block_rows, void* q, int64_t ldq,
                          void* scales, int64_t lds, tp_stream_t stream) {
  using namespace tp;
  return guarded([&]() -> tp_status {
    clear_error();
    if (rows < 0 || cols < 0) return fail(TP_ERR_INVALID_ARG, "negative size");
    if (block_rows != 1 && block_rows != kFp8Group)
      return fail(TP_ERR_INVALID_ARG, "block_rows must be 1 or %d, got %d", kFp8Group, block_rows);
    if (cols > 0x7FFFFFFF) return fail(TP_ERR_UNSUPPORTED, "sizes above 2^31-1 are not supported");
    const int64_t col_groups = (cols + kFp8Group - 1) / kFp8Group;
    if (ldx == 0) ldx = cols;
    if (ldq == 0) ldq = cols;
    if (lds == 0) lds = col_groups;
    if (ldx < cols || ldq < cols || lds < col_groups)
      return fail(TP_ERR_INVALID_ARG, "a row stride (ldx %lld, ldq %lld, lds %lld) is smaller than its row",
                  (long long)ldx, (long long)ldq, (long long)lds);
    if (rows == 0 || cols == 0) return TP_OK;
    if (x == nullptr || q == nullptr || scales == nullptr)
      return fail(TP_ERR_INVALID_ARG, "x, q or scales is NULL");
    if (cols % 16 != 0 || ldx % 8 != 0 || ldq % 16 != 0)
      return fail(TP_ERR_ALIGNMENT, "cols (%lld) and ldq (%lld) must be multiples of 16, ldx (%lld) of 8",
                  (long long)cols, (long long)ldq, (long long)ldx);
    if (!aligned16(x) || !aligned16(q)) return fail(TP_ERR_ALIGNMENT, "x or q is not 16-byte aligned");
    const int64_t row_groups = (rows + block_rows - 1) / block_rows;
    const int64_t per_cta = block_rows == 1 ? kQuantThreads / 8 : 1;
    if (row_groups > 0x7FFFFFFFll * per_cta / col_groups) return fail(TP_ERR_UNSUPPORTED, "too many groups");
    const int64_t blocks = (row_groups * col_groups + per_cta - 1) / per_cta;
    QuantParams p{};
    p.x = static_cast<const uint8_t*>(x);
    p.q = static_cast<uint8_t*>(q);
    p.scales = static_cast<uint8_t*>(scales);
    p.ldx = ldx * 2;
    p.ldq = ldq;
    p.lds = lds;
    p.rows = rows;
    p.cols = static_cast<int>(cols);
    p.col_groups = static_cast<int>(col_groups);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_pdl(block_rows == 1 ? quantize_rows_kernel : quantize_blocks_kernel,
                               dim3(static_cast<unsigned>(blocks)), dim3(kQuantThreads), 0, s, p);
    if (e != cudaSuccess) return cuda_fail(e, "quantiser launch");
    return TP_OK;
  });
}

tp_status tp_residual_norm(const tp_residual_norm_args* a, tp_stream_t stream) {
  using namespace tp;
  return guarded([&]() -> tp_status {
    clear_error();
    if (a == nullptr) return fail(TP_ERR_INVALID_ARG, "args is NULL");
    if (a->T < 0 || a->D < 0) return fail(TP_ERR_INVALID_ARG, "negative size");
    auto known = [](int k) { return k == TP_NORM_NONE || k == TP_NORM_RMS || k == TP_NORM_LAYER; };
    if (!known(a->norm) || !known(a->post_norm))
      return fail(TP_ERR_INVALID_ARG, "unknown norm %d or post_norm %d", (int)a->norm, (int)a->post_norm);
    if (!(a->eps >= 0.0f) || std::isinf(a->eps)) return fail(TP_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (a->D > TP_NORM_MAX_D)
      return fail(TP_ERR_UNSUPPORTED, "rows wider than %d are not supported, got %lld", TP_NORM_MAX_D, (long long)a->D);
    if (a->T > 0x7FFFFFF0) return fail(TP_ERR_UNSUPPORTED, "too many rows (%lld)", (long long)a->T);
    NormParams p{};
    p.ldx = a->ldx == 0 ? a->D : a->ldx;
    p.ldy = a->ldy == 0 ? a->D : a->ldy;
    p.ldh = a->ldh == 0 ? a->D : a->ldh;
    p.ldu = a->ldu == 0 ? a->D : a->ldu;
    const int64_t groups = (a->D + kFp8Group - 1) / kFp8Group;
    p.ld_us = a->ld_u_scales == 0 ? groups : a->ld_u_scales;
    p.ld_mod = a->ld_mod == 0 ? a->D : a->ld_mod;
    if (p.ldx < a->D || p.ldy < a->D || p.ldh < a->D || p.ldu < a->D || p.ld_mod < a->D || p.ld_us < groups)
      return fail(TP_ERR_INVALID_ARG, "a row stride is smaller than its row");
    if (a->T == 0 || a->D == 0) return TP_OK;
    if (a->x == nullptr) return fail(TP_ERR_INVALID_ARG, "x is NULL");
    if (a->h == nullptr && a->u == nullptr) return fail(TP_ERR_INVALID_ARG, "neither h nor u is wanted");
    if (a->y == nullptr && (a->h != nullptr || a->gate != nullptr || a->post_norm != TP_NORM_NONE))
      return fail(TP_ERR_INVALID_ARG, "h, gate and post_norm belong to a branch y, which is NULL");
    if ((a->post_weight != nullptr || a->post_bias != nullptr) && a->post_norm == TP_NORM_NONE)
      return fail(TP_ERR_INVALID_ARG, "post_weight or post_bias without a post_norm");
    if ((a->weight != nullptr || a->bias != nullptr) && a->norm == TP_NORM_NONE)
      return fail(TP_ERR_INVALID_ARG, "weight or bias without a norm");
    const bool fp8 = a->u != nullptr && a->u_scales != nullptr;
    if (a->u == nullptr && (a->u_scales != nullptr || a->scale != nullptr || a->shift != nullptr ||
                            a->norm != TP_NORM_NONE))
      return fail(TP_ERR_INVALID_ARG, "norm, scale, shift and u_scales belong to u, which is NULL");
    if (a->gate != nullptr || a->scale != nullptr || a->shift != nullptr) {
      if (a->rows_per_mod < 1 || a->mod_rows < 1)
        return fail(TP_ERR_INVALID_ARG, "rows_per_mod and mod_rows must be positive with a gate, scale or shift");
      if ((a->T - 1) / a->rows_per_mod >= a->mod_rows)
        return fail(TP_ERR_INVALID_ARG, "%lld rows, %lld to a modulation row, need more than %lld modulation rows",
                    (long long)a->T, (long long)a->rows_per_mod, (long long)a->mod_rows);
      p.rows_per_mod = static_cast<uint32_t>(a->rows_per_mod < a->T ? a->rows_per_mod : a->T);
    }
    const int64_t step = fp8 ? 16 : 8;
    if (a->D % step != 0 || p.ldu % step != 0)
      return fail(TP_ERR_ALIGNMENT, "D (%lld) and ldu (%lld) must be multiples of %lld", (long long)a->D,
                  (long long)p.ldu, (long long)step);
    if (p.ldx % 8 != 0 || p.ldy % 8 != 0 || p.ldh % 8 != 0 || p.ld_mod % 8 != 0)
      return fail(TP_ERR_ALIGNMENT, "ldx, ldy, ldh and ld_mod must be multiples of 8");
    const void* ptrs[] = {a->x, a->y, a->post_weight, a->post_bias, a->gate, a->weight, a->bias,
                          a->scale, a->shift, a->h, a->u};
    for (const void* q : ptrs)
      if (!aligned16(q)) return fail(TP_ERR_ALIGNMENT, "a pointer is not 16-byte aligned");
    p.x = static_cast<const __nv_bfloat16*>(a->x);
    p.y = static_cast<const __nv_bfloat16*>(a->y);
    p.post_weight = static_cast<const __nv_bfloat16*>(a->post_weight);
    p.post_bias = static_cast<const __nv_bfloat16*>(a->post_bias);
    p.weight = static_cast<const __nv_bfloat16*>(a->weight);
    p.bias = static_cast<const __nv_bfloat16*>(a->bias);
    p.gate = static_cast<const __nv_bfloat16*>(a->gate);
    p.scale = static_cast<const __nv_bfloat16*>(a->scale);
    p.shift = static_cast<const __nv_bfloat16*>(a->shift);
    p.h = static_cast<__nv_bfloat16*>(a->h);
    p.u = fp8 ? nullptr : static_cast<__nv_bfloat16*>(a->u);
    p.u8 = fp8 ? static_cast<uint8_t*>(a->u) : nullptr;
    p.u_scales = static_cast<uint8_t*>(a->u_scales);
    p.T = static_cast<int>(a->T);
    p.D = static_cast<int>(a->D);
    p.inv_d = 1.0f / static_cast<float>(p.D);
    p.post_norm = a->post_norm;
    p.norm = a->norm;
    p.alpha = a->alpha;
    p.eps = a->eps;
    p.sms = sm_count();
    if (p.sms <= 0) return fail(TP_ERR_CUDA, "cannot query the SM count of the current device");
    p.few_rows = a->T <= p.sms;
    return dispatch_norm(p, reinterpret_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
