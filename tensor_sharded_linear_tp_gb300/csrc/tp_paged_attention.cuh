// What the kernels of the attention over the paged cache share: their parameters, how a sequence's
// rows are cut into items and an item's keys into steps, and the join of partial results.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "tp_paged.h"

namespace tp {

// An item in `n` CTAs (0: none), whose parts are to be joined.
struct Join {
  int n, a, row0, rows, h, pad[3];
};

// Division by a number that the host knows, of n < 2^31: m = ceil(2^(31 + s) / d), s = ceil(log2 d), is less than
// 2^32 and off by less than d / 2^(31 + s) relative, so n m / 2^(31 + s) has the quotient's whole part.
struct Div {
  uint32_t m;
  int s;
#ifdef __CUDACC__
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * m) >> (31 + s));
  }
#endif
};
inline Div div_by(uint32_t d) {
  int s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  return {static_cast<uint32_t>(((uint64_t(1) << (31 + s)) + d - 1) / d), s};
}

struct AttendParams {
  BatchView b;
  int64_t ld_q, ldo, ld_page, ld_scales;
  int n_kv, group;             // KV heads of a rank, query heads of a KV head
  int heads;                   // n_ranks * n_kv
  Div by_kv, by_group;
  int causal, window;
  float scale_log2e;
  int per_item;                // 1: a CTA takes one item whole; 0: equal parts of all steps
  float* parts;                // workspace: two partial items a CTA, O and then (m, l) of each row
  float* early;                // workspace (paged_rows_kernel): a piece of each warp that it leaves behind
  float* carry;                // workspace: the piece that another one continues, of a CTA (paged_rows_kernel: of a warp, and the other)
  Join* joins;                 // workspace: the item that begins in a CTA and goes beyond it
  const __nv_bfloat16* q[TP_MAX_DEGREE];
  __nv_bfloat16* out[TP_MAX_DEGREE];
  const uint8_t *k[TP_MAX_DEGREE], *v[TP_MAX_DEGREE], *ks[TP_MAX_DEGREE], *vs[TP_MAX_DEGREE];
};
// The tensor maps of the codes, [pages][heads][tokens][D], boxes of one page's tokens (at most 32).
struct CodeMaps {
  CUtensorMap k[TP_MAX_DEGREE], v[TP_MAX_DEGREE];
};

// The keys of a piece, at most.  The tensor core's accumulators are fp32, but what a product has below the sum's last
// places is cut off, not rounded, so that a long sum falls short: by 0.05 % over 2^19 keys of equal weight (measured,
// either kernel), 0.1 % over 2^20, 0.3 over 2^21, 0.7 over 2^22, 2 over 2^23, and from some 2^26 on nothing is added any
// more.  Pieces are joined by sums that round.
constexpr int kLongestPiece = 1 << 19;

// One item: rows [row0, row0 + rows) of a sequence's n * group rows (token by token), and its steps.
struct Item {
  SeqView v;
  int row0, rows;
  int tile0, tiles;     // steps tile0 .. tile0 + tiles of the sequence's keys
  int key_lo, key_end;  // some row sees key_lo; none sees an earlier key, nor one from key_end on
};

template <int ROWS, int STEP>
__device__ __forceinline__ Item item_of(const AttendParams& p, const SeqView& v, int block) {
  Item it;
  it.v = v;
  it.row0 = block * ROWS;
  it.rows = static_cast<int>(min(static_cast<int64_t>(ROWS), static_cast<int64_t>(v.n) * p.group - it.row0));
  const int first = p.by_group(it.row0), last = p.by_group(it.row0 + max(it.rows, 1) - 1);
  it.key_end = p.causal ? max(min(static_cast<int64_t>(v.len), static_cast<int64_t>(v.pos0) + last + 1), int64_t(0)) : v.len;
  it.key_lo = p.window > 0 ? static_cast<int>(max(static_cast<int64_t>(v.pos0) + first - p.window + 1, int64_t(0))) : 0;
  it.tile0 = min(it.key_lo, it.key_end) / STEP;
  it.tiles = it.rows > 0 ? max(1, (it.key_end + STEP - 1) / STEP - it.tile0) : 0;   // (a row without keys is an item too)
  return it;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^e, 0 below fp32's normal range.
__device__ __forceinline__ float pow2(int e) {
  return e < -126 ? 0.0f : __uint_as_float(static_cast<uint32_t>(min(e, 127) + 127) << 23);
}
// A scale byte's value (NaN for 255).
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FFFFFFFu) : byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Some pieces of a row joined: the largest m, the sum of l 2^(m_i - m) and the sum of these times O.
struct Joined {
  float m, l;
  float4 o;
};
// Pieces first, first + step, ... below n in this order, eight of them read at once.
template <typename ML, typename O4>
__device__ __forceinline__ Joined join_pieces(int first, int step, int n, ML&& ml, O4&& o4) {
  Joined j{-INFINITY, 0.0f, make_float4(0, 0, 0, 0)};
#pragma unroll 1
  for (int i0 = first; i0 < n; i0 += 8 * step) {
    float2 v[8];
    float4 o[8];
    float m = j.m;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = make_float2(-INFINITY, 0.0f), o[k] = make_float4(0, 0, 0, 0);
      if (i0 + k * step < n) v[k] = ml(i0 + k * step), o[k] = o4(i0 + k * step);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, v[k].x);
    const float ref = m == -INFINITY ? 0.0f : m, keep = ex2(j.m - ref);
    j.m = m;
    j.l *= keep;
    j.o.x *= keep, j.o.y *= keep, j.o.z *= keep, j.o.w *= keep;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float w = v[k].y * ex2(v[k].x - ref);
      j.l += w;
      j.o.x += w * o[k].x, j.o.y += w * o[k].y, j.o.z += w * o[k].z, j.o.w += w * o[k].w;
    }
  }
  return j;
}

__device__ __forceinline__ void store_row4(const AttendParams& p, int a, int h, int row, int col, int D, const float4& v) {
  const int rank = p.by_kv(h), head = h - rank * p.n_kv;
  const int token = p.by_group(row), hq = row - token * p.group;
  __nv_bfloat16* dst = p.out[rank] + static_cast<int64_t>(a + token) * p.ldo + (static_cast<int64_t>(head) * p.group + hq) * D + col;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

// Part of a page (tokens from `token` on) and head into shared memory.
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, uint32_t bar, int token, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(0), "r"(token), "r"(head), "r"(page)
      : "memory");
}

// Where the steps of all items are cut: into n parts of q or q + 1 steps, the longer ones first.
struct Cuts {
  int64_t q, r;
  __device__ __forceinline__ Cuts(int64_t total, int64_t n) : q(total / n), r(total - q * n) {}
  __device__ __forceinline__ int64_t at(int64_t c) const { return c * q + min(c, r); }      // the first step of part c
  __device__ __forceinline__ int64_t part(int64_t u) const {                                // of step u
    return u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q;
  }
};

constexpr int kJoinThreads = 256;
template <int D, int GROUPS>
constexpr int kJoinRows = kJoinThreads / GROUPS / (D / 4);   // of a block

// Joins the items that lie in several CTAs: blocks (c, .) the one that begins in CTA c and goes beyond
// it (its piece in that CTA's second part, the others in the first parts of those behind).  GROUPS
// groups of threads take every GROUPS-th piece of a row each: a long item of few rows lies in many CTAs.
template <int D, int ROWS, int GROUPS>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ AttendParams p) {
  constexpr int PART = ROWS * (D + 2), QUADS = D / 4, PER = kJoinThreads / GROUPS;
  __shared__ Joined found[GROUPS > 1 ? kJoinThreads : 1];
  pdl_launch_dependents();
  pdl_wait();
  const Join join = p.joins[blockIdx.x];
  if (join.n == 0 || static_cast<int>(blockIdx.y) * kJoinRows<D, GROUPS> >= join.rows) return;
  const int group = threadIdx.x / PER, in = threadIdx.x % PER;
  const int row = blockIdx.y * kJoinRows<D, GROUPS> + in / QUADS, at = row * D + in % QUADS * 4;
  const float* own = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + 1) * PART;
  auto part = [&](int i) { return i == 0 ? own : own + (2 * i - 1) * static_cast<int64_t>(PART); };
  Joined j{-INFINITY, 0.0f, make_float4(0, 0, 0, 0)};
  if (row < join.rows)
    j = join_pieces(group, GROUPS, join.n, [&](int i) { return *reinterpret_cast<const float2*>(part(i) + ROWS * D + 2 * row); },
                    [&](int i) { return *reinterpret_cast<const float4*>(part(i) + at); });
  if constexpr (GROUPS > 1) {
    found[threadIdx.x] = j;
    __syncthreads();
    if (group > 0) return;
    j = join_pieces(0, 1, GROUPS, [&](int i) { return make_float2(found[i * PER + in].m, found[i * PER + in].l); },
                    [&](int i) {
                      const Joined& f = found[i * PER + in];
                      const float inv = f.l == 0.0f ? 0.0f : 1.0f / f.l;
                      return make_float4(f.o.x * inv, f.o.y * inv, f.o.z * inv, f.o.w * inv);
                    });
  }
  if (row >= join.rows) return;
  const float inv = j.l == 0.0f ? 0.0f : 1.0f / j.l;
  store_row4(p, join.a, join.h, join.row0 + row, in % QUADS * 4, D, make_float4(j.o.x * inv, j.o.y * inv, j.o.z * inv, j.o.w * inv));
}

// The kernel for many rows a KV head (tp_paged_tiles.cu).
size_t paged_tiles_part_floats(int head_dim);
tp_status launch_paged_tiles(int head_dim, int ctas, const AttendParams& p, const CodeMaps& maps, cudaStream_t stream);

}  // namespace tp
