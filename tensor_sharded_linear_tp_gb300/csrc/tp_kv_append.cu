// Appending keys and values to the paged 8-bit cache, with the position rotation of Q and K.
//
// One launch over every rank.  Its first blocks rotate Q (a warp takes one token and up to four
// times 32 lanes' worth of its heads); the others each quantise, for one KV head, the new tokens
// of one page, since these share a scale:
//     e = max(e_old if the page holds older tokens, least e with max|x| <= 448 * 2^e)
// A warp holds 16 tokens of the page in registers as fp32 (rotated), a page of P tokens is held by
// P / 16 warps, and the maximum is joined by one warp reduction and, for larger pages, through
// shared memory: every element is read once and written once.  Only where e grew are the older
// tokens' codes read and written again, scaled by 2^(e_old - e): exact but for codes that fall
// among the subnormal ones, since scales are powers of two.
//
// Which sequence and page a block has comes from the device's seq_start without a prefix sum
// (find_sequence), so that lengths may change between the replays of a graph.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "tp_e4m3.cuh"
#include "tp_internal.h"
#include "tp_paged.h"

namespace tp {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kQRounds = 4;   // rounds of heads a warp of the Q part takes

struct AppendParams {
  BatchView b;
  const __nv_bfloat16* qkv[TP_MAX_DEGREE];
  __nv_bfloat16* q_out[TP_MAX_DEGREE];
  uint8_t *k[TP_MAX_DEGREE], *v[TP_MAX_DEGREE], *ks[TP_MAX_DEGREE], *vs[TP_MAX_DEGREE];
  int64_t ld_qkv, ld_q, ld_page, ld_scales;
  const float* cos_sin;        // NULL: no rotation
  const int32_t* positions;
  int64_t ld_rope, n_positions;
  int style, rot;              // rot 0: no rotation
  int n_heads, n_kv;
  int q_units, q_blocks;       // units of kQRounds rounds of heads a token; blocks of the Q part
  int64_t kv_units;
  int slot_per, slot_gap;      // numbering of the pages (find_sequence)
};

// Two chunks of 8 elements that a thread holds of one head: for rotated elements x[i] and
// x[i + rot/2] are at the same place of chunk 0 and 1 (TP_ROPE_HALF), and no pair of neighbours is
// cut (TP_ROPE_PAIRS); behind them two neighbouring chunks.
struct Chunks {
  int c0, c1;
  bool turned;
};
__device__ __forceinline__ Chunks chunks_of(int part, int rot) {
  const int half = rot / 16;
  if (part < half) return {part, part + half, true};
  const int c = rot / 8 + 2 * (part - half);
  return {c, c + 1, false};
}

struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void load8(float* dst, const float* src) {
  *reinterpret_cast<float4*>(dst) = *reinterpret_cast<const float4*>(src);
  *reinterpret_cast<float4*>(dst + 4) = *reinterpret_cast<const float4*>(src + 4);
}
// The cosines and sines of a token's two chunks; NaN where its row is outside the table.
__device__ __forceinline__ void load_turn(Turn& t, const AppendParams& p, int64_t at, const Chunks& ch) {
  if (at < 0 || at >= p.n_positions) {
    bad_index(p.b);
#pragma unroll
    for (int i = 0; i < 8; ++i) t.c[i] = t.s[i] = __uint_as_float(0x7FFFFFFFu);
    return;
  }
  const float* row = p.cos_sin + at * p.ld_rope;
  if (p.style == TP_ROPE_HALF) {
    load8(t.c, row + 8 * ch.c0);
    load8(t.s, row + p.rot / 2 + 8 * ch.c0);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 4 * (h == 0 ? ch.c0 : ch.c1);
      *reinterpret_cast<float4*>(t.c + 4 * h) = *reinterpret_cast<const float4*>(row + i);
      *reinterpret_cast<float4*>(t.s + 4 * h) = *reinterpret_cast<const float4*>(row + p.rot / 2 + i);
    }
  }
}

__device__ __forceinline__ void unpack8(float* x, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = x * c - y * s;
  b = y * c + x * s;
}
// x: chunk c0 in [0, 8), chunk c1 in [8, 16).
__device__ __forceinline__ void rotate(float (&x)[16], const Turn& t, int style) {
  if (style == TP_ROPE_HALF) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(x[i], x[8 + i], t.c[i], t.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(x[2 * i], x[2 * i + 1], t.c[i], t.s[i]);
  }
}

// Q of one token: kQRounds rounds of 32 / kParts heads, a head held by kParts = D / 16 threads.
template <int D>
__device__ __forceinline__ void rotate_q(const AppendParams& p, int rank, int64_t unit, int lane) {
  constexpr int kParts = D / 16, kHeads = 32 / kParts;
  if (unit >= static_cast<int64_t>(p.b.T) * p.q_units) return;
  const int t = static_cast<int>(unit / p.q_units);
  const int h0 = static_cast<int>(unit - static_cast<int64_t>(t) * p.q_units) * kQRounds * kHeads + lane / kParts;
  const Chunks ch = chunks_of(lane % kParts, p.rot);
  const __nv_bfloat16* src = p.qkv[rank] + t * p.ld_qkv;
  uint4 raw[kQRounds][2];
#pragma unroll
  for (int i = 0; i < kQRounds; ++i) {
    const int h = h0 + i * kHeads;
    if (h < p.n_heads) {
      raw[i][0] = *reinterpret_cast<const uint4*>(src + h * D + 8 * ch.c0);
      raw[i][1] = *reinterpret_cast<const uint4*>(src + h * D + 8 * ch.c1);
    }
  }
  // The row's position; rows of no sequence are left alone.
  const int s = find_sequence(p.b, t, 1, 1, 0, lane);
  if (s < 0) return;
  const SeqView v = seq_view(p.b, s);
  const int i_new = t - v.a;
  if (i_new >= v.n) return;
  Turn turn;
  if (ch.turned) load_turn(turn, p, p.positions != nullptr ? p.positions[t] : v.pos0 + i_new, ch);
  __nv_bfloat16* dst = p.q_out[rank] + t * p.ld_q;
#pragma unroll
  for (int i = 0; i < kQRounds; ++i) {
    const int h = h0 + i * kHeads;
    if (h < p.n_heads) {
      if (ch.turned) {
        float x[16];
        unpack8(x, raw[i][0]);
        unpack8(x + 8, raw[i][1]);
        rotate(x, turn, p.style);
        raw[i][0] = pack8(x);
        raw[i][1] = pack8(x + 8);
      }
      *reinterpret_cast<uint4*>(dst + h * D + 8 * ch.c0) = raw[i][0];
      *reinterpret_cast<uint4*>(dst + h * D + 8 * ch.c1) = raw[i][1];
    }
  }
}

// Sixteen codes times a power of two (or NaN), rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  float x[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> (16 * i))));
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
        : "r"(h));
  }
  return e4m3x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
}

template <int D>
__device__ __forceinline__ void append_page(const AppendParams& p, int rank, int64_t block, uint32_t* warp_top) {
  constexpr int kParts = D / 16, kTokens = 32 / kParts, kRounds = 16 / kTokens;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int P = p.b.page_size, warps = P / 16;     // warps of a page
  const int64_t unit = block * (kWarps / warps) + warp / warps;
  const int64_t slot = unit / (2 * p.n_kv);
  const int rest = static_cast<int>(unit - slot * (2 * p.n_kv));
  const bool is_v = rest >= p.n_kv;
  const int head = is_v ? rest - p.n_kv : rest;

  // Which tokens [j0, j1) of which sequence, in which page.
  int j0 = 0, j1 = 0, row0 = 0;                    // the row of position j is row0 + j
  int64_t page = -1;
  const int s = unit < p.kv_units ? find_sequence(p.b, slot, p.slot_per, 1, p.slot_gap, lane) : -1;
  if (s >= 0) {
    const SeqView v = seq_view(p.b, s);
    const int64_t local = slot - (v.a / p.slot_per + static_cast<int64_t>(p.slot_gap) * s);
    const int64_t at = (max(v.pos0, 0) >> p.b.page_shift) + local;
    const int64_t end = static_cast<int64_t>(v.pos0) + v.n;
    if (v.n > 0 && v.pos0 < 0 && lane == 0) bad_index(p.b);
    if (at * P < end) {
      j0 = max(static_cast<int>(at * P), v.pos0);
      j1 = static_cast<int>(min((at + 1) * P, end));
      row0 = v.a - v.pos0;
      if (j0 < j1 && at * P < p.b.max_keys) page = p.b.page_table[s * p.b.ld_table + at];
      if (j0 < j1 && (page < 0 || page >= p.b.n_pages)) {
        bad_index(p.b);
        page = -1;
      }
      if (page < 0) j1 = j0;
    }
  }

  // This warp's 16 slots: the new values in fp32, and their largest magnitude.
  const int base = (j0 & ~(P - 1)) + 16 * (warp % warps);
  const int rot = is_v ? 0 : p.rot;
  const Chunks ch = chunks_of(lane % kParts, rot);
  const __nv_bfloat16* src = p.qkv[rank] + (p.n_heads + (is_v ? p.n_kv : 0) + head) * static_cast<int64_t>(D);
  float x[kRounds][16];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int j = base + i * kTokens + lane / kParts;
    if (j >= j0 && j < j1) {
      const int64_t row = row0 + j;
      const uint4* at = reinterpret_cast<const uint4*>(src + row * p.ld_qkv);
      unpack8(x[i], at[ch.c0]);
      unpack8(x[i] + 8, at[ch.c1]);
      if (ch.turned) {
        Turn t;
        load_turn(t, p, p.positions != nullptr ? p.positions[row] : j, ch);
        rotate(x[i], t, p.style);
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) top = max(top, abs_bits(x[i][k]));
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  uint8_t* scale = (is_v ? p.vs : p.ks)[rank] + page * p.ld_scales + head;
  const bool older = page >= 0 && (j0 & (P - 1)) != 0;
  const uint32_t old_byte = older ? *scale : 0u;
  if (lane == 0) warp_top[warp] = top;
  __syncthreads();   // (every warp has read the old scale as well)
  for (int w = warp / warps * warps, i = 0; i < warps; ++i) top = max(top, warp_top[w + i]);
  if (page < 0) return;
  const uint32_t byte = max(old_byte, top == 0u ? 0u : e8m0_of_amax(top));
  uint8_t* codes = (is_v ? p.v : p.k)[rank] + page * p.ld_page + static_cast<int64_t>(head) * P * D;
  if (warp % warps == 0 && lane == 0) *scale = static_cast<uint8_t>(byte);
  if (byte > old_byte && older) {   // the older tokens' codes at the new scale
    const float f = byte == 255u ? __uint_as_float(0x7FFFFFFFu)
                                 : byte - old_byte > 126u ? 0.0f : __uint_as_float((127u - (byte - old_byte)) << 23);
    const int end = min(16, (j0 & (P - 1)) - 16 * (warp % warps)) * (D / 16);
    uint4* at = reinterpret_cast<uint4*>(codes + 16 * (warp % warps) * D);
    for (int i = lane; i < end; i += 32) {
      const uint4 v = at[i];
      at[i] = make_uint4(rescale4(v.x, f), rescale4(v.y, f), rescale4(v.z, f), rescale4(v.w, f));
    }
  }
  const float inv = e8m0_inverse(byte);
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int j = base + i * kTokens + lane / kParts;
    if (j >= j0 && j < j1) {
      uint2* to = reinterpret_cast<uint2*>(codes + (j & (P - 1)) * D);
      float* y = x[i];
#pragma unroll
      for (int k = 0; k < 16; ++k) y[k] *= inv;
      to[ch.c0] = make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
      to[ch.c1] = make_uint2(e4m3x4(y[8], y[9], y[10], y[11]), e4m3x4(y[12], y[13], y[14], y[15]));
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ uint32_t warp_top[kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int rank = blockIdx.y;
  if (static_cast<int>(blockIdx.x) < p.q_blocks)
    rotate_q<D>(p, rank, static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), threadIdx.x & 31);
  else
    append_page<D>(p, rank, static_cast<int64_t>(blockIdx.x) - p.q_blocks, warp_top);
}

}  // namespace

tp_status check_paged(const tp_paged_cache* c, const tp_paged_batch* b, int64_t T, int n_heads, bool* empty) {
  if (c == nullptr || b == nullptr) return fail(TP_ERR_INVALID_ARG, "cache or batch is NULL");
  if (c->n_ranks < 1) return fail(TP_ERR_INVALID_ARG, "n_ranks must be >= 1, got %d", c->n_ranks);
  if (c->n_ranks > TP_MAX_DEGREE)
    return fail(TP_ERR_UNSUPPORTED, "n_ranks=%d above TP_MAX_DEGREE=%d", c->n_ranks, TP_MAX_DEGREE);
  if (c->n_kv_heads < 1 || n_heads < 0 || c->n_pages < 0 || T < 0 || b->n_seqs < 0 || b->max_new < 0 || b->max_pages < 0)
    return fail(TP_ERR_INVALID_ARG, "negative size, or no KV head");
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(TP_ERR_UNSUPPORTED, "head_dim must be 64 or 128, got %d", c->head_dim);
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return fail(TP_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128, got %d", c->page_size);
  constexpr int64_t kMost = int64_t(1) << 30;
  if (n_heads > 65535 || c->n_kv_heads > 65535 || T > kMost || c->n_pages > kMost || b->max_pages > kMost / c->page_size ||
      b->n_seqs > (1 << 24))
    return fail(TP_ERR_UNSUPPORTED, "sizes above 2^30 rows, pages or keys of a sequence, 65535 heads or 2^24 sequences");
  const int64_t page = static_cast<int64_t>(c->n_kv_heads) * c->page_size * c->head_dim;
  if ((c->ld_page != 0 && c->ld_page < page) || (c->ld_scales != 0 && c->ld_scales < c->n_kv_heads) ||
      (b->ld_table != 0 && b->ld_table < b->max_pages))
    return fail(TP_ERR_INVALID_ARG, "a stride (ld_page %lld, ld_scales %lld, ld_table %lld) is smaller than what it spans",
                (long long)c->ld_page, (long long)c->ld_scales, (long long)b->ld_table);
  if (c->ld_page > (int64_t(1) << 38)) return fail(TP_ERR_UNSUPPORTED, "ld_page above 2^38");
  *empty = T == 0 || b->n_seqs == 0 || b->max_new == 0;
  if (*empty) return TP_OK;
  if (c->k == nullptr || c->v == nullptr || c->k_scales == nullptr || c->v_scales == nullptr)
    return fail(TP_ERR_INVALID_ARG, "k, v, k_scales or v_scales is NULL");
  if (b->seq_start == nullptr || b->kv_len == nullptr || (b->page_table == nullptr && b->max_pages > 0))
    return fail(TP_ERR_INVALID_ARG, "seq_start, kv_len or page_table is NULL");
  if (((reinterpret_cast<uintptr_t>(b->seq_start) | reinterpret_cast<uintptr_t>(b->kv_len) |
        reinterpret_cast<uintptr_t>(b->page_table)) & 3u) != 0)
    return fail(TP_ERR_ALIGNMENT, "seq_start, kv_len and page_table must be 4-byte aligned");
  if (c->ld_page % 16 != 0) return fail(TP_ERR_ALIGNMENT, "ld_page (%lld) must be a multiple of 16", (long long)c->ld_page);
  for (int r = 0; r < c->n_ranks; ++r) {
    if (c->n_pages > 0 && (c->k[r] == nullptr || c->v[r] == nullptr || c->k_scales[r] == nullptr || c->v_scales[r] == nullptr))
      return fail(TP_ERR_INVALID_ARG, "rank %d's codes or scales are NULL", r);
    if (!aligned16(c->k[r]) || !aligned16(c->v[r]))
      return fail(TP_ERR_ALIGNMENT, "rank %d's codes are not 16-byte aligned", r);
  }
  return TP_OK;
}

BatchView batch_view(const tp_paged_cache& c, const tp_paged_batch& b, int64_t T, unsigned int* status) {
  BatchView v{};
  v.seq_start = b.seq_start;
  v.kv_len = b.kv_len;
  v.page_table = b.page_table;
  v.ld_table = b.ld_table != 0 ? b.ld_table : b.max_pages;
  v.n_seqs = b.n_seqs;
  v.max_new = b.max_new;
  v.T = static_cast<int>(T);
  v.max_keys = static_cast<int>(b.max_pages * c.page_size);
  v.n_pages = static_cast<int>(c.n_pages);
  v.page_size = c.page_size;
  v.page_shift = __builtin_ctz(static_cast<unsigned>(c.page_size));
  v.status = status;
  return v;
}

}  // namespace tp

extern "C" {

tp_status tp_kv_append_fp8(const tp_paged_cache* cache, const tp_paged_batch* batch, const void* const* qkv,
                           int64_t ld_qkv, int64_t T, int n_heads, const tp_rope* rope, void* const* q_out,
                           int64_t ld_q, tp_stream_t stream) {
  using namespace tp;
  return guarded([&]() -> tp_status {
    clear_error();
    bool empty = false;
    const tp_status st = check_paged(cache, batch, T, n_heads, &empty);
    if (st != TP_OK) return st;
    const tp_paged_cache& c = *cache;
    const int64_t wide = static_cast<int64_t>(n_heads) * c.head_dim;
    const int64_t row = wide + 2ll * c.n_kv_heads * c.head_dim;
    if ((ld_qkv != 0 && ld_qkv < row) || (ld_q != 0 && ld_q < wide))
      return fail(TP_ERR_INVALID_ARG, "a row stride (ld_qkv %lld, ld_q %lld) is smaller than its row", (long long)ld_qkv,
                  (long long)ld_q);
    if (rope != nullptr) {
      if (rope->style != TP_ROPE_HALF && rope->style != TP_ROPE_PAIRS)
        return fail(TP_ERR_INVALID_ARG, "unknown rotation style %d", static_cast<int>(rope->style));
      if (rope->rot_dim < 16 || rope->rot_dim > c.head_dim || rope->rot_dim % 16 != 0)
        return fail(TP_ERR_INVALID_ARG, "rot_dim must be a multiple of 16 up to head_dim %d, got %d", c.head_dim,
                    rope->rot_dim);
      if (rope->n_positions < 0 || (rope->ld != 0 && rope->ld < rope->rot_dim))
        return fail(TP_ERR_INVALID_ARG, "n_positions %lld, row stride %lld of a table of %d", (long long)rope->n_positions,
                    (long long)rope->ld, rope->rot_dim);
    }
    if (empty) return TP_OK;
    if (qkv == nullptr) return fail(TP_ERR_INVALID_ARG, "qkv is NULL");
    if (ld_qkv % 8 != 0 || ld_q % 8 != 0)
      return fail(TP_ERR_ALIGNMENT, "ld_qkv (%lld) and ld_q (%lld) must be multiples of 8", (long long)ld_qkv,
                  (long long)ld_q);
    if (rope != nullptr) {
      if (rope->cos_sin == nullptr && rope->n_positions > 0) return fail(TP_ERR_INVALID_ARG, "cos_sin is NULL");
      if (!aligned16(rope->cos_sin) || rope->ld % 4 != 0 || (reinterpret_cast<uintptr_t>(rope->positions) & 3u) != 0)
        return fail(TP_ERR_ALIGNMENT, "cos_sin is not 16-byte aligned, its row stride %lld no multiple of 4, or "
                    "positions not 4-byte aligned", (long long)rope->ld);
    }
    AppendParams p{};
    for (int r = 0; r < c.n_ranks; ++r) {
      if (qkv[r] == nullptr || (q_out != nullptr && n_heads > 0 && q_out[r] == nullptr))
        return fail(TP_ERR_INVALID_ARG, "qkv[%d] or q_out[%d] is NULL", r, r);
      if (!aligned16(qkv[r]) || (q_out != nullptr && !aligned16(q_out[r])))
        return fail(TP_ERR_ALIGNMENT, "qkv[%d] or q_out[%d] is not 16-byte aligned", r, r);
      p.qkv[r] = static_cast<const __nv_bfloat16*>(qkv[r]);
      p.q_out[r] = q_out != nullptr ? static_cast<__nv_bfloat16*>(q_out[r]) : nullptr;
      p.k[r] = static_cast<uint8_t*>(c.k[r]);
      p.v[r] = static_cast<uint8_t*>(c.v[r]);
      p.ks[r] = static_cast<uint8_t*>(c.k_scales[r]);
      p.vs[r] = static_cast<uint8_t*>(c.v_scales[r]);
    }
    unsigned int* status = status_word();
    if (status == nullptr) return fail(TP_ERR_CUDA, "cannot locate the kernel status word");
    p.b = batch_view(c, *batch, T, status);
    p.ld_qkv = ld_qkv != 0 ? ld_qkv : row;
    p.ld_q = ld_q != 0 ? ld_q : wide;
    p.ld_page = c.ld_page != 0 ? c.ld_page : static_cast<int64_t>(c.n_kv_heads) * c.page_size * c.head_dim;
    p.ld_scales = c.ld_scales != 0 ? c.ld_scales : c.n_kv_heads;
    if (rope != nullptr) {
      p.cos_sin = rope->cos_sin;
      p.positions = rope->positions;
      p.ld_rope = rope->ld != 0 ? rope->ld : rope->rot_dim;
      p.n_positions = rope->n_positions;
      p.style = rope->style;
      p.rot = rope->rot_dim;
    }
    p.n_heads = n_heads;
    p.n_kv = c.n_kv_heads;
    const int per_unit = kQRounds * 32 / (c.head_dim / 16);   // heads of one warp
    p.q_units = (n_heads + per_unit - 1) / per_unit;
    const int64_t q_blocks = q_out != nullptr ? (T * p.q_units + kWarps - 1) / kWarps : 0;
    // Pages of sequence s get the slots from seq_start[s] / page_size + 2 s on: n new tokens from any
    // position touch at most (n - 1) / page_size + 2 pages.  One new token touches one.
    const bool single = batch->max_new == 1;
    p.slot_per = single ? 0x7FFFFFFF : c.page_size;
    p.slot_gap = single ? 1 : 2;
    const int64_t slots = T / p.slot_per + static_cast<int64_t>(p.slot_gap) * batch->n_seqs;
    p.kv_units = slots * 2 * c.n_kv_heads;
    const int units_per_block = kWarps / (c.page_size / 16);
    const int64_t kv_blocks = (p.kv_units + units_per_block - 1) / units_per_block;
    if (q_blocks + kv_blocks > 0x7FFFFFFF) return fail(TP_ERR_UNSUPPORTED, "too many tokens and heads for one launch");
    p.q_blocks = static_cast<int>(q_blocks);
    const cudaError_t e =
        launch_pdl(c.head_dim == 128 ? kv_append_kernel<128> : kv_append_kernel<64>,
                   dim3(static_cast<unsigned>(q_blocks + kv_blocks), static_cast<unsigned>(c.n_ranks)), dim3(kThreads), 0,
                   reinterpret_cast<cudaStream_t>(stream), p);
    if (e != cudaSuccess) return cuda_fail(e, "cache append launch");
    return TP_OK;
  });
}

}  // extern "C"
