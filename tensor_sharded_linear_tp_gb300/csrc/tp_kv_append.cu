// Appending keys and values to the paged 8-bit cache, with the position rotation of Q and K.
//
// One launch over every rank.  Its first blocks each quantise the new tokens of one page for
// 128 / P of all ranks' KV heads, since a page's tokens share a head's scale:
//     e = max(e_old if the page holds older tokens, least e with max|x| <= 448 * 2^e)
// A warp holds 16 tokens of a page and head in registers, a page of P tokens is held by P / 16 warps, and
// the maximum is joined by one warp reduction and, for larger pages, through shared memory: every
// element is read once and written once.  Only where e grew are the older
// tokens' codes read and written again, scaled by 2^(e_old - e): exact but for codes that fall
// among the subnormal ones, since scales are powers of two.  The other blocks rotate Q (a warp takes one
// token and up to four times 32 lanes' worth of its heads).
//
// What bounds it: the bytes (Q, K and V read once as bf16, Q written, K and V as bytes), and close behind them the
// instructions: 14 an element of K and V.  A prompt of 4608 tokens, 4 ranks of 12 heads and 12 KV heads of 128
// (283 MB) takes 66 us, 0.64 of the copy rate (the pages' part 58 us alone, Q's 21; a warp loads its 16 tokens, waits, and needs
// their maximum before it can write: three CTAs an SM hide part of that).  Small calls are a launch: one token of 4
// ranks 3.1 us, a batch of 61 3.5 us, 7 chunks of odd lengths (21 MB) 8.6 us, against 3.1 of their bytes.
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
  int n_ranks, n_heads, n_kv;
  int first_head;              // one token a sequence: 0, or n_heads where Q is left alone
  int q_units, q_blocks;       // units of kQRounds rounds of heads a token and rank; blocks of the Q part
  int kv_groups;               // blocks of a page's K (and as many of its V)
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

// Pairs of fp32 values for the two-wide instructions (half the instructions: this kernel would issue them
// longer than it moves its bytes).
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
// The larger magnitude of three, NaN if any is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A thread's elements in fp32: pair i of chunk 0, then of chunk 1.
struct Values {
  uint64_t x[8];
};
__device__ __forceinline__ void unpack(Values& v, const uint4 (&raw)[2]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v.x[4 * c + i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
}

// The cosines and sines of a token's two chunks, from its row of the table: for TP_ROPE_HALF those of the
// elements of either chunk, for TP_ROPE_PAIRS of the first chunk's pairs, then of the second's.
struct Turn {
  uint64_t c[4], s[4];
};
__device__ __forceinline__ void load4(uint64_t* dst, const float* src) {
  const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(src);
  dst[0] = v.x, dst[1] = v.y;
}
__device__ __forceinline__ void turn_of(Turn& t, const float* row, int style, int rot, const Chunks& ch) {
  const int i = style == TP_ROPE_HALF ? 8 * ch.c0 : 4 * ch.c0, j = style == TP_ROPE_HALF ? 8 * ch.c0 + 4 : 4 * ch.c1;
  load4(t.c, row + i);
  load4(t.c + 2, row + j);
  load4(t.s, row + rot / 2 + i);
  load4(t.s + 2, row + rot / 2 + j);
}
// NaN where the row is outside the table.
__device__ __forceinline__ void load_turn(Turn& t, const AppendParams& p, int64_t at, const Chunks& ch) {
  if (at >= 0 && at < p.n_positions) {
    turn_of(t, p.cos_sin + at * p.ld_rope, p.style, p.rot, ch);
    return;
  }
  bad_index(p.b);
#pragma unroll
  for (int i = 0; i < 4; ++i) t.c[i] = t.s[i] = 0x7FFFFFFF7FFFFFFFull;
}
// (x1 c - x2 s, x2 c + x1 s) of each pair.
__device__ __forceinline__ void rotate(Values& v, const Turn& t, int style) {
  if (style == TP_ROPE_HALF) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t a = v.x[i], b = v.x[4 + i];
      v.x[i] = fma2(b, t.s[i] ^ 0x8000000080000000ull, mul2(a, t.c[i]));
      v.x[4 + i] = fma2(a, t.s[i], mul2(b, t.c[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 c = split2(t.c[i]), s = split2(t.s[i]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 x = split2(v.x[2 * i + k]);
        const float ck = k == 0 ? c.x : c.y, sk = k == 0 ? s.x : s.y;
        v.x[2 * i + k] = f2(fmaf(-x.y, sk, x.x * ck), fmaf(x.x, sk, x.y * ck));
      }
    }
  }
}
__device__ __forceinline__ uint4 pack_bf16x8(const uint64_t* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = split2(x[i]);
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint2 pack_e4m3x8(const uint64_t* x, uint64_t by) {
  float2 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = split2(mul2(x[i], by));
  return make_uint2(e4m3x4(v[0].x, v[0].y, v[1].x, v[1].y), e4m3x4(v[2].x, v[2].y, v[3].x, v[3].y));
}
// Bits of the largest magnitude as fp32 (a NaN's are the largest).
__device__ __forceinline__ uint32_t amax_bits(const Values& v) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = split2(v.x[i]);
    top = max_abs3(top, x.x, x.y);
  }
  return __float_as_uint(top) & 0x7FFFFFFFu;
}
__device__ __forceinline__ uint32_t amax_bits(const uint4 (&raw)[2]) {
  const uint32_t m = 0x7FFF7FFFu;
  uint32_t v = 0;
#pragma unroll
  for (int c = 0; c < 2; ++c)
    v = __vmaxu2(v, __vmaxu2(__vmaxu2(raw[c].x & m, raw[c].y & m), __vmaxu2(raw[c].z & m, raw[c].w & m)));
  return max(v & 0xFFFFu, v >> 16) << 16;
}

// Q of one token: kQRounds rounds of 32 / kParts heads, a head held by kParts = D / 16 threads.
template <int D>
__device__ __forceinline__ void rotate_q(const AppendParams& p, int64_t unit, int lane) {
  constexpr int kParts = D / 16, kHeads = 32 / kParts;
  const int per_token = p.q_units * p.n_ranks;
  if (unit >= static_cast<int64_t>(p.b.T) * per_token) return;
  const int t = static_cast<int>(unit / per_token), rest = static_cast<int>(unit - static_cast<int64_t>(t) * per_token);
  const int rank = rest / p.q_units, h0 = (rest - rank * p.q_units) * kQRounds * kHeads + lane / kParts;
  const Chunks ch = chunks_of(lane % kParts, p.rot);
  // Rows outside every sequence (padding) are not read.  (The row's loads wait for this and for find_sequence, which
  // ask at once, but not for seq_view: a token 3.1 us so, 3.4 behind seq_view.)
  const int begin = p.b.seq_start[0], end = p.b.seq_start[p.b.n_seqs];
  const int s = find_sequence(p.b, t, 1, 0, lane);
  if (t < begin || t >= end || s < 0) return;
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
        Values x;
        unpack(x, raw[i]);
        rotate(x, turn, p.style);
        raw[i][0] = pack_bf16x8(x.x);
        raw[i][1] = pack_bf16x8(x.x + 4);
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

// The rotation's rows for a page's tokens, where several heads of a block use them (a larger page has fewer in one).
constexpr int kTablePages = 32;                  // tokens of the largest page that has them in shared memory
struct alignas(16) Shared {
  float cs[kTablePages][128];
  uint32_t warp_top[kWarps];
};

template <int D>
__device__ __forceinline__ void append_page(const AppendParams& p, int64_t block, Shared& sh) {
  constexpr int kParts = D / 16, kTokens = 32 / kParts, kRounds = 16 / kTokens;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int P = p.b.page_size, warps = P / 16, heads = kWarps / warps;     // warps of a page and head, heads of a block
  const int64_t slot = block / (2 * p.kv_groups);
  const int rest = static_cast<int>(block - slot * (2 * p.kv_groups));
  const bool is_v = rest >= p.kv_groups;
  const int h = (is_v ? rest - p.kv_groups : rest) * heads + warp / warps;  // of all ranks'
  const bool mine = h < p.n_ranks * p.n_kv;
  const int rank = mine ? h / p.n_kv : 0, head = mine ? h - rank * p.n_kv : 0;

  // Which tokens [j0, j1) of which sequence, in which page (the same for the whole block).
  int j0 = 0, j1 = 0, row0 = 0;                    // the row of position j is row0 + j
  int64_t page = -1;
  const int s = find_sequence(p.b, slot, p.slot_per, p.slot_gap, lane);
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
    }
  }
  if (page < 0) return;

  // This warp's 16 slots: the new values as they are.
  const int base = (j0 & ~(P - 1)) + 16 * (warp % warps);
  const int rot = is_v ? 0 : p.rot;
  const Chunks ch = chunks_of(lane % kParts, rot);
  const __nv_bfloat16* src = p.qkv[rank] + (p.n_heads + (is_v ? p.n_kv : 0) + head) * static_cast<int64_t>(D);
  uint4 raw[kRounds][2];
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int j = base + i * kTokens + lane / kParts;
    raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
    if (mine && j >= j0 && j < j1) {
      const uint4* at = reinterpret_cast<const uint4*>(src + (static_cast<int64_t>(row0) + j) * p.ld_qkv);
      raw[i][0] = at[ch.c0];
      raw[i][1] = at[ch.c1];
    }
  }
  uint8_t* scale = (is_v ? p.vs : p.ks)[rank] + page * p.ld_scales + head;
  const bool older = mine && (j0 & (P - 1)) != 0;
  const uint32_t old_byte = older ? *scale : 0u;
  const bool shared_table = rot > 0 && P <= kTablePages;
  if (shared_table) {
    const int first = j0 & ~(P - 1), quads = rot / 4;
    for (int i = threadIdx.x; i < (j1 - j0) * quads; i += kThreads) {
      const int j = j0 + i / quads, c = i % quads;
      const int64_t at = p.positions != nullptr ? p.positions[row0 + j] : j;
      float4 v = make_float4(NAN, NAN, NAN, NAN);
      if (at >= 0 && at < p.n_positions) v = *reinterpret_cast<const float4*>(p.cos_sin + at * p.ld_rope + 4 * c);
      else bad_index(p.b);
      *reinterpret_cast<float4*>(&sh.cs[j - first][4 * c]) = v;
    }
    __syncthreads();
  }
  // Round i's values, rotated.  (Computed twice, for the maximum and for the codes: kept, they would take
  // half the warps' registers.)
  auto turned = [&](int i, Values& x) {
    const int j = base + i * kTokens + lane / kParts;
    unpack(x, raw[i]);
    if (j >= j0 && j < j1) {
      Turn t;
      if (shared_table) {
        turn_of(t, sh.cs[j & (P - 1)], p.style, p.rot, ch);
      } else {
        const int64_t row = static_cast<int64_t>(row0) + j;
        load_turn(t, p, p.positions != nullptr ? p.positions[row] : j, ch);
      }
      rotate(x, t, p.style);
    }
  };
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    if (ch.turned) {
      Values x;
      turned(i, x);
      top = max(top, amax_bits(x));
    } else {
      top = max(top, amax_bits(raw[i]));
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (warps > 1) {
    if (lane == 0) sh.warp_top[warp] = top;
    __syncthreads();
    for (int w = warp / warps * warps, i = 0; i < warps; ++i) top = max(top, sh.warp_top[w + i]);
  }
  if (!mine) return;
  const uint32_t byte = max(old_byte, top == 0u ? 0u : e8m0_of_amax(top));
  uint8_t* codes = (is_v ? p.v : p.k)[rank] + page * p.ld_page + static_cast<int64_t>(head) * P * D;
  __syncwarp();      // (every lane has the old scale)
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
#pragma unroll
    for (int c = 0; c < 2; ++c)      // (so that the compiler computes them again)
      asm volatile("" : "+r"(raw[i][c].x), "+r"(raw[i][c].y), "+r"(raw[i][c].z), "+r"(raw[i][c].w) : : "memory");
    const int j = base + i * kTokens + lane / kParts;
    if (j >= j0 && j < j1) {
      uint2* to = reinterpret_cast<uint2*>(codes + (j & (P - 1)) * D);
      Values x;
      if (ch.turned) turned(i, x);
      else unpack(x, raw[i]);
      to[ch.c0] = pack_e4m3x8(x.x, f2(inv, inv));
      to[ch.c1] = pack_e4m3x8(x.x + 4, f2(inv, inv));
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 3) kv_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ Shared sh;
  pdl_launch_dependents();
  pdl_wait();
  // The pages first: their blocks take longest, and Q's fill the SMs that they leave.  (Prompt of 4608 tokens: 67 us,
  // Q first 76, evenly mixed 75.)
  const int pages = static_cast<int>(gridDim.x) - p.q_blocks, block = static_cast<int>(blockIdx.x);
  if (block < pages)
    append_page<D>(p, block, sh);
  else
    rotate_q<D>(p, static_cast<int64_t>(block - pages) * kWarps + (threadIdx.x >> 5), threadIdx.x & 31);
}

// One new token a sequence at most (decoding; 61 sequences 3.5 us, 6.7 by the kernel above, whose blocks are for 16
// tokens and more): a warp takes kTokenRounds rounds of a token's heads, Q's,
// K's and V's alike, a head held by kParts threads.  No page is shared by two tokens here, so no block has
// to meet.
constexpr int kTokenWarps = 2, kTokenRounds = 2;
template <int D>
__global__ void __launch_bounds__(kTokenWarps * 32) kv_append_token_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kParts = D / 16, kHeads = 32 / kParts;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kTokenWarps + (threadIdx.x >> 5);
  const int per_token = p.q_units * p.n_ranks;
  if (unit >= static_cast<int64_t>(p.b.T) * per_token) return;
  const int t = static_cast<int>(unit / per_token), rest = static_cast<int>(unit - static_cast<int64_t>(t) * per_token);
  const int rank = rest / p.q_units, h0 = p.first_head + (rest - rank * p.q_units) * kTokenRounds * kHeads + lane / kParts;
  const Chunks ch = chunks_of(lane % kParts, p.rot);
  const int begin = p.b.seq_start[0], end = p.b.seq_start[p.b.n_seqs];
  const int s = find_sequence(p.b, t, 1, 0, lane);
  if (t < begin || t >= end || s < 0) return;
  const __nv_bfloat16* src = p.qkv[rank] + t * p.ld_qkv;
  const int n_all = p.n_heads + 2 * p.n_kv;
  uint4 raw[kTokenRounds][2];
#pragma unroll
  for (int i = 0; i < kTokenRounds; ++i) {
    const int h = h0 + i * kHeads;
    raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
    if (h < n_all) {
      raw[i][0] = *reinterpret_cast<const uint4*>(src + h * D + 8 * ch.c0);
      raw[i][1] = *reinterpret_cast<const uint4*>(src + h * D + 8 * ch.c1);
    }
  }
  const SeqView v = seq_view(p.b, s);
  if (t - v.a >= v.n) return;            // rows of no sequence are left alone
  const int pos = v.pos0;
  Turn turn;
  if (ch.turned) load_turn(turn, p, p.positions != nullptr ? p.positions[t] : pos, ch);
  int64_t page = -1;
  if (pos >= 0 && pos < p.b.max_keys) page = p.b.page_table[s * p.b.ld_table + (pos >> p.b.page_shift)];
  if (page < 0 || page >= p.b.n_pages) {
    if (lane == 0) bad_index(p.b);
    page = -1;
  }
  const int slot = pos & (p.b.page_size - 1);
  uint8_t* scale[kTokenRounds];
  uint32_t old_byte[kTokenRounds];
#pragma unroll
  for (int i = 0; i < kTokenRounds; ++i) {
    const int g = h0 + i * kHeads - p.n_heads;          // K's heads, then V's
    scale[i] = nullptr;
    old_byte[i] = 0;
    if (g >= 0 && g < 2 * p.n_kv && page >= 0) {
      scale[i] = g < p.n_kv ? p.ks[rank] + page * p.ld_scales + g : p.vs[rank] + page * p.ld_scales + (g - p.n_kv);
      if (slot > 0) old_byte[i] = *scale[i];
    }
  }
#pragma unroll
  for (int i = 0; i < kTokenRounds; ++i) {
    const int h = h0 + i * kHeads, g = h - p.n_heads;
    Values x;
    unpack(x, raw[i]);
    if (ch.turned && g < p.n_kv) rotate(x, turn, p.style);
    // (V is not rotated, but its threads hold the chunks of a rotated head: any will do)
    uint32_t top = amax_bits(x);
#pragma unroll
    for (int d = 1; d < kParts; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    const uint32_t byte = max(old_byte[i], top == 0u ? 0u : e8m0_of_amax(top));
    uint8_t* codes = nullptr;
    if (scale[i] != nullptr)
      codes = g < p.n_kv ? p.k[rank] + page * p.ld_page + static_cast<int64_t>(g) * p.b.page_size * D
                         : p.v[rank] + page * p.ld_page + static_cast<int64_t>(g - p.n_kv) * p.b.page_size * D;
    // Older tokens' codes at a larger scale, by the whole warp, one head after the other.
    const bool grew = codes != nullptr && slot > 0 && byte > old_byte[i];
    for (uint32_t m = __ballot_sync(0xffffffffu, grew && lane % kParts == 0); m != 0; m &= m - 1) {
      const int from = __ffs(m) - 1;
      const uint32_t nb = __shfl_sync(0xffffffffu, byte, from), ob = __shfl_sync(0xffffffffu, old_byte[i], from);
      uint4* at = reinterpret_cast<uint4*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(codes), from));
      const float f = nb == 255u ? __uint_as_float(0x7FFFFFFFu) : nb - ob > 126u ? 0.0f : __uint_as_float((127u - (nb - ob)) << 23);
#pragma unroll 4
      for (int j = lane; j < slot * (D / 16); j += 32) {
        const uint4 w = at[j];
        at[j] = make_uint4(rescale4(w.x, f), rescale4(w.y, f), rescale4(w.z, f), rescale4(w.w, f));
      }
    }
    if (codes != nullptr) {
      const float inv = e8m0_inverse(byte);
      uint2* to = reinterpret_cast<uint2*>(codes + slot * D);
      to[ch.c0] = pack_e4m3x8(x.x, f2(inv, inv));
      to[ch.c1] = pack_e4m3x8(x.x + 4, f2(inv, inv));
      if (lane % kParts == 0) *scale[i] = static_cast<uint8_t>(byte);
    } else if (g < 0) {
      __nv_bfloat16* dst = p.q_out[rank] + t * p.ld_q + h * D;
      *reinterpret_cast<uint4*>(dst + 8 * ch.c0) = ch.turned ? pack_bf16x8(x.x) : raw[i][0];
      *reinterpret_cast<uint4*>(dst + 8 * ch.c1) = ch.turned ? pack_bf16x8(x.x + 4) : raw[i][1];
    }
  }
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
    p.n_ranks = c.n_ranks;
    p.n_heads = n_heads;
    p.n_kv = c.n_kv_heads;
    cudaError_t e;
    if (batch->max_new == 1) {
      p.first_head = q_out != nullptr ? 0 : n_heads;
      const int heads = n_heads + 2 * c.n_kv_heads - p.first_head, per_warp = kTokenRounds * 32 / (c.head_dim / 16);
      p.q_units = (heads + per_warp - 1) / per_warp;
      const int64_t blocks = (T * p.q_units * c.n_ranks + kTokenWarps - 1) / kTokenWarps;
      if (blocks > 0x7FFFFFFF) return fail(TP_ERR_UNSUPPORTED, "too many tokens and heads for one launch");
      e = launch_pdl(c.head_dim == 128 ? kv_append_token_kernel<128> : kv_append_token_kernel<64>, dim3(static_cast<unsigned>(blocks)),
                     dim3(kTokenWarps * 32), 0, reinterpret_cast<cudaStream_t>(stream), p);
    } else {
      const int per_unit = kQRounds * 32 / (c.head_dim / 16);   // heads of one warp
      p.q_units = (n_heads + per_unit - 1) / per_unit;
      const int64_t q_blocks = q_out != nullptr ? (T * p.q_units * c.n_ranks + kWarps - 1) / kWarps : 0;
      // Pages of sequence s get the slots from seq_start[s] / page_size + 2 s on: n new tokens from any
      // position touch at most (n - 1) / page_size + 2 pages.
      p.slot_per = c.page_size;
      p.slot_gap = 2;
      const int64_t slots = T / p.slot_per + static_cast<int64_t>(p.slot_gap) * batch->n_seqs;
      const int heads = kWarps / (c.page_size / 16);            // of a block
      p.kv_groups = (c.n_ranks * c.n_kv_heads + heads - 1) / heads;
      const int64_t kv_blocks = slots * 2 * p.kv_groups;
      if (q_blocks + kv_blocks > 0x7FFFFFFF) return fail(TP_ERR_UNSUPPORTED, "too many tokens and heads for one launch");
      p.q_blocks = static_cast<int>(q_blocks);
      e = launch_pdl(c.head_dim == 128 ? kv_append_kernel<128> : kv_append_kernel<64>,
                     dim3(static_cast<unsigned>(q_blocks + kv_blocks)), dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream), p);
    }
    if (e != cudaSuccess) return cuda_fail(e, "cache append launch");
    return TP_OK;
  });
}

}  // extern "C"
