// Attention over the paged 8-bit cache (tp_paged.h, include/tp.h): few rows a KV head.
//
//     S = scale Q K^T,  O = softmax(S) V      one item = the rows of one sequence, KV head and rank
//
// What bounds it: the cache's bytes.  With R rows (new tokens x query heads of the KV head) a key
// costs 2 D bytes and 4 D R FLOP; at R <= 32 that is at most 64 FLOP a byte, a quarter of what the GPU
// has, so the keys and values stream through the SMs once and everything else has to keep out of
// their way.  Measured: 64 sequences of 50 to 8000 tokens, 8 KV heads of 6 query heads (569 MB) in 116 us, 0.72 of the
// copy rate (queueing and prologues take some 10 us, the last CTAs 10, the join 6); one sequence of 131000
// tokens 59 us, 0.67.  From 17 rows on it is the warps' own latency that bounds (eight of them an SM):
// 16 sequences 57 us with 12 rows, 67 with 18, 90 with 30, where the bytes take 24.
//
// * All keys of all items are one line of steps of 32 keys, cut into equal parts for the CTAs, and each
//   of them into equal parts for its warps.  Sequences of any lengths load the GPU evenly,
//   from a batch of short ones to one long one.  An item that lies in one warp is finished by it;
//   pieces of an item in several warps are joined in shared memory, pieces in several CTAs through the
//   workspace by a second launch, always in key order (no atomics).
// * A warp has a ring of steps of its own in shared memory, filled by its own asynchronous copies (swizzled so
//   that the loads below meet no bank twice; TMA's boxes of a page each took its issuing lane 700 to 1400
//   cycles a step: 128 us for the 64 sequences, not 116) and drained by itself: no barrier between warps.  What
//   bounds a warp is the latency of its own instructions (some 1700 cycles a step at 8 rows), so an SM has as
//   many as their registers and rings allow.
// * The products are S^T = K Q^T and O^T = V^T P^T on mma.sync m16n8k16 (keys, then head elements,
//   on M; rows on N), since so few rows would leave most of a tcgen05 tile's 128 empty.  K's
//   fragments are 32-bit words of the cache, converted two codes an instruction to fp16 (exact); V's need two
//   keys side by side, a byte permutation first; P^T's come from S^T's by a transposing move.
// * Scales stay out of the fragments: K's multiplies a score, V's the probability.
// * Up to 32 rows, 8 on N at a time, and a kernel for each 8 more (make_plan).
//
// Q enters as fp16 as well, each row scaled by a power of two to below 2^15, so that what it loses
// lies 2^-39 below its largest element; its factor goes into the scores.  P is 2^(s - m) (m the running maximum)
// times 2^(e - E + 14), e the exponent of the key's V page and E the largest so far: at most 2^14, so
// that fp16 keeps what is up to 2^-38 below the largest.  O is kept in units of 2^(E - 14).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "tp_internal.h"
#include "tp_paged_attention.cuh"
#include "tp_ptx.cuh"

namespace tp {
namespace {

constexpr int kStep = 32;                         // keys of a step
constexpr int kCtasPerSm = 2;
constexpr int kMaxSteps = kLongestPiece / kStep;  // of a piece

// A piece of an item in shared memory.
struct Piece {
  int64_t item_end;     // the step behind the item's last
  int valid, first, last;
  int early;            // in the workspace, since the warp went on to the next item; else in its (drained) ring
  int s, h, a, rows;
};
struct Start {          // where a warp's part begins
  int s, h, tile;
  int64_t at;           // its first step
};
// An item: the rows of a sequence (n new tokens x group) and KV head h of all ranks', and its steps.
struct RowsItem {
  int s, h, a, len, pos0;
  int rows, tile0, tiles, key_end;
};
template <int WARPS, int STAGES>
struct alignas(16) Ctrl {
  static constexpr int ITEMS = STAGES < 4 ? 4 : 8;   // more than are in the ring of steps at once
  uint32_t info[WARPS][STAGES][2];   // scale bytes of a step's two halves (load_pages)
  RowsItem item[WARPS][ITEMS];
  Piece piece[WARPS][2];
  Start start[WARPS];
  int64_t sums[WARPS];
};
__device__ __forceinline__ RowsItem rows_item(const AttendParams& p, int s, int h, const SeqView& v) {
  RowsItem it;
  it.s = s, it.h = h, it.a = v.a, it.len = v.len, it.pos0 = v.pos0;
  it.rows = v.n * p.group;
  const int64_t end = static_cast<int64_t>(v.pos0) + v.n;     // behind the last row's position
  it.key_end = p.causal ? static_cast<int>(max(min(static_cast<int64_t>(v.len), end), int64_t(0))) : v.len;
  const int lo = p.window > 0 ? max(v.pos0 - p.window + 1, 0) : 0;
  it.tile0 = min(lo, it.key_end) / kStep;
  it.tiles = it.rows > 0 ? max(1, (it.key_end + kStep - 1) / kStep - it.tile0) : 0;   // (a row without keys is an item too)
  return it;
}

template <int D, int NT>
struct Cfg {
  // Two CTAs an SM (kCtasPerSm): 12 warps of 168 registers, or 8 of 255 for more row tiles, whose O alone is
  // 32 registers each at D 128.
  static constexpr int WARPS = NT == 1 ? 6 : 4;
  static constexpr bool Q_SHARED = NT > 2;        // Q's fragments in shared memory, for want of registers
  static constexpr int THREADS = WARPS * 32;
  static constexpr int ROWS = 8 * NT;
  static constexpr uint32_t HALF = kStep * D;     // K's or V's bytes of a step
  static constexpr uint32_t STAGE = 2 * HALF;
  static constexpr int STAGES = (NT == 2 ? 3 : 2) * (128 / D);
  static constexpr uint32_t RING = STAGES * STAGE;                   // of one warp
  static constexpr uint32_t PIECE = ROWS * (D + 2) * 4;              // O, then (m, l) of each row
  static constexpr uint32_t OFF_Q = RING;                            // in a warp's own part
  static constexpr uint32_t OWN = RING + (Q_SHARED ? NT * (D / 16) * 32 * 8 : 0);
  static constexpr uint32_t OFF_CTRL = WARPS * OWN;
  static constexpr size_t SMEM = 1024 + OFF_CTRL + sizeof(Ctrl<WARPS, STAGES>);
  static_assert(PIECE <= OWN && kCtasPerSm * (SMEM + 1024) <= 228 * 1024, "shared memory");
};

// Two codes (the low or high half of a word) as fp16.
__device__ __forceinline__ uint32_t f16_lo(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
  return r;
}
__device__ __forceinline__ uint32_t f16_hi(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w >> 16)));
  return r;
}
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
// A step's data in shared memory: row `key`, 16-byte chunk c, swizzled.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int key, int c) {
  return static_cast<uint32_t>(key * D + ((c ^ (D == 128 ? key & 7 : (key >> 1) & 3)) << 4));
}

constexpr uint32_t kPageSeen = 0x10000;   // in a page's info, above its K and V scale bytes: some row sees it, and its index is valid

// The steps of a warp's part in the order they are loaded, ahead of the one that is worked on.
struct Loader {
  int s, h, rank, head;        // h = rank * n_kv + head
  uint32_t items;              // that it has begun
  int tile, tile_end;          // of the current item
  int page0;                   // the lanes hold pages page0 .. page0 + 31 of the sequence
  int my_page;
  uint32_t my_info;
  int len;                     // the sequence's keys
  const uint8_t *k, *v;        // the rank's codes
};

// 16 bytes into shared memory, or zeros (size 0), by the asynchronous copy of the calling thread.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, uint32_t size) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D>
__device__ __forceinline__ void load_pages(const AttendParams& p, Loader& ld, int first, int lane) {
  ld.page0 = first;
  const int64_t at = static_cast<int64_t>(first) + lane;
  ld.my_info = 0;
  ld.my_page = 0;
  // A page before every row's window may be gone, or another sequence's by now: its codes and scales take no part.
  // (The window's first key is read again here, once for 32 pages: kept by the loader, it would spill.)
  const int lo = p.window > 0 ? seq_view(p.b, ld.s).pos0 - p.window + 1 : 0;
  if ((at << p.b.page_shift) < ld.len && ((at + 1) << p.b.page_shift) > lo) {
    ld.my_page = p.b.page_table[ld.s * p.b.ld_table + at];
    if (ld.my_page >= 0 && ld.my_page < p.b.n_pages) {
      const int64_t sc = static_cast<int64_t>(ld.my_page) * p.ld_scales + ld.head;
      ld.my_info = kPageSeen | p.ks[ld.rank][sc] | (static_cast<uint32_t>(p.vs[ld.rank][sc]) << 8);
    } else {
      bad_index(p.b);
    }
  }
}

template <int D, int NT>
__device__ __forceinline__ void issue_step(const AttendParams& p, Loader& ld, int stage, uint32_t ring, Ctrl<Cfg<D, NT>::WARPS, Cfg<D, NT>::STAGES>* ctl,
                                           int first_tile, int warp, int lane) {
  using C = Cfg<D, NT>;
  if (ld.tile == ld.tile_end) {   // the next item: the next head, or the next sequence's first
    if (++ld.h == p.heads) ld.h = 0, ++ld.s;
    RowsItem it;
    for (;; ++ld.s) {
      it = rows_item(p, ld.s, ld.h, seq_view(p.b, ld.s));
      if (it.tiles > 0 || ld.s + 1 >= p.b.n_seqs) break;
    }
    if (lane == 0) ctl->item[warp][ld.items % Ctrl<C::WARPS, C::STAGES>::ITEMS] = it;
    ld.tile = ld.items == 0 ? first_tile : it.tile0;
    ld.tile_end = it.tile0 + it.tiles;
    ld.len = it.len;
    ld.page0 = -64;
    ld.rank = p.by_kv(ld.h);
    ld.head = ld.h - ld.rank * p.n_kv;
    ld.k = p.k[ld.rank];
    ld.v = p.v[ld.rank];
    ++ld.items;
    // Its rows of Q into L2: they are read when the step before is done.
#pragma unroll 1
    for (int i = lane; i < it.rows * (D / 64); i += 32) {
      const int r = i / (D / 64), token = p.by_group(r);
      const __nv_bfloat16* q = p.q[ld.rank] + static_cast<int64_t>(it.a + token) * p.ld_q +
                               (static_cast<int64_t>(ld.head) * p.group + (r - token * p.group)) * D + (i % (D / 64)) * 64;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
    }
  }
  const int key0 = ld.tile * kStep, page = key0 >> p.b.page_shift;
  const bool two = p.b.page_size == 16;
  if (page < ld.page0 || page + (two ? 1 : 0) >= ld.page0 + 32) load_pages<D>(p, ld, page, lane);
  constexpr int kChunks = D / 16, kKeysAtOnce = 32 / kChunks;   // 16-byte chunks of a key; keys of a copy
  const int chunk = lane % kChunks, row = lane / kChunks;
  const uint32_t dst = ring + stage * C::STAGE;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int src = page - ld.page0 + (two ? i : 0), key = key0 + 16 * i;
    const uint32_t info = __shfl_sync(0xffffffffu, ld.my_info, src);
    const int at = __shfl_sync(0xffffffffu, ld.my_page, src);
    // (A page that is not there, or that no row sees: zeros, nothing is read.)
    const uint32_t size = (info & kPageSeen) != 0 ? 16 : 0;
    const int64_t off = at * p.ld_page + (static_cast<int64_t>(ld.head) * p.b.page_size + (key & (p.b.page_size - 1)) + row) * D + chunk * 16;
    const uint8_t* none = reinterpret_cast<const uint8_t*>(p.q[0]);
    const uint8_t *k = ld.k + off, *v = ld.v + off;
#pragma unroll
    for (int j = 0; j < 16; j += kKeysAtOnce) {
      const uint32_t to = dst + chunk_at<D>(16 * i + j + row, chunk);
      copy16(to, size != 0 ? k + j * D : none, size);
      copy16(to + C::HALF, size != 0 ? v + j * D : none, size);
    }
    if (lane == 0) ctl->info[warp][stage][i] = info;
  }
  ++ld.tile;
}

// What a warp knows of its item: Q's fragments (unless in shared memory), the softmax's state.
template <int D, int NT>
struct State {
  uint32_t q[Cfg<D, NT>::Q_SHARED ? 1 : NT][D / 16][2];
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2], ck[NT][2];   // of the rows 8 nt + 2 t and + 1
  int hi_all, lo_all;                    // every row sees [lo_all, hi_all)
  int e_v;
};

// Q's rows into fragments: row g of tile nt, elements 32 t .. 32 t + 31 (16 at D 64) in the k order
// that K's words give (word j: elements 4 j .. 4 j + 3 of them).
template <int D, int NT>
__device__ __forceinline__ void load_item(const AttendParams& p, const RowsItem& it, State<D, NT>& st, uint32_t q_at, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const int rank = p.by_kv(it.h), head = it.h - rank * p.n_kv;
  constexpr int W = D / 16;
  int hi_all = 0x7FFFFFFF, lo_all = 0;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 8 * nt + g;
    uint4 raw[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) raw[i] = make_uint4(0, 0, 0, 0);
    if (r < it.rows) {
      const int token = p.by_group(r), hq = r - token * p.group;
      const __nv_bfloat16* src = p.q[rank] + static_cast<int64_t>(it.a + token) * p.ld_q +
                                 (static_cast<int64_t>(head) * p.group + hq) * D + t * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) raw[i] = reinterpret_cast<const uint4*>(src)[i];
    }
    const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
    top = max(top & 0xFFFFu, top >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // top < 2^(E - 126), E its exponent field: times 2^(141 - E) the row is below 2^15.  (2^127 at most, which
    // is enough for rows below 2^-112.)  A NaN or an infinity makes the row NaN.
    const int E = static_cast<int>(top >> 7), up = min(141 - E, 127);
    const float f = E == 255 ? 0.0f : pow2(up);
    float back = p.scale_log2e * pow2(-(up / 2)) * pow2(up / 2 - up);
    if (E == 255) back = __uint_as_float(0x7FFFFFFFu);
#pragma unroll
    for (int j = 0; j < W; ++j) {
      uint32_t q[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t v = E == 255 ? 0u : w[2 * j + i];
        q[i] = f16_pair(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xFFFF0000u) * f);
      }
      if constexpr (Cfg<D, NT>::Q_SHARED)
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(q_at + ((j * NT + nt) * 32 + lane) * 8), "r"(q[0]), "r"(q[1]) : "memory");
      else
        st.q[nt][j][0] = q[0], st.q[nt][j][1] = q[1];
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      st.ck[nt][c] = __shfl_sync(0xffffffffu, back, 4 * (2 * t + c));
      st.m[nt][c] = -INFINITY;
      st.l[nt][c] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) st.o[nt][i][c] = 0.0f;
  }
  const int first = it.pos0, last = it.pos0 + p.by_group(max(it.rows, 1) - 1);
  if (p.causal) hi_all = first + 1;
  if (p.window > 0) lo_all = last - p.window + 1;
  st.hi_all = min(hi_all, it.len);
  st.lo_all = lo_all;
  st.e_v = -1000;
}

// One step of 32 keys from shared memory.
template <int D, int NT>
__device__ __forceinline__ void step(const AttendParams& p, const RowsItem& it, State<D, NT>& st, uint32_t data, uint32_t q_at, uint32_t info0, uint32_t info1, int key0,
                                     int lane) {
  using C = Cfg<D, NT>;
  constexpr int W = D / 16;       // words of K a lane has of a key = 16-element steps of the head
  const int g = lane >> 2, t = lane & 3;
  const uint32_t info[2] = {info0, info1};
  const bool partial = key0 < st.lo_all || key0 + kStep > st.hi_all ||
                       (info0 & info1 & kPageSeen) == 0 || (info0 & 0xFFu) == 255u || (info0 & 0xFF00u) == 0xFF00u ||
                       (info1 & 0xFFu) == 255u || (info1 & 0xFF00u) == 0xFF00u;   // (warp-uniform)
  float x[2][NT][4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[mt][nt][c] = 0.0f;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    uint32_t ka[2][4], kb[2][4];    // keys 16 mt + g and + 8, four words of a lane
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const int at = D == 128 ? 2 * t + c : t;
      const uint4 a = lds128(data + chunk_at<D>(16 * mt + g, at)), b = lds128(data + chunk_at<D>(16 * mt + g + 8, at));
      ka[mt][0] = a.x, ka[mt][1] = a.y, ka[mt][2] = a.z, ka[mt][3] = a.w;
      kb[mt][0] = b.x, kb[mt][1] = b.y, kb[mt][2] = b.z, kb[mt][3] = b.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 4 * c + i;
      uint32_t a[2][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) a[mt][0] = f16_lo(ka[mt][i]), a[mt][1] = f16_lo(kb[mt][i]), a[mt][2] = f16_hi(ka[mt][i]), a[mt][3] = f16_hi(kb[mt][i]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint2 q;
        if constexpr (C::Q_SHARED) q = lds64(q_at + ((j * NT + nt) * 32 + lane) * 8);
        else q = make_uint2(st.q[nt][j][0], st.q[nt][j][1]);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) mma(x[mt][nt], a[mt][0], a[mt][1], a[mt][2], a[mt][3], q.x, q.y);
      }
    }
  }
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    // Scores in log2 units.  A page whose K or V is NaN makes its keys' scores NaN (its V enters as 0).
    const float ks = (info[mt] & 0xFF00u) == 0xFF00u ? __uint_as_float(0x7FFFFFFFu) : e8m0_value(info[mt] & 0xFFu);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[mt][nt][c] *= st.ck[nt][c & 1] * ks;
    if (partial) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int row = 8 * nt + 2 * t + c, pos = it.pos0 + p.by_group(row);      // keys [lo, hi) are seen
          const int hi = row < it.rows && (info[mt] & kPageSeen) != 0 ? (p.causal ? min(it.len, pos + 1) : it.len) : 0;
          const int lo = p.window > 0 ? pos - p.window + 1 : 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = key0 + 16 * mt + g + 8 * i;
            if (key >= hi || key < lo) x[mt][nt][c + 2 * i] = -INFINITY;
          }
        }
    }
  }
  // The running maximum of each row, and the largest V exponent.
  bool grew = false;
  float alpha[NT][2], ms[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float mx = fmaxf(fmaxf(x[0][nt][c], x[0][nt][c + 2]), fmaxf(x[1][nt][c], x[1][nt][c + 2]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      const float m_new = fmaxf(st.m[nt][c], mx);
      ms[nt][c] = m_new == -INFINITY ? 0.0f : m_new;
      grew |= m_new > st.m[nt][c];
      alpha[nt][c] = ex2(st.m[nt][c] - ms[nt][c]);
      st.m[nt][c] = m_new;
    }
  int e[2], e_new = st.e_v;
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    const int byte = static_cast<int>((info[mt] >> 8) & 0xFFu);
    e[mt] = byte == 255 || (info[mt] & kPageSeen) == 0 ? -127 : byte - 127;
    e_new = max(e_new, e[mt]);
  }
  if (__any_sync(0xffffffffu, grew) || e_new > st.e_v) {
    const float f = pow2(max(st.e_v - e_new, -127));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        st.l[nt][c] *= alpha[nt][c];
        alpha[nt][c] *= f;
      }
#pragma unroll
      for (int i = 0; i < W; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) st.o[nt][i][c] *= alpha[nt][c & 1];
    }
    st.e_v = e_new;
  }
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    // P^T as the B operand: S^T has a key a lane group, B wants a row a lane group.
    const float f = pow2(e[mt] - e_new + 14);
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float y[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        y[c] = ex2(x[mt][nt][c] - ms[nt][c & 1]);
        st.l[nt][c & 1] += y[c];
      }
      pb[nt][0] = transpose8x8(f16_pair(y[0] * f, y[1] * f));
      pb[nt][1] = transpose8x8(f16_pair(y[2] * f, y[3] * f));
    }
    // V^T: lane (g, t) has elements W g .. of the keys 2 t, 2 t + 1, 2 t + 8 and 2 t + 9.
    constexpr int VW = D / 32;    // words of a key
    uint32_t v[4][VW];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int key = 16 * mt + 2 * t + (k & 1) + 8 * (k >> 1);
      if constexpr (D == 128) {
        const uint4 w = lds128(data + C::HALF + chunk_at<D>(key, g));
        v[k][0] = w.x, v[k][1] = w.y, v[k][2] = w.z, v[k][3] = w.w;
      } else {
        const uint2 w = lds64(data + C::HALF + chunk_at<D>(key, g >> 1) + 8 * (g & 1));
        v[k][0] = w.x, v[k][1] = w.y;
      }
      // What no row sees may hold anything, a NaN times 0 among it.
      if (partial && (key0 + key >= it.key_end || (info[mt] & kPageSeen) == 0 || (info[mt] & 0xFF00u) == 0xFF00u)) {
#pragma unroll
        for (int i = 0; i < VW; ++i) v[k][i] = 0;
      }
    }
#pragma unroll
    for (int i = 0; i < VW; ++i) {
      const uint32_t ab = __byte_perm(v[0][i], v[1][i], 0x5140), cd = __byte_perm(v[2][i], v[3][i], 0x5140);
      const uint32_t ab2 = __byte_perm(v[0][i], v[1][i], 0x7362), cd2 = __byte_perm(v[2][i], v[3][i], 0x7362);
      const uint32_t a0 = f16_lo(ab), a1 = f16_hi(ab), a2 = f16_lo(cd), a3 = f16_hi(cd);
      const uint32_t b0 = f16_lo(ab2), b1 = f16_hi(ab2), b2 = f16_lo(cd2), b3 = f16_hi(cd2);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma(st.o[nt][2 * i], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
        mma(st.o[nt][2 * i + 1], b0, b1, b2, b3, pb[nt][0], pb[nt][1]);
      }
    }
  }
}

// Ends an item's piece: O / l to the output where the piece is the whole item, else to `piece`
// with the rows' m and l.
template <int D, int NT>
__device__ __forceinline__ void end_piece(const AttendParams& p, const RowsItem& it, State<D, NT>& st, bool whole, float* piece, int lane) {
  using C = Cfg<D, NT>;
  const int g = lane >> 2, t = lane & 3;
  const int rank = p.by_kv(it.h), head = it.h - rank * p.n_kv;
  const float fe = e8m0_value(static_cast<uint32_t>(max(st.e_v, -127) + 127));
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float l = st.l[nt][c];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const float inv = l == 0.0f ? 0.0f : 0x1p-14f / l;
      float o[D / 8];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        o[2 * i] = st.o[nt][i][c] * inv * fe;
        o[2 * i + 1] = st.o[nt][i][c + 2] * inv * fe;
      }
      const int row = 8 * nt + 2 * t + c;   // elements D/8 g .. of it
      if (!whole) {
        float* dst = piece + row * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < D / 8; i += 4) *reinterpret_cast<float4*>(dst + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        if (g == 0) *reinterpret_cast<float2*>(piece + C::ROWS * D + 2 * row) = make_float2(st.m[nt][c], l);
      } else if (row < it.rows) {
        const int token = p.by_group(row), hq = row - token * p.group;
        __nv_bfloat16* dst = p.out[rank] + static_cast<int64_t>(it.a + token) * p.ldo +
                             (static_cast<int64_t>(head) * p.group + hq) * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < D / 8; i += 8)
          reinterpret_cast<uint4*>(dst)[i / 8] = make_uint4(pack_bf16(o[i], o[i + 1]), pack_bf16(o[i + 2], o[i + 3]),
                                                            pack_bf16(o[i + 4], o[i + 5]), pack_bf16(o[i + 6], o[i + 7]));
      }
    }
}

// Joins two pieces of an item, the second of which continues the first: to the output where `to` is NULL, else to `to`, which may be
// the first.  (A small rolled loop: only items of more than kMaxSteps steps in a warp come here.)  Warp-collective.
template <int D, int NT>
__device__ __forceinline__ void join_two(const AttendParams& p, const RowsItem& it, const float* a, const float* b, float* to, int lane) {
  using C = Cfg<D, NT>;
  auto ml = [&](const float* piece, int row) { return *reinterpret_cast<const float2*>(piece + C::ROWS * D + 2 * row); };
  __syncwarp();
#pragma unroll 1
  for (int i = lane * 4; i < C::ROWS * D; i += 128) {
    const int row = i / D;
    const Joined j = join_pieces(0, 1, 2, [&](int k) { return ml(k == 0 ? a : b, row); },
                                 [&](int k) { return *reinterpret_cast<const float4*>((k == 0 ? a : b) + i); });
    const float inv = j.l == 0.0f ? 0.0f : 1.0f / j.l;
    const float4 o = make_float4(j.o.x * inv, j.o.y * inv, j.o.z * inv, j.o.w * inv);
    if (to != nullptr) *reinterpret_cast<float4*>(to + i) = o;
    else if (row < it.rows) store_row4(p, it.a, it.h, row, i - row * D, D, o);
  }
  __syncwarp();
  if (to != nullptr && lane < C::ROWS) {
    const float2 x = ml(a, lane), y = ml(b, lane);
    const float m = fmaxf(x.x, y.x), ref = m == -INFINITY ? 0.0f : m;
    *reinterpret_cast<float2*>(to + C::ROWS * D + 2 * lane) = make_float2(m, x.y * ex2(x.x - ref) + y.y * ex2(y.x - ref));
  }
  __syncwarp();
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::THREADS, kCtasPerSm) paged_rows_kernel(const __grid_constant__ AttendParams p) {
  using C = Cfg<D, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto* ctl = reinterpret_cast<Ctrl<C::WARPS, C::STAGES>*>(base + C::OFF_CTRL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = ptx::smem_addr(base) + warp * C::OWN, q_at = ring + C::OFF_Q;
  pdl_launch_dependents();
  if (lane == 0) ctl->piece[warp][0].valid = ctl->piece[warp][1].valid = 0;
  __syncwarp();
  pdl_wait();

  // This CTA's steps [u0, u1) of `total`, and the item and step at which this warp's part begins.
  int64_t u0 = 0, u1 = 0, total = 0, n_cta = 1;
  Start my{0, 0, 0, 0};
  int count = 0;
  if (p.per_item) {
    my.s = blockIdx.x;
    my.h = blockIdx.y;
    const RowsItem it = rows_item(p, my.s, my.h, seq_view(p.b, my.s));
    u1 = total = it.tiles;
    const int from = it.tiles * warp / C::WARPS;
    my.at = from;
    my.tile = from + it.tile0;
    count = it.tiles * (warp + 1) / C::WARPS - from;
  } else {
    // Sequences are dealt to the threads in runs; a scan of their steps finds the cuts.
    const int run = (p.b.n_seqs + C::THREADS - 1) / C::THREADS;
    const int s0 = min(static_cast<int>(threadIdx.x) * run, p.b.n_seqs), s1 = min(s0 + run, p.b.n_seqs);
    int64_t mine = 0, upto = 0, before = 0;
    // (First the sums, then the sequence in which each warp's part begins.)
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
      for (int s = s0; s < s1 && (pass == 0 || before < u1); ++s) {
        const RowsItem it = rows_item(p, s, 0, seq_view(p.b, s));
        const int64_t steps = static_cast<int64_t>(it.tiles) * p.heads;
        if (pass == 0) {
          mine += steps;
          continue;
        }
        const int64_t after = before + steps;
        if (after > u0) {
#pragma unroll 1
          for (int w = 0; w < C::WARPS; ++w) {
            const int64_t at = u0 + static_cast<int>(u1 - u0) * w / C::WARPS;
            if (at >= before && at < after) {
              const int64_t off = at - before;
              const int h = off <= 0x7FFFFFFF ? static_cast<int>(off) / it.tiles : static_cast<int>(off / it.tiles);
              ctl->start[w] = {s, h, it.tile0 + static_cast<int>(off - static_cast<int64_t>(h) * it.tiles), at};
            }
          }
        }
        before = after;
      }
      if (pass == 1) break;
      upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      if (lane == 31) ctl->sums[warp] = upto;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < C::WARPS; ++w) {
        total += ctl->sums[w];
        if (w < warp) upto += ctl->sums[w];
      }
      before = upto - mine;
      // (At least one step a warp, so that no CTA between two others is empty.)
      n_cta = min(static_cast<int64_t>(gridDim.x), (total + C::WARPS - 1) / C::WARPS);
      if (blockIdx.x < n_cta) {
        const Cuts cuts(total, n_cta);
        u0 = cuts.at(blockIdx.x);
        u1 = cuts.at(blockIdx.x + 1);
      }
    }
    __syncthreads();
    my = ctl->start[warp];
    count = static_cast<int>(u1 - u0) * (warp + 1) / C::WARPS - static_cast<int>(u1 - u0) * warp / C::WARPS;
  }

  // The loader and the worker walk the same steps, the loader STAGES ahead; it leaves the items for the
  // worker in ctl->item.  (One loop with one copy of either's code: what a call costs before its first step is
  // mostly the fetch of its instructions.)
  if (count > 0) {
    Loader ld{};
    ld.s = my.s, ld.h = my.h - 1;      // (the first step begins an item for it)
    int stage = 0, tile = my.tile, from = 0;
    uint32_t items = 0;
    enum { kNothing, kItem, kSameItem } begin = kItem;     // what begins: another item, or another piece of the item
    RowsItem it{};
    State<D, NT> st;
#pragma unroll 1
    for (int k = -C::STAGES; k < count; ++k) {
      if (k >= 0) {
        if (begin != kNothing) {
          if (begin == kItem) {
            it = ctl->item[warp][items % Ctrl<C::WARPS, C::STAGES>::ITEMS];
            if (items > 0) tile = it.tile0;
            ++items;
            from = tile;
          }
          begin = kNothing;
          load_item<D, NT>(p, it, st, q_at, lane);
        }
        copies_wait<C::STAGES - 1>();
        __syncwarp();   // every lane's copies of the step are there
        const uint32_t info0 = ctl->info[warp][stage][0], info1 = ctl->info[warp][stage][1];
        step<D, NT>(p, it, st, ring + stage * C::STAGE, q_at, info0, info1, tile * kStep, lane);
        ++tile;
        __syncwarp();   // every lane has read the stage
        const int end = it.tile0 + it.tiles;
        const bool go_on = tile != end && k + 1 != count;
        if (!go_on || (tile - from) % kMaxSteps == 0) {
          const bool first = from == it.tile0, last = tile == end, whole = first && last;
          // A piece that the warp's part cuts: its first (0) or its last (1).
          const int place = first ? 1 : 0, early = k + 1 < count;
          const int64_t my_piece = static_cast<int64_t>(blockIdx.x) * C::WARPS + warp;
          float *carry = p.carry + my_piece * 2 * (C::PIECE / 4), *early_piece = p.early + my_piece * (C::PIECE / 4);
          float* to = go_on ? carry : early ? early_piece : reinterpret_cast<float*>(base + warp * C::OWN);
          const bool cont = tile - from > kMaxSteps;     // another piece of the item, in `carry`, was before
          end_piece<D, NT>(p, it, st, whole && !cont, cont ? carry + C::PIECE / 4 : to, lane);
          if (cont) join_two<D, NT>(p, it, carry, carry + C::PIECE / 4, whole ? nullptr : to, lane);
          if (!whole && !go_on && lane == 0)
            ctl->piece[warp][place] = Piece{my.at + k + 1 + (end - tile), 1, first, last, early, it.s, it.h, it.a, it.rows};
          begin = go_on ? kSameItem : kItem;
        }
      }
      if (k + C::STAGES < count) issue_step<D, NT>(p, ld, stage, ring, ctl, my.tile, warp, lane);
      copies_commit();   // (a group a step, empty ones behind the last, so that all but the newest STAGES - 1 are step k's)
      __syncwarp();      // (what lane 0 has written down of items and steps)
      if (++stage == C::STAGES) stage = 0;
    }
  }
  __syncthreads();

  // Pieces of one item lie in consecutive warps, in key order.
  Join join{};
#pragma unroll 1
  for (int i = 0; i < 2 * C::WARPS;) {
    const Piece lead = ctl->piece[i >> 1][i & 1];
    if (!lead.valid) {
      ++i;
      continue;
    }
    // Its pieces: `members` (bits) up to i.
    uint32_t members = 0;
    bool last = false;
#pragma unroll 1
    for (; i < 2 * C::WARPS; ++i) {
      const Piece& q = ctl->piece[i >> 1][i & 1];
      if (!q.valid) continue;
      if (q.s != lead.s || q.h != lead.h) break;
      members |= 1u << i;
      last = q.last;
    }
    const bool whole = lead.first && last;
    float* part = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (lead.first ? 1 : 0)) * (C::PIECE / 4);
#pragma unroll 1
    for (int at = threadIdx.x * 4; at < C::ROWS * D; at += C::THREADS * 4) {
      const int row = at / D, col = at - row * D;
      float top = -INFINITY, sum = 0.0f;
      float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll 1
      for (uint32_t m = members; m != 0; m &= m - 1) {
        const int w = (__ffs(m) - 1) >> 1, place = (__ffs(m) - 1) & 1;
        const float* piece = ctl->piece[w][place].early ? p.early + (static_cast<int64_t>(blockIdx.x) * C::WARPS + w) * (C::PIECE / 4)
                                                        : reinterpret_cast<const float*>(base + w * C::OWN);
        const float2 ml = *reinterpret_cast<const float2*>(piece + C::ROWS * D + 2 * row);
        const float4 o = *reinterpret_cast<const float4*>(piece + at);
        const float mx = fmaxf(top, ml.x), ref = mx == -INFINITY ? 0.0f : mx, keep = ex2(top - ref), add = ml.y * ex2(ml.x - ref);
        top = mx;
        sum = sum * keep + add;
        acc.x = acc.x * keep + add * o.x, acc.y = acc.y * keep + add * o.y, acc.z = acc.z * keep + add * o.z, acc.w = acc.w * keep + add * o.w;
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const float4 o = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (whole) {
        if (row < lead.rows) store_row4(p, lead.a, lead.h, row, col, D, o);
      } else {
        *reinterpret_cast<float4*>(part + at) = o;
        if (col == 0) *reinterpret_cast<float2*>(part + C::ROWS * D + 2 * row) = make_float2(top, sum);
      }
    }
    if (lead.first && !last)
      join = Join{static_cast<int>(Cuts(total, n_cta).part(lead.item_end - 1) - blockIdx.x) + 1, lead.a, 0, lead.rows, lead.h, {}};
  }
  if (!p.per_item && threadIdx.x == 0) p.joins[blockIdx.x] = join;
}

// The tensor map of a rank's codes: [n_pages][n_kv][page_size][D] bytes, a box of the tokens of one
// page that a step takes.
tp_status encode_pages(CUtensorMap* m, const void* codes, const tp_paged_cache& c, int64_t ld_page) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  if (fn == nullptr) return fail(TP_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t D = static_cast<cuuint64_t>(c.head_dim), P = static_cast<cuuint64_t>(c.page_size);
  const cuuint64_t dims[4] = {D, P, static_cast<cuuint64_t>(c.n_kv_heads), static_cast<cuuint64_t>(c.n_pages)};
  const cuuint64_t strides[3] = {D, D * P, static_cast<cuuint64_t>(ld_page)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(c.head_dim), static_cast<cuuint32_t>(c.page_size < kStep ? c.page_size : kStep), 1, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(codes), dims, strides, box, ones,
                        CU_TENSOR_MAP_INTERLEAVE_NONE,
                        c.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(TP_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", static_cast<int>(r));
  return TP_OK;
}

tp_status current_device(int* dev) {
  const cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (*dev < 0 || *dev >= 64) return fail(TP_ERR_UNSUPPORTED, "device index %d", *dev);
  return TP_OK;
}

// Which kernel takes a call, and how.
struct Plan {
  bool tiles;            // more than 32 rows a sequence and KV head: paged_tiles_kernel
  int row_tiles;         // of 8 rows, else
  bool per_item;         // a CTA an item, no second launch; else equal parts of all steps
  int ctas;              // of those parts
  int pieces;            // that a CTA leaves behind (AttendParams::early)
  size_t part_bytes, ws_bytes;
  bool carry;            // an item may be longer than a piece: workspace to go on from
};

Plan make_plan(const tp_paged_cache& c, const tp_paged_batch& b, int group, int sms) {
  Plan pl{};
  const int64_t rows = static_cast<int64_t>(b.max_new) * group;
  // The fewest row tiles that hold them: one tile on the kernel for two takes 138 us, not 116 (64 sequences of 6 rows),
  // 12 rows on four 261, not 152, and 18 on four 90, not 67 (16 sequences).  The other kernel, whose time hardly
  // depends on the rows, takes 104 us where 30 rows of 16 sequences take 90, 102 for 67 with 18 rows and 57 with 12,
  // 300 for 116 of the 64 sequences, but 40 for 46 with 30 rows of 4 sequences of up to 9000.
  pl.tiles = rows > 32;
  pl.row_tiles = rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : 4;
  const int64_t items = static_cast<int64_t>(b.n_seqs) * c.n_ranks * c.n_kv_heads;
  const int64_t keys = b.max_pages * c.page_size;
  // Few short items: each by one CTA, no second launch.  Otherwise equal parts.  (One token, 8 KV heads over
  // 200 keys: 8.9 us so, 14.5 in parts; 500: 10.8 and 14.4; 1000: 14.9 and 14.3; 2000: 22.6 and 14.2.  Of 12
  // sequences of 500: 12.2 and 16.6; 1000: 17.4 and 20.0; 2000: 27.9 and 27.5.)
  pl.per_item = !pl.tiles && items <= sms && keys <= 1024;
  pl.ctas = pl.tiles ? sms : sms * kCtasPerSm;
  if (!pl.per_item) {
    // A CTA's Join, its two partial items and (paged_rows_kernel) a piece of each warp; where there can be longer items
    // than a piece is, a piece to go on from (paged_rows_kernel: of each warp, and its next one).
    pl.part_bytes = pl.tiles ? paged_tiles_part_floats(c.head_dim) * 4
                             : static_cast<size_t>(8 * pl.row_tiles) * (c.head_dim + 2) * 4;
    pl.pieces = pl.tiles ? 0 : pl.row_tiles == 1 ? Cfg<128, 1>::WARPS : Cfg<128, 2>::WARPS;
    pl.carry = keys > kLongestPiece;
    const int carried = !pl.carry ? 0 : pl.tiles ? 1 : 2 * pl.pieces;
    pl.ws_bytes = static_cast<size_t>(pl.ctas) * ((2 + pl.pieces + carried) * pl.part_bytes + sizeof(Join));
  }
  return pl;
}

template <int D, int NT>
tp_status launch(const Plan& pl, const AttendParams& p, cudaStream_t stream) {
  using C = Cfg<D, NT>;
  struct Raised {
    std::once_flag once;
    cudaError_t err = cudaSuccess;
  };
  static Raised raised[64];
  int dev = 0;
  tp_status st = current_device(&dev);
  if (st != TP_OK) return st;
  Raised& r = raised[dev];
  std::call_once(r.once, [&] {
    r.err = cudaFuncSetAttribute(paged_rows_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::SMEM));
  });
  if (r.err != cudaSuccess) return cuda_fail(r.err, "cudaFuncSetAttribute(max dynamic shared memory)");
  const dim3 grid = pl.per_item ? dim3(static_cast<unsigned>(p.b.n_seqs), static_cast<unsigned>(p.heads))
                                : dim3(static_cast<unsigned>(pl.ctas));
  cudaError_t e = launch_pdl(paged_rows_kernel<D, NT>, grid, dim3(C::THREADS), C::SMEM, stream, p);
  if (e == cudaSuccess && !pl.per_item)
    e = launch_pdl(paged_join_kernel<D, C::ROWS, 64 / C::ROWS>, dim3(static_cast<unsigned>(pl.ctas), C::ROWS / kJoinRows<D, 64 / C::ROWS>), dim3(kJoinThreads), 0,
                   stream, p);
  if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
  return TP_OK;
}

template <int D>
tp_status launch_rows(const Plan& pl, const AttendParams& p, cudaStream_t stream) {
  switch (pl.row_tiles) {
    case 1: return launch<D, 1>(pl, p, stream);
    case 2: return launch<D, 2>(pl, p, stream);
    case 3: return launch<D, 3>(pl, p, stream);
    default: return launch<D, 4>(pl, p, stream);
  }
}

tp_status check_attention(const tp_paged_cache* c, const tp_paged_batch* b, int64_t T, int n_heads, bool* empty) {
  const tp_status st = check_paged(c, b, T, n_heads, empty);
  if (st != TP_OK) return st;
  if (n_heads < 1 || n_heads % c->n_kv_heads != 0)
    return fail(TP_ERR_INVALID_ARG, "n_heads (%d) must be a multiple of n_kv_heads (%d)", n_heads, c->n_kv_heads);
  if (static_cast<int64_t>(T) * (n_heads / c->n_kv_heads) + b->n_seqs > 0x7FFFFFFF ||
      static_cast<int64_t>(c->n_ranks) * c->n_kv_heads > 65535)
    return fail(TP_ERR_UNSUPPORTED, "more than 2^31-1 rows of a KV head, or 65535 KV heads of all ranks");
  if (static_cast<double>(b->n_seqs) * c->n_ranks * c->n_kv_heads * (static_cast<double>(b->max_pages) * c->page_size) > 0x1p40)
    return fail(TP_ERR_UNSUPPORTED, "page tables of more than 2^40 keys, over all KV heads");   // (a CTA counts its steps in 32 bits)
  return TP_OK;
}

}  // namespace
}  // namespace tp

extern "C" {

size_t tp_attention_paged_workspace_bytes(const tp_paged_cache* cache, const tp_paged_batch* batch, int64_t T, int n_heads) {
  using namespace tp;
  size_t bytes = 0;
  (void)guarded([&]() -> tp_status {
    clear_error();
    bool empty = false;
    const tp_status st = check_attention(cache, batch, T, n_heads, &empty);
    if (st != TP_OK || empty) return st;
    const int sms = sm_count();
    if (sms <= 0) return fail(TP_ERR_CUDA, "no CUDA device");
    bytes = make_plan(*cache, *batch, n_heads / cache->n_kv_heads, sms).ws_bytes;
    return TP_OK;
  });
  return bytes;
}

tp_status tp_attention_paged_fp8(const tp_paged_cache* cache, const tp_paged_batch* batch, const void* const* q,
                                 int64_t ld_q, int64_t T, int n_heads, float scale, int causal, int window,
                                 void* workspace, size_t ws_bytes, void* const* out, int64_t ldo, tp_stream_t stream) {
  using namespace tp;
  return guarded([&]() -> tp_status {
    clear_error();
    bool empty = false;
    tp_status st = check_attention(cache, batch, T, n_heads, &empty);
    if (st != TP_OK) return st;
    const tp_paged_cache& c = *cache;
    const int64_t wide = static_cast<int64_t>(n_heads) * c.head_dim;
    if ((ld_q != 0 && ld_q < wide) || (ldo != 0 && ldo < wide))
      return fail(TP_ERR_INVALID_ARG, "a row stride (ld_q %lld, ldo %lld) is smaller than its row", (long long)ld_q, (long long)ldo);
    if ((causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal))
      return fail(TP_ERR_INVALID_ARG, "causal must be 0 or 1, and window >= 0 and 0 without causal; got %d, %d", causal, window);
    const float scale_log2e = scale * 1.4426950408889634f;
    if (!(scale_log2e - scale_log2e == 0.0f)) return fail(TP_ERR_INVALID_ARG, "scale must be finite, and below 2^127");
    if (empty) return TP_OK;
    if (q == nullptr || out == nullptr) return fail(TP_ERR_INVALID_ARG, "q or out is NULL");
    if (ld_q % 8 != 0 || ldo % 8 != 0)
      return fail(TP_ERR_ALIGNMENT, "ld_q (%lld) and ldo (%lld) must be multiples of 8", (long long)ld_q, (long long)ldo);
    AttendParams p{};
    for (int r = 0; r < c.n_ranks; ++r) {
      p.k[r] = static_cast<const uint8_t*>(c.k[r]);
      p.v[r] = static_cast<const uint8_t*>(c.v[r]);
      if (q[r] == nullptr || out[r] == nullptr) return fail(TP_ERR_INVALID_ARG, "q[%d] or out[%d] is NULL", r, r);
      if (!aligned16(q[r]) || !aligned16(out[r]))
        return fail(TP_ERR_ALIGNMENT, "q[%d] or out[%d] is not 16-byte aligned", r, r);
      p.q[r] = static_cast<const __nv_bfloat16*>(q[r]);
      p.out[r] = static_cast<__nv_bfloat16*>(out[r]);
      p.ks[r] = static_cast<const uint8_t*>(c.k_scales[r]);
      p.vs[r] = static_cast<const uint8_t*>(c.v_scales[r]);
    }
    const int sms = sm_count();
    if (sms <= 0) return fail(TP_ERR_CUDA, "no CUDA device");
    const Plan pl = make_plan(c, *batch, n_heads / c.n_kv_heads, sms);
    if (pl.ws_bytes > 0 && (workspace == nullptr || ws_bytes < pl.ws_bytes))
      return fail(TP_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace == nullptr ? size_t(0) : ws_bytes, pl.ws_bytes);
    if (pl.ws_bytes > 0 && !aligned16(workspace)) return fail(TP_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
    unsigned int* status = status_word();
    if (status == nullptr) return fail(TP_ERR_CUDA, "cannot locate the kernel status word");
    const int64_t ld_page = c.ld_page != 0 ? c.ld_page : static_cast<int64_t>(c.n_kv_heads) * c.page_size * c.head_dim;
    p.b = batch_view(c, *batch, T, status);
    p.ld_q = ld_q != 0 ? ld_q : wide;
    p.ldo = ldo != 0 ? ldo : wide;
    p.ld_page = ld_page;
    p.ld_scales = c.ld_scales != 0 ? c.ld_scales : c.n_kv_heads;
    p.n_kv = c.n_kv_heads;
    p.group = n_heads / c.n_kv_heads;
    p.heads = c.n_ranks * c.n_kv_heads;
    p.by_kv = div_by(static_cast<uint32_t>(p.n_kv));
    p.by_group = div_by(static_cast<uint32_t>(p.group));
    p.causal = causal;
    p.window = window <= p.b.max_keys ? window : 0;
    p.scale_log2e = scale_log2e;
    p.per_item = pl.per_item ? 1 : 0;
    if (!pl.per_item) {
      p.joins = static_cast<Join*>(workspace);
      p.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.ctas * sizeof(Join));
      p.early = reinterpret_cast<float*>(reinterpret_cast<char*>(p.parts) + 2 * pl.ctas * pl.part_bytes);
      p.carry = reinterpret_cast<float*>(reinterpret_cast<char*>(p.early) + static_cast<size_t>(pl.ctas) * pl.pieces * pl.part_bytes);
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (pl.tiles) {
      CodeMaps maps{};
      for (int r = 0; r < c.n_ranks && c.n_pages > 0; ++r) {
        st = encode_pages(&maps.k[r], c.k[r], c, ld_page);
        if (st == TP_OK) st = encode_pages(&maps.v[r], c.v[r], c, ld_page);
        if (st != TP_OK) return st;
      }
      return launch_paged_tiles(c.head_dim, pl.ctas, p, maps, s);
    }
    return c.head_dim == 128 ? launch_rows<128>(pl, p, s) : launch_rows<64>(pl, p, s);
  });
}

}  // extern "C"
