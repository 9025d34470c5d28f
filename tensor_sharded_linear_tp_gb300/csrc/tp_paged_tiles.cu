// Attention over the paged 8-bit cache, many rows a KV head (prompts, chunks): tcgen05.
//
//     S = scale Q K^T,  O = softmax(S) V,  an item = 256 rows (new tokens x query heads of the KV
//     head, token by token) of one sequence, KV head and rank, over its steps of 128 keys
//
// All steps of all items are one line, cut into equal parts, one for each CTA (one an SM): a CTA takes
// pieces of items one after the other, and pieces of an item in several CTAs are joined by a second
// launch (tp_paged_attention.cuh).  So neither the causal triangle nor ragged lengths leave SMs idle.
//
// CTA (512 threads):
//   warps 0..3    the codes' way: 16-byte loads of the pages, a step ahead in registers, two codes an
//                 instruction to fp16 (exact), times the page's scale relative to the largest one (a
//                 power of two), into a ring of two K and two V tiles, 128-byte swizzled.  What no row sees is 0.
//   warps 4..7    softmax of stream 0, warps 8..11 of stream 1, a row a thread (its TMEM lane).
//   warp 12       one thread issues the MMAs.
//   warp 13       one thread finds the pieces, ahead of the others.
// The two streams keep the tensor core busy in turn: while one's softmax runs, the other's products
// do.  With more than 128 rows each stream has 128 of them, over every step; otherwise both have
// the same rows, stream 0 the even steps and stream 1 the odd ones, and they are joined at the end.
//
// Tensor memory: S_g in columns [128 g, 128 g + 128), its P over the first 64 as fp16 pairs; O_g in
// [256 + D g, + D).  Per turn: S = Q K^T (K-major operands), P.V with P from tensor memory and V
// as stored (MN-major).  A stream's S of the next turn follows its P.V in the issue order, so that it
// may overwrite P.
//
// Numbers: Q enters as fp16, each row times a power of two to below 2^15 (what that loses lies 2^-39
// below its largest element).  K's codes enter times 2^(e - E + 7), E the largest exponent of the step's pages,
// V's likewise with E the largest so far: at most 448 * 2^7 < 65504, and what is 2^-40 below the largest is
// lost.  P = 2^(s - m + 7) with the running maximum m raised only where a row exceeds it by more than 8, so P
// is at most 2^15; l sums the unrounded P, O stays in units of 2^(E - 7).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "tp_internal.h"
#include "tp_paged_attention.cuh"
#include "tp_ptx.cuh"

namespace tp {
namespace {

constexpr int kThreads = 512;
constexpr int kKeys = 128;                        // keys of a step
constexpr int kRows = 256;                        // rows of an item
constexpr int kInfos = 4;                         // steps whose Info is kept: those in the ring and the one in the softmax
constexpr uint32_t SUB = 16384;                   // 128 rows x 64 fp16, 128-byte swizzled
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// What the softmax has to know of a step's pages.
struct Info {
  int e_k, e_v;            // exponents that the step's K and V are relative to
  uint32_t unseen, nan;    // by 16 keys: the page is out of bounds; K or V is NaN
};

// A piece of an item: steps from .. from + n of its sequence's keys (n = 0: no more pieces).
struct PieceInfo {
  int s, h;               // sequence; rank and KV head
  int a, len, pos0;       // SeqView
  int row0, rows;         // the item's rows
  int key_end, from, n;
  int first, last;        // does it hold the item's first and last step

  // Turns of the two streams: with both on the same rows (split) turn u is step u, else step u / 2; stream u % 2.
  __device__ __forceinline__ bool split() const { return rows <= 128; }
  __device__ __forceinline__ int turns() const { return split() ? n : 2 * n; }
};
constexpr int kPieces = 4;
constexpr int kPieceReaders = 4 + 8 + 1;   // warps of the codes' way and the softmax, the MMA thread

struct alignas(16) TilesCtrl {
  uint64_t q_full[2];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t info_full[kInfos];
  uint64_t pair;           // both streams' softmax threads
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint64_t drain;
  PieceInfo piece[kPieces];
  uint32_t tmem_base;
  int abort;
  Info info[kInfos];
  int64_t sums[kThreads / 32];
  int64_t total;
  struct {
    int s, h, block, tile;
  } start;
  float ml[128][3];        // stream 1's m, l and exponent of V of each row, for the join of the streams
};

template <int D>
struct Dims {
  static constexpr int HALVES = D / 64;
  static constexpr uint32_t TILE = HALVES * SUB;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = 2 * TILE;
  static constexpr uint32_t OFF_V = OFF_K + 2 * TILE;
  static constexpr uint32_t DATA = OFF_V + 2 * TILE;
  static constexpr size_t SMEM = 1024 + DATA + sizeof(TilesCtrl);
  static_assert(SMEM <= 232448, "shared memory");
};

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned int* status,
                                     bool ignore_abort = false) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0) {
      if (!ignore_abort && *abort_flag) return false;
      if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        atomicOr(status, TP_DEVSTATUS_TIMEOUT);
        return false;
      }
    }
  }
}

__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two codes as fp16, times a power of two (also as fp16, twice).
__device__ __forceinline__ uint32_t scaled_pair(uint32_t codes, uint32_t by) {
  uint32_t r;
  asm("{\n\t.reg .b32 t;\n\tcvt.rn.f16x2.e4m3x2 t, %1;\n\tmul.rn.f16x2 %0, t, %2;\n\t}"
      : "=r"(r)
      : "h"(static_cast<uint16_t>(codes)), "r"(by));
  return r;
}
// 2^e as fp16 in both halves, 0 below its least subnormal value; e <= 7 here.
__device__ __forceinline__ uint32_t f16_pow2(int e) {
  const uint32_t h = e >= -14 ? static_cast<uint32_t>(e + 15) << 10 : e >= -24 ? 1u << (e + 24) : 0u;
  return h * 0x10001u;
}

// The pieces of a CTA's part, one after the other, handed to the other warps through ctl->piece; and
// the item that begins in the part and goes beyond it.  One thread.
__device__ __forceinline__ void hand_out_pieces(const AttendParams& p, TilesCtrl* ctl, int64_t u0, int64_t u1, int64_t total, int64_t n_cta) {
  int s = ctl->start.s, h = ctl->start.h, block = ctl->start.block, from = ctl->start.tile;
  int64_t at = u0;
  Join join{};
  SeqView v{0, 0, 0, 0};
  if (u1 > u0) v = seq_view(p.b, s);
  for (uint32_t k = 0;; ++k) {
    if (!wait(ptx::smem_addr(&ctl->piece_empty[k % kPieces]), ((k / kPieces) & 1) ^ 1u, &ctl->abort, p.b.status)) break;
    PieceInfo& out = ctl->piece[k % kPieces];
    const bool more = at < u1;
    out.n = 0;
    if (more) {
      const Item it = item_of<kRows, kKeys>(p, v, block);
      const int left = it.tile0 + it.tiles - from, n = static_cast<int>(min(static_cast<int64_t>(left), u1 - at));
      out = PieceInfo{s, h, v.a, v.len, v.pos0, it.row0, it.rows, it.key_end, from, n, from == it.tile0, n == left};
      at += n;
      if (out.first && !out.last) {
        // CTA c holds step u where c is the largest with cut(c) <= u.
        const int64_t u = at + left - n - 1;
        const int64_t c_last = ((u + 1) * n_cta + total - 1) / total - 1;
        join = Join{static_cast<int>(c_last - blockIdx.x) + 1, v.a, it.row0, it.rows, h, {}};
      }
    }
    ptx::mbar_arrive(ptx::smem_addr(&ctl->piece_full[k % kPieces]));
    if (!more) break;
    if (at < u1) {
      if (static_cast<int64_t>(++block) * kRows >= static_cast<int64_t>(v.n) * p.group) {
        block = 0;
        if (++h == p.heads) {
          h = 0;
          do {
            v = seq_view(p.b, ++s);
          } while (v.n == 0 && s + 1 < p.b.n_seqs);
        }
      }
      from = item_of<kRows, kKeys>(p, v, block).tile0;
    }
  }
  p.joins[blockIdx.x] = join;
}

// The k-th piece (its n is 0 behind the last, or where a wait gave up).  Warp-collective for the warps
// that call it as a whole.
__device__ __forceinline__ const PieceInfo* get_piece(TilesCtrl* ctl, const PieceInfo* none, uint32_t k, unsigned int* status) {
  const bool ok = wait(ptx::smem_addr(&ctl->piece_full[k % kPieces]), (k / kPieces) & 1, &ctl->abort, status);
  return ok ? &ctl->piece[k % kPieces] : none;
}

// Steps of sequence v's items together, over one head, added up by a warp (every lane has the sum).
__device__ __forceinline__ int64_t sequence_steps(const AttendParams& p, const SeqView& v, int lane) {
  const int64_t blocks = (static_cast<int64_t>(v.n) * p.group + kRows - 1) / kRows;
  int64_t sum = 0;
  for (int64_t b = lane; b < blocks; b += 32) sum += item_of<kRows, kKeys>(p, v, static_cast<int>(b)).tiles;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return sum;
}

// Finds this CTA's part [u0, u1) of all steps and where it begins (ctl->start).  Every warp sums a run
// of sequences, 32 at a time: a lane takes a sequence of one item, the whole warp one of several.
// Block-collective.
__device__ __forceinline__ void find_part(const AttendParams& p, TilesCtrl* ctl, int64_t& u0, int64_t& u1, int64_t& total, int64_t& n_cta) {
  constexpr int kW = kThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int batches = (p.b.n_seqs + 31) / 32, run = (batches + kW - 1) / kW;
  const int b0 = min(warp * run, batches), b1 = min(b0 + run, batches);
  auto batch_steps = [&](int b, SeqView& v) -> int64_t {    // of this lane's sequence, all heads
    const int s = b * 32 + lane;
    v = SeqView{0, 0, 0, 0};
    if (s < p.b.n_seqs) v = seq_view(p.b, s);
    const int64_t rows = static_cast<int64_t>(v.n) * p.group;
    int64_t mine = rows > 0 && rows <= kRows ? item_of<kRows, kKeys>(p, v, 0).tiles : 0;
    for (uint32_t many = __ballot_sync(0xffffffffu, rows > kRows); many != 0; many &= many - 1) {
      const int src = __ffs(many) - 1;
      SeqView w;
      w.a = 0;
      w.n = __shfl_sync(0xffffffffu, v.n, src);
      w.len = __shfl_sync(0xffffffffu, v.len, src);
      w.pos0 = __shfl_sync(0xffffffffu, v.pos0, src);
      const int64_t sum = sequence_steps(p, w, lane);
      if (lane == src) mine = sum;
    }
    return mine * p.heads;
  };
  int64_t sum = 0;
  SeqView v;
  for (int b = b0; b < b1; ++b) sum += batch_steps(b, v);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) ctl->sums[warp] = sum;
  __syncthreads();
  int64_t before = 0;
  total = 0;
  for (int w = 0; w < kW; ++w) {
    if (w < warp) before += ctl->sums[w];
    total += ctl->sums[w];
  }
  n_cta = min(static_cast<int64_t>(gridDim.x), total);
  u0 = u1 = 0;
  if (blockIdx.x < n_cta) {
    u0 = cut(total, blockIdx.x, n_cta);
    u1 = cut(total, blockIdx.x + 1, n_cta);
  }
  if (u1 > u0 && u0 >= before && u0 < before + sum) {    // (one warp)
    for (int b = b0; b < b1; ++b) {
      const int64_t mine = batch_steps(b, v);
      int64_t upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      const int64_t all = __shfl_sync(0xffffffffu, upto, 31);
      if (u0 < before + all) {
        const bool here = u0 >= before + upto - mine && u0 < before + upto;
        const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        int64_t at = __shfl_sync(0xffffffffu, u0 - (before + upto - mine), src);
        const int64_t one = __shfl_sync(0xffffffffu, mine, src) / p.heads;
        const int s = b * 32 + src;
        const SeqView w = seq_view(p.b, s);
        const int h = static_cast<int>(at / one);
        at -= h * one;
        for (int first = 0;; first += 32) {              // the item in which step `at` of the head lies
          const bool is = static_cast<int64_t>(first + lane) * kRows < static_cast<int64_t>(w.n) * p.group;
          const Item it = item_of<kRows, kKeys>(p, w, is ? first + lane : 0);
          const int64_t tiles = is ? it.tiles : 0;
          int64_t to = tiles;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, to, d);
            if (lane >= d) to += o;
          }
          const bool hit = at >= to - tiles && at < to;
          if (hit) {
            ctl->start.s = s;
            ctl->start.h = h;
            ctl->start.block = first + lane;
            ctl->start.tile = it.tile0 + static_cast<int>(at - (to - tiles));
          }
          const int64_t whole = __shfl_sync(0xffffffffu, to, 31);
          if (__any_sync(0xffffffffu, hit) || whole == 0) break;
          at -= whole;
        }
        break;
      }
      before += all;
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- the codes' way (warps 0..3)

// A warp's rows of a tile: 32 keys, key 32 warp + 8 i + lane / 4, and of it 16-byte chunks lane % 4 and 4 more.
template <int D>
struct Raw {
  uint4 v[4][D / 64];
};

// Pages of a sequence and head, 32 at a time, a page a lane.
struct Pages {
  int page0, page;
  uint32_t info;     // as in the rows kernel: K's and V's scale byte, and that the index is valid
};
constexpr uint32_t kSeen = 0x10000;

__device__ __forceinline__ void load_pages(const AttendParams& p, Pages& pg, const PieceInfo& w, int first, int lane) {
  pg.page0 = first;
  pg.page = 0;
  pg.info = 0;
  const int64_t at = static_cast<int64_t>(first) + lane;
  if ((at << p.b.page_shift) < w.len) {
    pg.page = p.b.page_table[w.s * p.b.ld_table + at];
    if (pg.page >= 0 && pg.page < p.b.n_pages) {
      const int rank = w.h / p.n_kv, head = w.h - rank * p.n_kv;
      const int64_t sc = static_cast<int64_t>(pg.page) * p.ld_scales + head;
      pg.info = kSeen | p.ks[rank][sc] | (static_cast<uint32_t>(p.vs[rank][sc]) << 8);
    } else {
      bad_index(p.b);
    }
  }
}

// What a warp keeps of a step: where its two groups of 16 keys are, and their scales.
struct Scales {
  uint32_t info[2];
  int e_k, e_v;         // the largest exponents of the step's pages
  uint32_t unseen, nan;
};
struct Step {
  int64_t off[2];       // of the group's page and head in the codes, -1: not there
  int key0;
  Scales scales;
};

// get_piece for a whole warp: null behind the last.
__device__ __forceinline__ const PieceInfo* warp_piece(TilesCtrl* ctl, uint32_t k, unsigned int* status) {
  const PieceInfo* w = get_piece(ctl, nullptr, k, status);
  return __all_sync(0xffffffffu, w != nullptr) && w->n > 0 ? w : nullptr;
}

template <int D>
__device__ __forceinline__ Step locate(const AttendParams& p, Pages& pg, const PieceInfo& w, int tile, int warp, int lane) {
  Step st;
  st.key0 = tile * kKeys;
  const int shift = p.b.page_shift, first = st.key0 >> shift, pages = max(kKeys >> shift, 1);
  if (first < pg.page0 || first + pages > pg.page0 + 32) load_pages(p, pg, w, first, lane);
  const int head = w.h - w.h / p.n_kv * p.n_kv;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int key = st.key0 + 32 * warp + 16 * i, src = (key >> shift) - pg.page0;
    st.scales.info[i] = __shfl_sync(0xffffffffu, pg.info, src);
    const int page = __shfl_sync(0xffffffffu, pg.page, src);
    st.off[i] = (st.scales.info[i] & kSeen) != 0
                    ? page * p.ld_page + (static_cast<int64_t>(head) * p.b.page_size + (key & (p.b.page_size - 1))) * D
                    : -1;
  }
  // Lane i < 8: the page of the step's i-th 16 keys.
  const uint32_t mine = __shfl_sync(0xffffffffu, pg.info, ((st.key0 + 16 * (lane & 7)) >> shift) - pg.page0);
  const uint32_t k = mine & 0xFFu, v = (mine >> 8) & 0xFFu;
  const bool seen = (mine & kSeen) != 0;
  // (Keys behind the sequence's last are never seen; their pages are not there either.)
  const bool there = st.key0 + 16 * (lane & 7) < w.len;
  st.scales.unseen = __ballot_sync(0xffffffffu, !seen && there) & 0xFFu;
  st.scales.nan = __ballot_sync(0xffffffffu, seen && (k == 255u || v == 255u)) & 0xFFu;
  st.scales.e_k = __reduce_max_sync(0xffffffffu, seen && k != 255u ? static_cast<int>(k) - 127 : -127);
  st.scales.e_v = __reduce_max_sync(0xffffffffu, seen && v != 255u ? static_cast<int>(v) - 127 : -127);
  return st;
}

template <int D>
__device__ __forceinline__ void load_raw(Raw<D>& r, const uint8_t* codes, const Step& st, int key_end, int warp, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = 8 * (i & 1) + (lane >> 2);       // of the group of 16
    const bool there = st.off[i >> 1] >= 0 && st.key0 + 32 * warp + 16 * (i >> 1) + key < key_end;
    const uint4* at = reinterpret_cast<const uint4*>(codes + st.off[i >> 1] + key * D) + (lane & 3);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) r.v[i][c] = there ? at[4 * c] : make_uint4(0, 0, 0, 0);
  }
}

// To fp16 in the tile at `tile`: element d of a key is in sub-tile d / 64, 16-byte chunk (d % 64) / 8 of
// the key's row, swizzled.  Eight lanes store two keys' chunks of one parity each: no bank twice.
template <int D>
__device__ __forceinline__ void store_tile(const Raw<D>& r, uint32_t tile, const uint32_t (&by)[2], int warp, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 32 * warp + 8 * i + (lane >> 2);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const uint32_t w[4] = {r.v[i][c].x, r.v[i][c].y, r.v[i][c].z, r.v[i][c].w};
      uint32_t h[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[2 * k] = scaled_pair(w[k], by[i >> 1]);
        h[2 * k + 1] = scaled_pair(w[k] >> 16, by[i >> 1]);
      }
      const uint32_t dst = tile + c * SUB + row * 128;
      const int chunk = 2 * (lane & 3), x = row & 7;
      ptx::st_shared_v4(dst + ((chunk ^ x) << 4), h[0], h[1], h[2], h[3]);
      ptx::st_shared_v4(dst + (((chunk + 1) ^ x) << 4), h[4], h[5], h[6], h[7]);
    }
  }
}

template <int D>
__device__ __forceinline__ void codes_way(const AttendParams& p, TilesCtrl* ctl, uint32_t sbase, int warp, int lane) {
  using M = Dims<D>;
  volatile int* abort_flag = &ctl->abort;
  uint32_t k = 0;
  const PieceInfo* w = warp_piece(ctl, k, p.b.status);
  if (w == nullptr) return;
  Pages pg{-64, 0, 0};
  Raw<D> rk, rv;
  int tile = w->from, end = tile + w->n, key_end = w->key_end, h = w->h, s = w->s;   // of the step that is loaded next
  int e_run = -1000;                         // V's exponent in the piece so far
  Step next = locate<D>(p, pg, *w, tile, warp, lane);
  load_raw<D>(rk, p.k[h / p.n_kv], next, key_end, warp, lane);
  load_raw<D>(rv, p.v[h / p.n_kv], next, key_end, warp, lane);
  for (uint32_t t = 0;; ++t) {
    const Scales st = next.scales;
    e_run = max(e_run, st.e_v);
    const int e_now = e_run;
    // The step behind this one, in this piece or the next.
    bool more = true;
    if (++tile == end) {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl->piece_empty[k % kPieces]));
      w = warp_piece(ctl, ++k, p.b.status);
      more = w != nullptr;
      if (more) {
        if (w->s != s || w->h != h) pg.page0 = -64;
        tile = w->from, end = tile + w->n, key_end = w->key_end, h = w->h, s = w->s;
        e_run = -1000;
      }
    }
    if (more) next = locate<D>(p, pg, *w, tile, warp, lane);
    const uint32_t stage = t & 1, parity = ((t >> 1) & 1) ^ 1u;
    uint32_t by[2];
    // K: the tile two steps back has been multiplied.
    if (!__all_sync(0xffffffffu, wait(ptx::smem_addr(&ctl->k_empty[stage]), parity, abort_flag, p.b.status))) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) by[i] = (st.info[i] & 0xFFu) == 255u ? 0u : f16_pow2(static_cast<int>(st.info[i] & 0xFFu) - 127 - st.e_k + 7);
    if (st.nan != 0) {      // a NaN page's codes are NaN: 0 instead (the softmax knows)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          if ((st.info[i >> 1] & 0xFFu) == 255u) rk.v[i][c] = make_uint4(0, 0, 0, 0);
          if ((st.info[i >> 1] & 0xFF00u) == 0xFF00u) rv.v[i][c] = make_uint4(0, 0, 0, 0);
        }
    }
    store_tile<D>(rk, sbase + M::OFF_K + stage * M::TILE, by, warp, lane);
    if (warp == 0 && lane == 0) {
      // (The slot's last reader was done before the tile two steps back could be multiplied.)
      ctl->info[t % kInfos] = Info{st.e_k, e_now, st.unseen, st.nan};
      ptx::mbar_arrive(ptx::smem_addr(&ctl->info_full[t % kInfos]));
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl->k_full[stage]));
    if (more) load_raw<D>(rk, p.k[h / p.n_kv], next, key_end, warp, lane);
    // V.
    if (!__all_sync(0xffffffffu, wait(ptx::smem_addr(&ctl->v_empty[stage]), parity, abort_flag, p.b.status))) return;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      by[i] = (st.info[i] & 0xFF00u) == 0xFF00u ? 0u : f16_pow2(static_cast<int>((st.info[i] >> 8) & 0xFFu) - 127 - e_now + 7);
    store_tile<D>(rv, sbase + M::OFF_V + stage * M::TILE, by, warp, lane);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl->v_full[stage]));
    if (!more) return;
    load_raw<D>(rv, p.v[h / p.n_kv], next, key_end, warp, lane);
  }
}

// ---------------------------------------------------------------- the MMAs (one thread)

template <int D>
__device__ __forceinline__ void issue_mmas(const AttendParams& p, TilesCtrl* ctl, uint32_t sbase, uint32_t tmem) {
  using M = Dims<D>;
  volatile int* abort_flag = &ctl->abort;
  // fp16 operands, fp32 accumulators (the operand formats' codes are 0).
  constexpr uint32_t idesc = (1u << 4) | ((kKeys >> 3) << 17) | ((128u >> 4) << 24);
  constexpr uint32_t idesc_pv = (1u << 4) | ((static_cast<uint32_t>(D) >> 3) << 17) | ((128u >> 4) << 24) | ptx::kIdescMnMajorB;
  uint32_t base = 0;                      // steps before this piece
  uint32_t q_uses[2] = {0, 0}, p_uses[2] = {0, 0};
  bool ok = true;
  for (uint32_t k = 0; ok; ++k) {
    const PieceInfo* w = get_piece(ctl, nullptr, k, p.b.status);
    if (w == nullptr || w->n == 0) break;
    const bool split = w->split();
    const int turns = w->turns(), n = w->n;
    ptx::mbar_arrive(ptx::smem_addr(&ctl->piece_empty[k % kPieces]));
    auto issue_s = [&](int u) {
      const int g = u & 1, step = split ? u : u >> 1;
      const uint32_t t = base + step;
      if ((split || g == 0) && !wait(ptx::smem_addr(&ctl->k_full[t & 1]), (t >> 1) & 1, abort_flag, p.b.status)) return false;
      ptx::tc_fence_after();
      const uint32_t kb = sbase + M::OFF_K + (t & 1) * M::TILE, qb = sbase + M::OFF_Q + (split ? 0 : g) * M::TILE;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t sub = (kk >> 2) * SUB, k4 = 2u * (kk & 3);
        ptx::umma_bf16(tmem + g * kKeys, ptx::sw128_kmajor_desc(qb + sub) + k4, ptx::sw128_kmajor_desc(kb + sub) + k4, idesc, kk > 0 ? 1u : 0u);
      }
      ptx::umma_commit(ptx::smem_addr(&ctl->s_full[g]));
      if (split || g == 1) ptx::umma_commit(ptx::smem_addr(&ctl->k_empty[t & 1]));
      return true;
    };
    for (int g = 0; g < (split ? 1 : 2) && ok; ++g)
      ok = wait(ptx::smem_addr(&ctl->q_full[g]), q_uses[g]++ & 1, abort_flag, p.b.status);
    for (int u = 0; u < 2 && u < turns && ok; ++u) ok = issue_s(u);
    for (int u = 0; u < turns && ok; ++u) {
      const int g = u & 1, step = split ? u : u >> 1;
      const uint32_t t = base + step;
      ok = ((!split && g == 1) || wait(ptx::smem_addr(&ctl->v_full[t & 1]), (t >> 1) & 1, abort_flag, p.b.status)) &&
           wait(ptx::smem_addr(&ctl->p_full[g]), p_uses[g]++ & 1, abort_flag, p.b.status);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint64_t vdesc = ptx::sw128_mnmajor_desc(sbase + M::OFF_V + (t & 1) * M::TILE, SUB, 1024);
#pragma unroll
      for (int kk = 0; kk < kKeys / 16; ++kk)
        ptx::umma_bf16_ts(tmem + 2 * kKeys + g * D, tmem + g * kKeys + kk * 8, vdesc + kk * (2048u >> 4), idesc_pv,
                          (u >= 2 || kk > 0) ? 1u : 0u);
      if (split || g == 1) ptx::umma_commit(ptx::smem_addr(&ctl->v_empty[t & 1]));
      if (u + 2 < turns)
        ok = issue_s(u + 2);
      else
        ptx::umma_commit(ptx::smem_addr(&ctl->o_done[g]));
    }
    base += n;
  }
  ptx::umma_commit(ptx::smem_addr(&ctl->drain));
  wait(ptx::smem_addr(&ctl->drain), 0, abort_flag, p.b.status, true);
}

// ---------------------------------------------------------------- softmax (a row a thread)

// The row's Q as fp16 in its tile, times a power of two; returns what the scores have to be multiplied
// with (log2 units), NaN where the row holds a NaN or an infinity.
template <int D>
__device__ __forceinline__ float load_q(const AttendParams& p, const PieceInfo& w, int row, bool sees, uint32_t tile, int lane_row) {
  uint4 raw[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) raw[i] = make_uint4(0, 0, 0, 0);
  if (row < w.rows) {
    const int r = w.row0 + row, token = r / p.group, hq = r - token * p.group;
    const int rank = w.h / p.n_kv, head = w.h - rank * p.n_kv;
    const uint4* src = reinterpret_cast<const uint4*>(p.q[rank] + static_cast<int64_t>(w.a + token) * p.ld_q +
                                                      (static_cast<int64_t>(head) * p.group + hq) * D);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) raw[i] = src[i];
  }
  uint32_t* words = reinterpret_cast<uint32_t*>(raw);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < D / 2; ++i) top = __vmaxu2(top, words[i] & 0x7FFF7FFFu);
  top = max(top & 0xFFFFu, top >> 16);
  const int E = static_cast<int>(top >> 7);             // top < 2^(E - 126): times 2^(141 - E) below 2^15
  float f0 = pow2((141 - E) / 2);
  const float f1 = pow2(141 - E - (141 - E) / 2);
  float back = fabsf(p.scale_log2e) * pow2((E - 141) / 2) * pow2(E - 141 - (E - 141) / 2);
  if (p.scale_log2e < 0.0f) f0 = -f0;                   // (so that the largest score is the largest product)
  const bool zero = E == 255 || p.scale_log2e == 0.0f;
  if (E == 255) back = __uint_as_float(0x7FFFFFFFu);
  if (!sees) back = 1.0f;
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = zero ? 0u : words[4 * c + i];
      h[i] = f16_pair(__uint_as_float(v << 16) * f0 * f1, __uint_as_float(v & 0xFFFF0000u) * f0 * f1);
    }
    ptx::st_shared_v4(tile + (c >> 3) * SUB + lane_row * 128 + (((c & 7) ^ (lane_row & 7)) << 4), h[0], h[1], h[2], h[3]);
  }
  return back;
}

struct RowState {
  float m, l;
  int e_v;
};

// A step of the row: its scores from tensor memory, P over them, O rescaled where m or V's exponent grew.
template <int D>
__device__ __forceinline__ void softmax_step(RowState& st, const Info& info, float back, int lo, int hi, uint32_t s_addr, uint32_t o_addr, bool fresh) {
  uint32_t sv[kKeys];
#pragma unroll
  for (int i = 0; i < 4; ++i) ptx::tmem_ld_32x32b_x32(s_addr + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * i]));
  // (c is kept above 0, so that it may multiply the -infinity of a masked key; smaller ones make every score 0.)
  float c = back * pow2(info.e_k - 7);
  if (c < 0x1p-100f) c = 0x1p-100f;
  ptx::tmem_ld_wait();
  if (__any_sync(0xffffffffu, lo > 0 || hi < kKeys)) {
#pragma unroll
    for (int t = 0; t < kKeys; ++t)
      if (t < lo || t >= hi) sv[t] = 0xFF800000u;
  }
  if ((info.unseen | info.nan) != 0) {
#pragma unroll
    for (int t = 0; t < kKeys; ++t) {
      if ((info.unseen >> (t >> 4)) & 1) sv[t] = 0xFF800000u;
      else if (((info.nan >> (t >> 4)) & 1) && t >= lo && t < hi) sv[t] = 0x7FFFFFFFu;
    }
  }
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int t = 0; t < kKeys; t += 2) mx[(t >> 1) & 3] = max3(mx[(t >> 1) & 3], __uint_as_float(sv[t]), __uint_as_float(sv[t + 1]));
  const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
  float alpha = 1.0f;
  if (mt > st.m + 8.0f || (st.m == -INFINITY && mt > st.m)) {
    alpha = ex2(st.m - mt);
    st.m = mt;
    st.l *= alpha;
  }
  if (info.e_v > st.e_v) {
    alpha *= pow2(max(st.e_v - info.e_v, -127));
    st.e_v = info.e_v;
  }
  const bool rescale = !fresh && __any_sync(0xffffffffu, alpha != 1.0f);
  const float shift = 7.0f - (st.m == -INFINITY ? 0.0f : st.m);
  const uint64_t c2 = f2(c, c), s2 = f2(shift, shift);
  uint64_t ls[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    // Packed in place: the pair of column t comes from entries 2 t and 2 t + 1.
    uint32_t* pk = &sv[32 * half];
#pragma unroll
    for (int t = 0; t < 32; ++t) {
      const uint64_t x2 = fma2(f2(__uint_as_float(sv[64 * half + 2 * t]), __uint_as_float(sv[64 * half + 2 * t + 1])), c2, s2);
      float x0, x1;
      f2_split(x2, x0, x1);
      const float p0 = ex2(x0), p1 = ex2(x1);
      ls[t & 3] = add2(ls[t & 3], f2(p0, p1));
      pk[t] = f16_pair(p0, p1);
    }
    ptx::tmem_st_32x32b_x32(s_addr + 32 * half, *reinterpret_cast<uint32_t(*)[32]>(pk));
  }
  if (rescale) {
#pragma unroll 1
    for (int col = 0; col < D; col += 32) {
      uint32_t v[32];
      ptx::tmem_ld_32x32b_x32(o_addr + col, v);
      ptx::tmem_ld_wait();
#pragma unroll
      for (int t = 0; t < 32; ++t) v[t] = __float_as_uint(__uint_as_float(v[t]) * alpha);
      ptx::tmem_st_32x32b_x32(o_addr + col, v);
    }
  }
  ptx::tmem_st_wait();
  float a0, a1;
  f2_split(add2(add2(ls[0], ls[1]), add2(ls[2], ls[3])), a0, a1);
  st.l += a0 + a1;
}

template <int D>
__device__ __forceinline__ void softmax_rows(const AttendParams& p, TilesCtrl* ctl, uint32_t sbase, uint32_t tmem, int g, int warp, int lane) {
  using M = Dims<D>;
  volatile int* abort_flag = &ctl->abort;
  const int q = warp & 3, lane_row = 32 * q + lane;
  const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
  const uint32_t s_addr = tmem + lane_base + g * kKeys, o_addr = tmem + lane_base + 2 * kKeys + g * D;
  uint32_t base = 0, s_uses = 0, pair_uses = 0, o_uses[2] = {0, 0};
  // Both streams' threads meet (a bounded wait, as every other).
  auto meet = [&]() {
    const uint32_t bar = ptx::smem_addr(&ctl->pair);
    ptx::mbar_arrive(bar);
    return __all_sync(0xffffffffu, wait(bar, pair_uses++ & 1, abort_flag, p.b.status));
  };
  for (uint32_t k = 0;; ++k) {
    const PieceInfo* piece = warp_piece(ctl, k, p.b.status);
    if (piece == nullptr) return;
    const PieceInfo& w = *piece;
    const bool split = w.split();
    const int turns = w.turns(), from = w.from, n = w.n;
    const int row = (split ? 0 : 128 * g) + lane_row;
    const int pos = w.pos0 + (w.row0 + row) / p.group;
    int lo = 0, hi = 0x40000000;          // keys [lo, hi) are seen (by the row; what none needs is not masked)
    if (row < w.rows) {
      hi = p.causal ? min(w.len, pos + 1) : w.len;
      lo = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
    }
    float back;
    if (!split || g == 0) {
      back = load_q<D>(p, w, row, hi > lo, sbase + M::OFF_Q + g * M::TILE, lane_row);
      if (split) ctl->ml[lane_row][0] = back;
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(ptx::smem_addr(&ctl->q_full[g]));
    }
    if (split) {
      if (!meet()) return;
      if (g == 1) back = ctl->ml[lane_row][0];
    }
    RowState st{-INFINITY, 0.0f, -1000};
    bool fresh = true;
    for (int u = g; u < turns; u += 2) {
      const int step = split ? u : u >> 1;
      if (!__all_sync(0xffffffffu, wait(ptx::smem_addr(&ctl->s_full[g]), s_uses++ & 1, abort_flag, p.b.status))) return;
      ptx::tc_fence_after();
      const uint32_t t = base + step;
      if (!__all_sync(0xffffffffu, wait(ptx::smem_addr(&ctl->info_full[t % kInfos]), (t / kInfos) & 1, abort_flag, p.b.status))) return;
      const Info info = ctl->info[t % kInfos];
      const int key0 = (from + step) * kKeys;
      softmax_step<D>(st, info, back, lo - key0, hi - key0, s_addr, o_addr, fresh);
      fresh = false;
      ptx::tc_fence_before();
      ptx::mbar_arrive(ptx::smem_addr(&ctl->p_full[g]));
    }
    base += n;
    // O of this stream (and where both have the same rows of the other one) is complete.
    const bool whole = w.first && w.last;
    const int n_streams = split ? min(turns, 2) : 1;
    if (split && g == 1) {
      ctl->ml[lane_row][0] = st.m;
      ctl->ml[lane_row][1] = st.l;
      ctl->ml[lane_row][2] = __int_as_float(st.e_v);
    }
    bool ok = true;
    for (int i = 0; i < 2; ++i)
      if (!split || i < n_streams) {
        // (A phase that this stream does not wait for has ended before the next one that it does: the
        // MMAs of a piece follow all of the piece before.)
        if (split || i == g) ok = wait(ptx::smem_addr(&ctl->o_done[i]), o_uses[i] & 1, abort_flag, p.b.status) && ok;
        ++o_uses[i];
      }
    if (!__all_sync(0xffffffffu, ok)) return;
    ptx::tc_fence_after();
    if (split && !meet()) return;
    if (!split || g == 0) {
      // O = sum over streams of O_i 2^(E_i - 7) 2^(m_i - m) / sum of l_i 2^(m_i - m).
      float m = st.m, l = st.l, w0 = 1.0f, w1 = 0.0f, e0, e1 = 0.0f;
      e0 = e8m0_value(static_cast<uint32_t>(max(st.e_v, -127) + 127));
      if (n_streams == 2) {
        const float m1 = ctl->ml[lane_row][0], l1 = ctl->ml[lane_row][1];
        e1 = e8m0_value(static_cast<uint32_t>(max(__float_as_int(ctl->ml[lane_row][2]), -127) + 127));
        m = fmaxf(st.m, m1);
        const float ref = m == -INFINITY ? 0.0f : m;
        w0 = ex2(st.m - ref), w1 = ex2(m1 - ref);
        l = st.l * w0 + l1 * w1;
      }
      const float inv = l == 0.0f ? 0.0f : 0x1p-7f / l;
      w0 *= inv, w1 *= inv;
      const int r = w.row0 + row, token = r / p.group, hq = r - token * p.group;
      const int rank = w.h / p.n_kv, head = w.h - rank * p.n_kv;
      __nv_bfloat16* dst = p.out[rank] + static_cast<int64_t>(w.a + token) * p.ldo + (static_cast<int64_t>(head) * p.group + hq) * D;
      constexpr int PART = kRows * (D + 2);
      float* part = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (w.first ? 1 : 0)) * PART;
#pragma unroll 1
      for (int col = 0; col < D; col += 32) {
        uint32_t v[32];
        ptx::tmem_ld_32x32b_x32(o_addr + col, v);
        ptx::tmem_ld_wait();
        float o[32];
#pragma unroll
        for (int t = 0; t < 32; ++t) o[t] = __uint_as_float(v[t]) * w0 * e0;
        if (n_streams == 2) {
          ptx::tmem_ld_32x32b_x32(o_addr + D + col, v);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int t = 0; t < 32; ++t) o[t] += __uint_as_float(v[t]) * w1 * e1;
        }
        if (row < w.rows) {
          if (whole) {
#pragma unroll
            for (int t = 0; t < 32; t += 8)
              *reinterpret_cast<uint4*>(dst + col + t) = make_uint4(pack_bf16(o[t], o[t + 1]), pack_bf16(o[t + 2], o[t + 3]),
                                                                    pack_bf16(o[t + 4], o[t + 5]), pack_bf16(o[t + 6], o[t + 7]));
          } else {
#pragma unroll
            for (int t = 0; t < 32; t += 4) *reinterpret_cast<float4*>(part + row * D + col + t) = make_float4(o[t], o[t + 1], o[t + 2], o[t + 3]);
          }
        }
      }
      if (!whole && row < w.rows) *reinterpret_cast<float2*>(part + kRows * D + 2 * row) = make_float2(m, l);
      ptx::tc_fence_before();
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl->piece_empty[k % kPieces]));
    if (split && !meet()) return;               // stream 1's O and state have been read
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) paged_tiles_kernel(const __grid_constant__ AttendParams p) {
  using M = Dims<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TilesCtrl* ctl = reinterpret_cast<TilesCtrl*>(base + M::DATA);
  const uint32_t sbase = ptx::smem_addr(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_addr(&ctl->q_full[i]), 128);
      ptx::mbar_init(ptx::smem_addr(&ctl->k_full[i]), 4);
      ptx::mbar_init(ptx::smem_addr(&ctl->k_empty[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->v_full[i]), 4);
      ptx::mbar_init(ptx::smem_addr(&ctl->v_empty[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->s_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->p_full[i]), 128);
      ptx::mbar_init(ptx::smem_addr(&ctl->o_done[i]), 1);
    }
    for (int i = 0; i < kInfos; ++i) ptx::mbar_init(ptx::smem_addr(&ctl->info_full[i]), 1);
    ptx::mbar_init(ptx::smem_addr(&ctl->pair), 256);
    for (int i = 0; i < kPieces; ++i) {
      ptx::mbar_init(ptx::smem_addr(&ctl->piece_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->piece_empty[i]), kPieceReaders);
    }
    ptx::mbar_init(ptx::smem_addr(&ctl->drain), 1);
    ctl->abort = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 12) {
    ptx::tmem_alloc(ptx::smem_addr(&ctl->tmem_base), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  pdl_wait();
  int64_t u0, u1, total, n_cta;
  find_part(p, ctl, u0, u1, total, n_cta);

  // 512 threads of 128 registers: 104 + 176 + 176 + 56 a warpgroup's thread.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    codes_way<D>(p, ctl, sbase, warp, lane);
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    softmax_rows<D>(p, ctl, sbase, tmem, (warp - 4) >> 2, warp, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 12) {
      if (lane == 0) issue_mmas<D>(p, ctl, sbase, tmem);
    } else if (warp == 13 && lane == 0) {
      hand_out_pieces(p, ctl, u0, u1, total, n_cta);
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int D>
tp_status launch(int ctas, const AttendParams& p, cudaStream_t stream) {
  using M = Dims<D>;
  struct Raised {
    std::once_flag once;
    cudaError_t err = cudaSuccess;
  };
  static Raised raised[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= 64) return fail(TP_ERR_UNSUPPORTED, "device index %d", dev);
  Raised& r = raised[dev];
  std::call_once(r.once, [&] {
    cudaFuncAttributes a{};
    r.err = cudaFuncGetAttributes(&a, paged_tiles_kernel<D>);
    // The warpgroups' shares of registers add up to what the block is launched with, 128 a thread.
    if (r.err == cudaSuccess && a.numRegs != 128) r.err = cudaErrorInvalidKernelImage;
    if (r.err == cudaSuccess)
      r.err = cudaFuncSetAttribute(paged_tiles_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(M::SMEM));
  });
  if (r.err != cudaSuccess) return cuda_fail(r.err, "paged_tiles_kernel's attributes");
  e = launch_pdl(paged_tiles_kernel<D>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), M::SMEM, stream, p);
  if (e == cudaSuccess)
    e = launch_pdl(paged_join_kernel<D, kRows>, dim3(static_cast<unsigned>(ctas), kRows / kJoinRows), dim3(kJoinThreads), 0, stream, p);
  if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
  return TP_OK;
}

}  // namespace

size_t paged_tiles_part_floats(int head_dim) { return static_cast<size_t>(kRows) * (head_dim + 2); }

tp_status launch_paged_tiles(int head_dim, int ctas, const AttendParams& p, cudaStream_t stream) {
  return head_dim == 128 ? launch<128>(ctas, p, stream) : launch<64>(ctas, p, stream);
}

}  // namespace tp
