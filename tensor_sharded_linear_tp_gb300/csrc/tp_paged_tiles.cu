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
//   warps 0..3    the codes' way (two for K, two for V): a step's codes from shared memory, two an
//                 instruction to fp16 (exact), times the page's scale relative to the largest one (a power
//                 of two), into a ring of two K and two V tiles, 128-byte swizzled.  What no row sees is 0.
//   warps 4..7    softmax of stream 0, warps 8..11 of stream 1, a row a thread (its TMEM lane).
//   warp 12       issues the MMAs.
//   warp 13       finds the pieces, ahead of the others, and asks their rows of Q into L2.
//   warp 14       finds a step's pages and scales, and has its codes loaded by TMA.
// The two streams keep the tensor core busy in turn: while one's softmax runs, the other's products
// do.  With more than 128 rows each stream has 128 of them, over every step; otherwise both have
// the same rows, stream 0 the even steps and stream 1 the odd ones, and they are joined at the end.
//
// Tensor memory: S_g in columns [128 g, 128 g + 128), its P (fp16 pairs) over the first 32 and the
// last 32 of them; O_g in [256 + D g, + D).  Per turn: S = Q K^T (K-major operands), P.V with P from tensor memory and V
// as stored (MN-major).  A stream's S of the next turn follows its P.V in the issue order, so that it
// may overwrite P.
//
// Numbers: Q enters as fp16, each row times a power of two to below 2^15 (what that loses lies 2^-39
// below its largest element).  K's codes enter times 2^(e - E + 7), E the largest exponent of the step's pages,
// V's likewise with E the largest so far: at most 448 * 2^7 < 65504, and off by at most half of fp16's least step, 2^-25 in
// units of 2^(E - 7), so 2^(E - 32); but from e = E - 32 down the factor itself is 0 and with it the page, which is at
// most 448 * 2^(E - 32).  (Factors in two parts would keep those pages: the codes' warps have no registers left for them,
// and a prompt of 4608 tokens took 340 us, not 331.)  P = 2^(s - m + 6) with the running maximum m raised only
// where a row exceeds it by more than 9, so P is at most 2^15 and what is 2^-31 below the largest is lost; l sums the
// unrounded P, O stays in units of 2^(E - 7).
//
// What bounds it: at 256 rows a key costs 2 D bytes of the cache, 4 D 256 FLOP and 256 exponentials; a step's
// products take 2048 cycles of the tensor core, its exponentials 1024 of an SM's rate, and measured it takes
// 4300 (D 128): a stream's softmax is some 1700 cycles from S to P, in turn with the other's, on schedulers that also
// convert the codes (without the softmax's arithmetic a chunk took 158 us, not 222; the epilogue and Q's loads are 3 and 5 %).  A
// prompt of 4608 tokens, 48 heads: 330 us, 790 TFLOP/s, 0.41 of the measured bf16 rate (135 us); a chunk of 300 tokens,
// 48 query on 8 KV heads, over 30011: 222 us, 0.52 (115 us).  With at most 128 rows each stream has steps of its own, and what bounds them
// is the one step of codes that fits beside the fp16 tiles: 2.6 us for 128 keys (48 rows of 16 sequences 104 us, where the
// bytes take 24).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <mutex>

#include "tp_internal.h"
#include "tp_paged_attention.cuh"
#include "tp_ptx.cuh"

namespace tp {
namespace {

constexpr int kThreads = 512;
constexpr int kKeys = 128;                        // keys of a step
constexpr int kRows = 256;                        // rows of an item
constexpr int kInfos = 8;                         // steps whose Info is kept: seven are in use (see pages_way)
constexpr float kBias = 6.0f, kSlack = 9.0f;     // P = 2^(s - m + kBias), m raised by scores above m + kSlack
constexpr uint32_t SUB = 16384;                   // 128 rows x 64 fp16, 128-byte swizzled
constexpr int kMaxSteps = kLongestPiece / kKeys;  // of a piece
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// A step's pages, by 16 keys.
struct alignas(16) Info {
  int e_k, e_v;            // exponents that the step's K and V are relative to
  uint32_t unseen, nan;    // bits: the page is out of bounds, or before every row's window; K or V is NaN
  uint32_t by[2][8];       // what K's and V's codes are multiplied with, as fp16 twice; kZero where they enter as 0
  int keys;                // of the step's keys, those that some row sees; the others enter as 0
};
constexpr uint32_t kZero = 0xFFFFFFFFu;

// A piece of an item: steps from .. from + n of its sequence's keys (n = 0: no more pieces).
struct PieceInfo {
  int s, h;               // sequence; rank and KV head
  int a, len, pos0;       // SeqView
  int row0, rows;         // the item's rows
  int key_lo, key_end;    // some row sees key_lo; none sees an earlier key, nor one from key_end on
  int from, n;
  int first, last;        // does it, with what it continues, hold the item's first step; does it hold the last one
  int cont, cut;          // it continues the piece before, and is continued by the next, for kMaxSteps: through p.carry

  // Turns of the two streams: with both on the same rows (split) turn u is step u, else step u / 2; stream u % 2.
  __device__ __forceinline__ bool split() const { return rows <= 128; }
  __device__ __forceinline__ int turns() const { return split() ? n : 2 * n; }
};
constexpr int kPieces = 4;
constexpr int kPieceReaders = 8 + 1 + 1;   // the warps of the softmax, of the MMAs and of the pages

struct alignas(16) TilesCtrl {
  uint64_t q_full[2];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_half[2], p_full[2], o_done[2];
  uint64_t info_full[kInfos];
  uint64_t raw_full[2], raw_empty[2];   // K's and V's codes of a step
  uint64_t pair;           // both streams' softmax threads
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint64_t drain;
  PieceInfo piece[kPieces];
  uint32_t tmem_base;
  int abort;
  Info info[kInfos];
  int64_t sums[kThreads / 32];
  struct {
    int s, h, block, tile;
  } start;
};

static_assert(sizeof(Info) % 16 == 0 && offsetof(Info, by) % 16 == 0 && offsetof(TilesCtrl, info) % 16 == 0, "read as uint4");

template <int D>
struct Dims {
  static constexpr int HALVES = D / 64;
  static constexpr uint32_t TILE = HALVES * SUB;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = 2 * TILE;
  static constexpr uint32_t OFF_V = OFF_K + 2 * TILE;
  static constexpr uint32_t OFF_RAW = OFF_V + 2 * TILE;    // codes of a step: K, then V
  static constexpr uint32_t RAW = kKeys * D;
  static constexpr uint32_t DATA = OFF_RAW + 2 * RAW;
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

// The pieces of a CTA's part, one after the other, handed to the other warps through ctl->piece, their
// rows of Q asked into L2; and the item that begins in the part and goes beyond it.  Warp 13, every lane
// the same but for the rows.
template <int D>
__device__ __forceinline__ void hand_out_pieces(const AttendParams& p, TilesCtrl* ctl, int64_t u0, int64_t u1, int64_t total, int64_t n_cta, int lane) {
  int s = ctl->start.s, h = ctl->start.h, block = ctl->start.block, from = ctl->start.tile;
  int64_t at = u0;
  bool first = false, cont = false;
  Join join{};
  SeqView v{0, 0, 0, 0};
  if (u1 > u0) v = seq_view(p.b, s);
  for (uint32_t k = 0;; ++k) {
    if (!__all_sync(0xffffffffu, wait(ptx::smem_addr(&ctl->piece_empty[k % kPieces]), ((k / kPieces) & 1) ^ 1u, &ctl->abort, p.b.status))) break;
    const bool more = at < u1;
    PieceInfo out{};
    if (more) {
      const Item it = item_of<kRows, kKeys>(p, v, block);
      const int left = it.tile0 + it.tiles - from, most = static_cast<int>(min(static_cast<int64_t>(left), u1 - at)), n = min(most, kMaxSteps);
      if (!cont) first = from == it.tile0;
      out = PieceInfo{s, h, v.a, v.len, v.pos0, it.row0, it.rows, it.key_lo, it.key_end, from, n, first, n == left, cont, n < most};
      at += n;
      cont = n < most;
      from += n;
      if (first && n == most && n < left) {
        const int64_t c_last = Cuts(total, n_cta).part(at + left - n - 1);
        join = Join{static_cast<int>(c_last - blockIdx.x) + 1, v.a, it.row0, it.rows, h, {}};
      }
    }
    if (lane == 0) {
      ctl->piece[k % kPieces] = out;
      ptx::mbar_arrive(ptx::smem_addr(&ctl->piece_full[k % kPieces]));
    }
    if (!more) break;
    const int rank = p.by_kv(h), head = h - rank * p.n_kv;
#pragma unroll 1
    for (int row = lane; row < out.rows; row += 32) {
      const int r = out.row0 + row, token = p.by_group(r);
      const __nv_bfloat16* q = p.q[rank] + static_cast<int64_t>(v.a + token) * p.ld_q +
                               (static_cast<int64_t>(head) * p.group + (r - token * p.group)) * D;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
      if (D == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64));
    }
    if (at < u1 && !cont) {
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
  if (lane == 0) p.joins[blockIdx.x] = join;
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
    const Cuts cuts(total, n_cta);
    u0 = cuts.at(blockIdx.x);
    u1 = cuts.at(blockIdx.x + 1);
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

// Pages of a sequence and head, 32 at a time, a page a lane.
struct Pages {
  int page0, page;
  uint32_t info;     // K's and V's scale byte, and that the index is valid
};
constexpr uint32_t kSeen = 0x10000;

__device__ __forceinline__ void load_pages(const AttendParams& p, Pages& pg, const PieceInfo& w, int first, int lane) {
  pg.page0 = first;
  pg.page = 0;
  pg.info = 0;
  const int64_t at = static_cast<int64_t>(first) + lane;
  // (The pages before every row's window may be gone, or have become another sequence's.  What is left out here no later
  // item of the sequence needs: their windows begin further on.)
  if ((at << p.b.page_shift) < w.len && ((at + 1) << p.b.page_shift) > w.key_lo) {
    pg.page = p.b.page_table[w.s * p.b.ld_table + at];
    if (pg.page >= 0 && pg.page < p.b.n_pages) {
      const int rank = p.by_kv(w.h), head = w.h - rank * p.n_kv;
      const int64_t sc = static_cast<int64_t>(pg.page) * p.ld_scales + head;
      pg.info = kSeen | p.ks[rank][sc] | (static_cast<uint32_t>(p.vs[rank][sc]) << 8);
    } else {
      bad_index(p.b);
    }
  }
}

// get_piece for a whole warp: null behind the last.
__device__ __forceinline__ const PieceInfo* warp_piece(TilesCtrl* ctl, uint32_t k, unsigned int* status) {
  const PieceInfo* w = get_piece(ctl, nullptr, k, status);
  return __all_sync(0xffffffffu, w != nullptr) && w->n > 0 ? w : nullptr;
}

// The pages' way (warp 14): where a step's keys are and what their scales are, for the others; and
// their codes into shared memory by TMA, a box a page (of 32 keys at most).
template <int D>
__device__ __forceinline__ void pages_way(const AttendParams& p, const CodeMaps& maps, TilesCtrl* ctl, uint32_t sbase, int lane) {
  using M = Dims<D>;
  volatile int* abort_flag = &ctl->abort;
  const int shift = p.b.page_shift, boxes = p.b.page_size == 16 ? 8 : 4, box_keys = kKeys / boxes;
  Pages pg{-64, 0, 0};
  int s = -1, h = -1;
  uint32_t t = 0;
  bool ok = true;
  // This lane's box of a step, and the bytes of all.
  struct Boxes {
    bool load;
    int rank, head, page, token;
    uint32_t bytes;
  };
  auto copy = [&](int i, const Boxes& b, uint32_t step) {
    const uint32_t full = ptx::smem_addr(&ctl->raw_full[i]);
    if (!__all_sync(0xffffffffu, wait(ptx::smem_addr(&ctl->raw_empty[i]), (step & 1) ^ 1u, abort_flag, p.b.status))) return false;
    if (lane == 0) ptx::mbar_arrive_expect_tx(full, b.bytes);
    __syncwarp();
    if (b.load)
      tma_load_page(sbase + M::OFF_RAW + i * M::RAW + lane * box_keys * D, i == 0 ? &maps.k[b.rank] : &maps.v[b.rank], full, b.token,
                    b.head, b.page);
    return true;
  };
  Boxes before{};
  for (uint32_t k = 0; ok; ++k) {
    const PieceInfo* piece = warp_piece(ctl, k, p.b.status);
    if (piece == nullptr) break;
    const PieceInfo w = *piece;
    if (w.s != s || w.h != h) pg.page0 = -64, s = w.s, h = w.h;
    const int rank = p.by_kv(w.h), head = w.h - rank * p.n_kv;
    int e_run = -127;
    for (int tile = w.from; tile < w.from + w.n && ok; ++tile, ++t) {
      const int key0 = tile * kKeys, first = key0 >> shift;
      if (first < pg.page0 || first + max(kKeys >> shift, 1) > pg.page0 + 32) load_pages(p, pg, w, first, lane);
      // Lane i < 8: the page of the step's i-th 16 keys (and lanes behind them the same again).
      const int key16 = key0 + 16 * (lane & 7);
      const uint32_t mine = __shfl_sync(0xffffffffu, pg.info, (key16 >> shift) - pg.page0);
      const uint32_t kb = mine & 0xFFu, vb = (mine >> 8) & 0xFFu;
      // (A page that an item before this one saw may lie before this one's windows.)
      const bool seen = (mine & kSeen) != 0 && ((key16 >> shift) + 1) << shift > w.key_lo, nan = seen && (kb == 255u || vb == 255u);
      const uint32_t unseen = __ballot_sync(0xffffffffu, !seen && key16 < w.len) & 0xFFu;   // (behind the last key nothing is seen anyway)
      const uint32_t nans = __ballot_sync(0xffffffffu, nan) & 0xFFu;
      const int e_k = __reduce_max_sync(0xffffffffu, seen && !nan ? static_cast<int>(kb) - 127 : -127);
      e_run = max(e_run, __reduce_max_sync(0xffffffffu, seen && !nan ? static_cast<int>(vb) - 127 : -127));
      // The box of lane i < boxes.
      const int key_box = key0 + box_keys * (lane & (boxes - 1));
      const uint32_t box_info = __shfl_sync(0xffffffffu, pg.info, (key_box >> shift) - pg.page0);
      const int box_page = __shfl_sync(0xffffffffu, pg.page, (key_box >> shift) - pg.page0);
      const bool load = lane < boxes && (box_info & kSeen) != 0 && key_box < w.key_end && ((key_box >> shift) + 1) << shift > w.key_lo;
      const int n_boxes = __popc(__ballot_sync(0xffffffffu, load));
      // (V's codes of step t - 3 have been taken, so V of step t - 4 is stored, P.V of step t - 6 done and
      // with it everything that reads that step's Info.)
      Info& info = ctl->info[t % kInfos];
      if (lane < 8) {
        info.by[0][lane] = seen && !nan ? f16_pow2(static_cast<int>(kb) - 127 - e_k + 7) : kZero;
        info.by[1][lane] = seen && !nan ? f16_pow2(static_cast<int>(vb) - 127 - e_run + 7) : kZero;
      }
      if (lane == 0) info.e_k = e_k, info.e_v = e_run, info.unseen = unseen, info.nan = nans, info.keys = w.key_end - key0;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl->info_full[t % kInfos]));
      // K of this step, V of the one before: K is needed first, and V's place is free late.
      const Boxes now{load, rank, head, box_page, key_box & (p.b.page_size - 1), static_cast<uint32_t>(n_boxes) * box_keys * D};
      ok = copy(0, now, t) && (t == 0 || copy(1, before, t - 1));
      before = now;
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&ctl->piece_empty[k % kPieces]));
  }
  if (ok && t > 0) copy(1, before, t - 1);
  // The last copies land before the CTA can exit.
  for (int i = 0; i < 2 && t > 0; ++i) wait(ptx::smem_addr(&ctl->raw_full[i]), (t - 1) & 1, abort_flag, p.b.status, true);
}

// The codes' way: warps 0 and 1 take K, 2 and 3 V, each 64 keys of every step, from shared memory to fp16
// in their tile, once the tile two steps back has been multiplied.
template <int D>
__device__ __forceinline__ void codes_way(const AttendParams& p, TilesCtrl* ctl, uint32_t sbase, int64_t steps, int warp, int lane) {
  using M = Dims<D>;
  constexpr int C = D / 64;                  // 16-byte chunks of a key that a lane has: lane % 4 and 4 more
  volatile int* abort_flag = &ctl->abort;
  const int is_v = warp >> 1;
  // Eight lanes have two keys r and r ^ 5 of a group of eight: their chunks meet no bank twice, neither
  // where they are read (rows of D bytes, swizzled) nor where they are written (rows of 128).
  const int r8 = (lane >> 3) ^ ((lane & 4) != 0 ? 5 : 0), row0 = 64 * (warp & 1) + r8;   // keys row0 + 8 i
  const uint32_t full = ptx::smem_addr(is_v ? &ctl->v_full[0] : &ctl->k_full[0]);
  const uint32_t empty = ptx::smem_addr(is_v ? &ctl->v_empty[0] : &ctl->k_empty[0]);
  const uint32_t raw_full = ptx::smem_addr(&ctl->raw_full[is_v]), raw_empty = ptx::smem_addr(&ctl->raw_empty[is_v]);
  const uint32_t src = sbase + M::OFF_RAW + is_v * M::RAW + row0 * D + (((lane & 3) ^ (D == 128 ? r8 : r8 >> 1 & 3)) << 4);
  // Element d of a key is in sub-tile d / 64, 16-byte chunk (d % 64) / 8 of the key's row, swizzled.
  const uint32_t dst0 = sbase + (is_v ? M::OFF_V : M::OFF_K) + row0 * 128 + (((2 * (lane & 3)) ^ r8) << 4);
  for (uint32_t t = 0; t < steps; ++t) {
    if (!__all_sync(0xffffffffu, wait(raw_full, t & 1, abort_flag, p.b.status))) return;
    const uint32_t stage = t & 1;
    if (!__all_sync(0xffffffffu, wait(empty + 8 * stage, ((t >> 1) & 1) ^ 1u, abort_flag, p.b.status))) return;
    const Info& info = ctl->info[t % kInfos];
    const uint4 by4 = *reinterpret_cast<const uint4*>(&info.by[is_v][4 * (warp & 1)]);
    const int keys = info.keys - row0;
    const uint32_t by[4] = {by4.x, by4.y, by4.z, by4.w};
    const bool zeros = __any_sync(0xffffffffu, by4.x == kZero || by4.y == kZero || by4.z == kZero || by4.w == kZero || keys <= 56);
    const uint32_t dst = dst0 + stage * M::TILE;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      uint4 raw[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(raw[i].x), "=r"(raw[i].y), "=r"(raw[i].z), "=r"(raw[i].w)
                     : "r"((src ^ (c * 64)) + i * 8 * D) : "memory");
      if (zeros) {
        // Codes that are not there, of NaN pages or behind the last key that is seen (any content): 0.
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (by[i >> 1] == kZero || 8 * i >= keys) raw[i] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w}, f = by[i >> 1] == kZero ? 0u : by[i >> 1];
        uint32_t h[8];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          h[2 * n] = scaled_pair(x[n], f);
          h[2 * n + 1] = scaled_pair(x[n] >> 16, f);
        }
        ptx::st_shared_v4(dst + c * SUB + i * 1024, h[0], h[1], h[2], h[3]);
        ptx::st_shared_v4((dst ^ 16) + c * SUB + i * 1024, h[4], h[5], h[6], h[7]);
      }
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
    // The codes are handed back only now that every lane's loads have arrived (the stores needed them).  Handed back when the
    // loads had been issued, they were overtaken by the next step's box: the MMAs' operands keep loads waiting that long.
    if (lane == 0) {
      ptx::mbar_arrive(raw_empty);
      ptx::mbar_arrive(full + 8 * stage);
    }
  }
}

// ---------------------------------------------------------------- the MMAs (warp 12)

// Column of S_g's region in which P's 16 keys kk are: the first 64 keys in columns 0..31, the last 64 in 96..127.
__host__ __device__ constexpr uint32_t p_column(int kk) { return kk < 4 ? 8u * kk : 64u + 8u * kk; }

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}

// The two streams' turns alternate, so that one's softmax runs while the other's products do (with a warp for
// each stream they fell into step, both in the softmax and then both waiting for the tensor core: a step of
// 5000 cycles, not 4300).  The whole warp runs the loop, so that addresses stay in uniform registers; one lane issues.
template <int D>
__device__ __forceinline__ void issue_mmas(const AttendParams& p, TilesCtrl* ctl, uint32_t sbase, uint32_t tmem) {
  using M = Dims<D>;
  volatile int* abort_flag = &ctl->abort;
  const bool issuer = elect_one();
  auto wait_all = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity, abort_flag, p.b.status)); };
  // fp16 operands, fp32 accumulators (the operand formats' codes are 0).
  constexpr uint32_t idesc = (1u << 4) | ((kKeys >> 3) << 17) | ((128u >> 4) << 24);
  constexpr uint32_t idesc_pv = (1u << 4) | ((static_cast<uint32_t>(D) >> 3) << 17) | ((128u >> 4) << 24) | ptx::kIdescMnMajorB;
  const uint64_t q0 = ptx::sw128_kmajor_desc(sbase + M::OFF_Q), k0 = ptx::sw128_kmajor_desc(sbase + M::OFF_K);
  const uint64_t v0 = ptx::sw128_mnmajor_desc(sbase + M::OFF_V, SUB, 1024);
  const uint32_t k_full = ptx::smem_addr(&ctl->k_full[0]), k_empty = ptx::smem_addr(&ctl->k_empty[0]);
  const uint32_t v_full = ptx::smem_addr(&ctl->v_full[0]), v_empty = ptx::smem_addr(&ctl->v_empty[0]);
  const uint32_t s_full = ptx::smem_addr(&ctl->s_full[0]), p_half = ptx::smem_addr(&ctl->p_half[0]), p_full = ptx::smem_addr(&ctl->p_full[0]);
  uint32_t base = 0;                      // steps before this piece
  uint32_t q_uses1 = 0, p_uses0 = 0, p_uses1 = 0;
  bool ok = true;
  for (uint32_t k = 0; ok; ++k) {
    const PieceInfo* w = warp_piece(ctl, k, p.b.status);
    if (w == nullptr) break;
    const bool split = w->split();
    const int turns = w->turns(), n = w->n;
    __syncwarp();
    if (issuer) ptx::mbar_arrive(ptx::smem_addr(&ctl->piece_empty[k % kPieces]));
    // Turn u: P.V of turn u - 2 of the same stream first (none for u < 2), then S of turn u (none behind the last).
    for (int u = 0; u < turns + 2 && ok; ++u) {
      const uint32_t g = u & 1;
      const uint32_t t = base + (split ? u : u >> 1), stage = t & 1;                       // S's step
      const uint32_t tv = t - (split ? 2 : 1), stage_v = tv & 1;                           // P.V's
      if (u < 2) {
        if (g == 0) ok = wait_all(ptx::smem_addr(&ctl->q_full[0]), k & 1);
        if (g == 1 && !split) ok = wait_all(ptx::smem_addr(&ctl->q_full[1]), q_uses1++ & 1);
      }
      // What is there by now is waited for before P, which is not.
      if (u >= 2 && (split || g == 0)) ok = ok && wait_all(v_full + 8 * stage_v, (tv >> 1) & 1);
      if (u < turns && (split || g == 0)) ok = ok && wait_all(k_full + 8 * stage, (t >> 1) & 1);
      if (u >= 2) {
        const uint64_t vdesc = v0 + stage_v * (M::TILE >> 4);
        const uint32_t parity = (g != 0 ? p_uses1++ : p_uses0++) & 1, o = tmem + 2 * kKeys + g * D, pr = tmem + g * kKeys;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          ok = ok && wait_all((half == 0 ? p_half : p_full) + 8 * g, parity);
          if (!ok) break;
          ptx::tc_fence_after();
          if (issuer) {
#pragma unroll
            for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
              ptx::umma_bf16_ts(o, pr + p_column(kk), vdesc + kk * (2048u >> 4), idesc_pv, (u >= 4 || kk > 0) ? 1u : 0u);
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      ptx::tc_fence_after();
      if (issuer) {
        if (u < turns) {
          const uint64_t qdesc = q0 + (split ? 0u : g * (M::TILE >> 4)), kdesc = k0 + stage * (M::TILE >> 4);
          const uint32_t to = tmem + g * kKeys;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            ptx::umma_bf16(to, qdesc + (kk >> 2) * (SUB >> 4) + 2 * (kk & 3), kdesc + (kk >> 2) * (SUB >> 4) + 2 * (kk & 3), idesc,
                           kk > 0 ? 1u : 0u);
          ptx::umma_commit(s_full + 8 * g);
          if (split || g == 1) ptx::umma_commit(k_empty + 8 * stage);
        } else if (u >= 2) {
          ptx::umma_commit(ptx::smem_addr(&ctl->o_done[0]) + 8 * g);
        }
        if (u >= 2 && (split || g == 1)) ptx::umma_commit(v_empty + 8 * stage_v);
      }
      __syncwarp();
    }
    base += n;
  }
  if (issuer) ptx::umma_commit(ptx::smem_addr(&ctl->drain));
  wait(ptx::smem_addr(&ctl->drain), 0, abort_flag, p.b.status, true);
}

// ---------------------------------------------------------------- softmax (a row a thread)

// The warp's 32 rows of Q as fp16 in its tile, each times a power of two: copied there as they are,
// then converted in place by the row's thread, in small rolled loops (this runs once a piece: what it costs is
// mostly the fetch of its instructions).  at: of this lane's row in q, in elements, negative where there is
// none.  Returns what the row's scores have to be multiplied with (log2 units), NaN where it holds a NaN or
// an infinity.
template <int D>
__device__ __forceinline__ float load_q(const AttendParams& p, const __nv_bfloat16* q, int64_t at, uint32_t tile, int q4, int lane) {
  constexpr int kLanes = D / 8, kRowsAtOnce = 32 / kLanes;   // lanes of a row; rows of a copy
  const int sub = lane % kLanes;
#pragma unroll 2
  for (int r0 = 0; r0 < 32; r0 += kRowsAtOnce) {
    const int r = r0 + lane / kLanes;
    const int64_t from = __shfl_sync(0xffffffffu, at, r);
    const uint32_t dst = tile + (sub >> 3) * SUB + (32 * q4 + r) * 128 + (((sub & 7) ^ (r & 7)) << 4);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(q + max(from, int64_t(0)) + sub * 8), "r"(from >= 0 ? 16 : 0)
                 : "memory");     // (a row that is not there: zeros, nothing is read)
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  const uint32_t row = tile + (32 * q4 + lane) * 128;
  auto chunk = [&](int c) { return row + (c >> 3) * SUB + (((c & 7) ^ (lane & 7)) << 4); };
  auto load = [&](uint32_t from, uint32_t (&w)[4]) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from) : "memory");
  };
  uint32_t top = 0;
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    uint32_t w[4];
    load(chunk(c), w);
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu)));
  }
  top = max(top & 0xFFFFu, top >> 16);
  const int E = static_cast<int>(top >> 7);             // top < 2^(E - 126): times 2^(141 - E) below 2^15
  const bool zero = E == 255 || p.scale_log2e == 0.0f;
  // (the sign of scale goes into Q, so that the largest score is the largest product)
  const float f0 = zero ? 0.0f : copysignf(pow2((141 - E) / 2), p.scale_log2e), f1 = pow2(141 - E - (141 - E) / 2);
#pragma unroll 2
  for (int c = 0; c < D / 8; ++c) {
    uint32_t w[4];
    load(chunk(c), w);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t v = zero ? 0u : w[k];
      w[k] = f16_pair(__uint_as_float(v << 16) * f0 * f1, __uint_as_float(v & 0xFFFF0000u) * f0 * f1);
    }
    ptx::st_shared_v4(chunk(c), w[0], w[1], w[2], w[3]);
  }
  return E == 255 ? __uint_as_float(0x7FFFFFFFu) : fabsf(p.scale_log2e) * pow2((E - 141) / 2) * pow2(E - 141 - (E - 141) / 2);
}

struct RowState {
  float m, l;
  int e_v;
};

// Ones from bit a up to below bit b (both taken into 0 .. 32).
__device__ __forceinline__ uint32_t bits(int a, int b) {
  a = min(max(a, 0), 32), b = min(max(b, 0), 32);
  return b <= a ? 0u : (0xFFFFFFFFu >> (32 - (b - a))) << a;
}
// The 32 keys from t0 on of a step that a row sees, and those whose page is NaN.
struct Seen {
  uint32_t seen, nan;
};
__device__ __forceinline__ Seen seen_chunk(const Info& info, int t0, int lo, int hi) {
  const uint32_t u = info.unseen >> (t0 >> 4), n = info.nan >> (t0 >> 4);
  auto spread = [](uint32_t w) { return (w & 1 ? 0xFFFFu : 0u) | (w & 2 ? 0xFFFF0000u : 0u); };
  return Seen{bits(lo - t0, hi - t0) & ~spread(u), spread(n)};
}
__device__ __forceinline__ void mask_chunk(uint32_t (&sv)[32], const Info& info, int t0, int lo, int hi) {
  Seen s = seen_chunk(info, t0, lo, hi);
  asm volatile("" : "+r"(s.seen), "+r"(s.nan));   // (the same keys are masked twice: not from 64 results kept meanwhile)
#pragma unroll
  for (int t = 0; t < 32; ++t) {
    sv[t] = (s.nan >> t) & 1 ? 0x7FFFFFFFu : sv[t];
    sv[t] = (s.seen >> t) & 1 ? sv[t] : 0xFF800000u;
  }
}
__device__ __forceinline__ float max_chunk(const uint32_t (&sv)[32], float top) {
  float mx[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int t = 0; t < 32; t += 2) mx[(t >> 1) & 3] = max3(mx[(t >> 1) & 3], __uint_as_float(sv[t]), __uint_as_float(sv[t + 1]));
  return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}
// P of 32 keys, stored as 16 columns.
__device__ __forceinline__ void exp_chunk(const uint32_t (&sv)[32], uint64_t c2, uint64_t s2, uint64_t (&ls)[2], uint32_t to) {
  uint32_t pk[16];
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    const uint64_t x2 = fma2(f2(__uint_as_float(sv[2 * t]), __uint_as_float(sv[2 * t + 1])), c2, s2);
    float x0, x1;
    f2_split(x2, x0, x1);
    const float p0 = ex2(x0), p1 = ex2(x1);
    ls[t & 1] = add2(ls[t & 1], f2(p0, p1));
    pk[t] = f16_pair(p0, p1);
  }
  ptx::tmem_st_32x32b_x16(to, pk);
}

// A step of the row: its scores from tensor memory, P over them, O rescaled where m or V's exponent
// grew.
template <int D>
__device__ __forceinline__ void softmax_step(RowState& st, const Info& info, float back, int lo, int hi, bool edge, uint32_t s_addr, uint32_t o_addr, bool fresh, uint32_t p_half) {
  uint32_t x[4][32];
#pragma unroll
  for (int i = 0; i < 4; ++i) ptx::tmem_ld_32x32b_x32(s_addr + 32 * i, x[i]);
  // (c is kept above 0, so that it may multiply the -infinity of a masked key; smaller ones make every score 0.)
  float c = back * pow2(info.e_k - 7);
  if (c < 0x1p-100f) c = 0x1p-100f;
  ptx::tmem_ld_wait();
  if (edge) {
#pragma unroll
    for (int i = 0; i < 4; ++i) mask_chunk(x[i], info, 32 * i, lo, hi);
  }
  float mt = -INFINITY;
  {
    float mx[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) mx[i] = max_chunk(x[i], -INFINITY);
    mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
  }
  float alpha = 1.0f;
  if (mt > st.m + kSlack) {      // (m is -infinity at first)
    alpha = ex2(st.m - mt);
    st.m = mt;
    st.l *= alpha;
  }
  if (info.e_v > st.e_v) {
    alpha *= pow2(max(st.e_v - info.e_v, -127));
    st.e_v = info.e_v;
  }
  const bool rescale = !fresh && __any_sync(0xffffffffu, alpha != 1.0f);
  const float shift = kBias - (st.m == -INFINITY ? 0.0f : st.m);
  const uint64_t c2 = f2(c, c), s2 = f2(shift, shift);
  uint64_t ls[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
  if (rescale) {      // (O is complete up to the step before: S follows its P.V in the tensor core)
#pragma unroll 1
    for (int col = 0; col < D; col += 16) {
      uint32_t v[16];
      ptx::tmem_ld_32x32b_x16(o_addr + col, v);
      ptx::tmem_ld_wait();
#pragma unroll
      for (int t = 0; t < 16; ++t) v[t] = __float_as_uint(__uint_as_float(v[t]) * alpha);
      ptx::tmem_st_32x32b_x16(o_addr + col, v);
    }
  }
  // P of the first 64 keys is multiplied while that of the others is computed.
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    exp_chunk(x[i], c2, s2, ls, s_addr + p_column(2 * i));
    if (i == 1) {
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      ptx::mbar_arrive(p_half);
    }
  }
  ptx::tmem_st_wait();
  float a0, a1;
  f2_split(add2(ls[0], ls[1]), a0, a1);
  st.l += a0 + a1;
}

// 32 rows of 128 bytes each in shared memory (a row a lane's, swizzled) to `to` + the rows' offsets (in
// bytes, negative: left out), four whole rows an instruction.  Warp-collective.
__device__ __forceinline__ void store_rows(char* to, int64_t offset, uint32_t stage, int lane) {
  __syncwarp();
#pragma unroll 2
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "r"(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4)) : "memory");
    const int64_t at = __shfl_sync(0xffffffffu, offset, r);
    if (at >= 0) *reinterpret_cast<uint4*>(to + at + (lane & 7) * 16) = x;
  }
  __syncwarp();
}

template <int D>
__device__ __forceinline__ void softmax_rows(const AttendParams& p, TilesCtrl* ctl, uint8_t* smem, uint32_t sbase, uint32_t tmem, int g, int warp, int lane) {
  using M = Dims<D>;
  volatile int* abort_flag = &ctl->abort;
  // Stream 1's m, l and exponent of V of each row, for the join of the streams: in the second tile of Q,
  // which is idle where both streams have the same rows.
  float(*ml)[3] = reinterpret_cast<float(*)[3]>(smem + M::OFF_Q + M::TILE);
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
    const int pos = w.pos0 + p.by_group(w.row0 + row);
    int lo = 0, hi = 0x40000000;          // keys [lo, hi) are seen (by the row; what none needs is not masked)
    if (row < w.rows) {
      hi = p.causal ? min(w.len, pos + 1) : w.len;
      lo = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
    }
    // Where the row is in q and out, in elements from the first rank's (negative: nowhere).
    const int rank = p.by_kv(w.h);
    int64_t token = -1, column = 0;
    if (row < w.rows) {
      const int r = w.row0 + row;
      token = p.by_group(r);
      column = (static_cast<int64_t>(w.h - rank * p.n_kv) * p.group + (r - token * p.group)) * D;
      token += w.a;
    }
    float back;
    if (!split || g == 0) {
      back = load_q<D>(p, p.q[rank], token < 0 ? -1 : token * p.ld_q + column, sbase + M::OFF_Q + g * M::TILE, q, lane);
      if (hi <= lo) back = 1.0f;
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(ptx::smem_addr(&ctl->q_full[g]));
    }
    if (split) {
      if (!meet()) return;      // (stream 1 is done with the piece before, which may have used the second tile)
      if (g == 0) ml[lane_row][0] = back;
      if (!meet()) return;
      if (g == 1) back = ml[lane_row][0];
    }
    RowState st{-INFINITY, 0.0f, -1000};
    bool fresh = true;
    for (int u = g; u < turns; u += 2) {
      const int step = split ? u : u >> 1;
      if (!__all_sync(0xffffffffu, wait(ptx::smem_addr(&ctl->s_full[g]), s_uses++ & 1, abort_flag, p.b.status))) return;
      ptx::tc_fence_after();
      const uint32_t t = base + step;
      if (!__all_sync(0xffffffffu, wait(ptx::smem_addr(&ctl->info_full[t % kInfos]), (t / kInfos) & 1, abort_flag, p.b.status))) return;
      const Info& info = ctl->info[t % kInfos];
      const int key0 = (from + step) * kKeys;
      // edge: some row does not see every key of the step.
      const bool edge = __any_sync(0xffffffffu, lo > key0 || hi < key0 + kKeys || (info.unseen | info.nan) != 0);
      softmax_step<D>(st, info, back, lo - key0, hi - key0, edge, s_addr, o_addr, fresh, ptx::smem_addr(&ctl->p_half[g]));
      fresh = false;
      ptx::tc_fence_before();
      ptx::mbar_arrive(ptx::smem_addr(&ctl->p_full[g]));
    }
    base += n;
    // O of this stream (and where both have the same rows of the other one) is complete.
    const bool whole = w.first && w.last, cont = w.cont;
    const int n_streams = split ? min(turns, 2) : 1;
    if (split && g == 1) {
      ml[lane_row][0] = st.m;
      ml[lane_row][1] = st.l;
      ml[lane_row][2] = __int_as_float(st.e_v);
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
        const float m1 = ml[lane_row][0], l1 = ml[lane_row][1];
        e1 = e8m0_value(static_cast<uint32_t>(max(__float_as_int(ml[lane_row][2]), -127) + 127));
        m = fmaxf(st.m, m1);
        const float ref = m == -INFINITY ? 0.0f : m;
        w0 = ex2(st.m - ref), w1 = ex2(m1 - ref);
        l = st.l * w0 + l1 * w1;
      }
      constexpr int PART = kRows * (D + 2);
      float* carry = p.carry + static_cast<int64_t>(blockIdx.x) * PART;
      float f2 = 0.0f;      // of the piece that this one continues, an O / l
      if (cont && row < w.rows) {
        const float2 c = *reinterpret_cast<const float2*>(carry + kRows * D + 2 * row);
        const float m1 = m;
        m = fmaxf(m1, c.x);
        const float ref = m == -INFINITY ? 0.0f : m, by = ex2(m1 - ref);
        f2 = c.y * ex2(c.x - ref);
        w0 *= by, w1 *= by;
        l = l * by + f2;
      }
      const float inv = l == 0.0f ? 0.0f : 0x1p-7f / l;
      w0 *= inv, w1 *= inv, f2 *= inv * 0x1p7f;
      float* part = w.cut ? carry : p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (w.first ? 1 : 0)) * PART;
      char* to = whole ? reinterpret_cast<char*>(p.out[rank]) : reinterpret_cast<char*>(part);
      const int64_t offset = token < 0 ? -1 : whole ? (token * p.ldo + column) * 2 : static_cast<int64_t>(row) * D * 4;
      // (Q's tile is idle: every S of this piece is done.)
      const uint32_t stage = sbase + M::OFF_Q + g * M::TILE + q * 4096;
      const float f0 = w0 * e0, f1 = w1 * e1;
      const int per = whole ? 64 : 32;     // columns of 128 bytes
#pragma unroll 1
      for (int col = 0; col < D; col += 16) {
        uint32_t v[16];
        float o[16];
        ptx::tmem_ld_32x32b_x16(o_addr + col, v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int t = 0; t < 16; ++t) o[t] = __uint_as_float(v[t]) * f0;
        if (n_streams == 2) {
          ptx::tmem_ld_32x32b_x16(o_addr + D + col, v);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int t = 0; t < 16; ++t) o[t] += __uint_as_float(v[t]) * f1;
        }
        if (cont && row < w.rows) {
#pragma unroll
          for (int t = 0; t < 16; t += 4) {
            const float4 c = *reinterpret_cast<const float4*>(carry + row * D + col + t);
            o[t] += c.x * f2, o[t + 1] += c.y * f2, o[t + 2] += c.z * f2, o[t + 3] += c.w * f2;
          }
        }
        const int at = col & (per - 1);
        const uint32_t line = stage + lane * 128;
        if (whole) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            ptx::st_shared_v4(line + ((((at >> 3) + i) ^ (lane & 7)) << 4), pack_bf16(o[8 * i], o[8 * i + 1]), pack_bf16(o[8 * i + 2], o[8 * i + 3]),
                              pack_bf16(o[8 * i + 4], o[8 * i + 5]), pack_bf16(o[8 * i + 6], o[8 * i + 7]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            ptx::st_shared_v4(line + ((((at >> 2) + i) ^ (lane & 7)) << 4), __float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]),
                              __float_as_uint(o[4 * i + 2]), __float_as_uint(o[4 * i + 3]));
        }
        if (at + 16 == per) store_rows(to + (col - at) * (whole ? 2 : 4), offset, stage, lane);
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
__global__ void __launch_bounds__(kThreads, 1) paged_tiles_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ CodeMaps maps) {
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
      ptx::mbar_init(ptx::smem_addr(&ctl->raw_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->raw_empty[i]), 2);
      ptx::mbar_init(ptx::smem_addr(&ctl->k_full[i]), 2);
      ptx::mbar_init(ptx::smem_addr(&ctl->k_empty[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->v_full[i]), 2);
      ptx::mbar_init(ptx::smem_addr(&ctl->v_empty[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->s_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->p_half[i]), 128);
      ptx::mbar_init(ptx::smem_addr(&ctl->p_full[i]), 128);
      ptx::mbar_init(ptx::smem_addr(&ctl->o_done[i]), 1);
    }
    for (int i = 0; i < kInfos; ++i) ptx::mbar_init(ptx::smem_addr(&ctl->info_full[i]), 1);
    ptx::mbar_init(ptx::smem_addr(&ctl->drain), 1);
    ptx::mbar_init(ptx::smem_addr(&ctl->pair), 256);
    for (int i = 0; i < kPieces; ++i) {
      ptx::mbar_init(ptx::smem_addr(&ctl->piece_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->piece_empty[i]), kPieceReaders);
    }
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

  // 512 threads of 128 registers: 64 + 192 + 192 + 64 a warpgroup's thread.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    codes_way<D>(p, ctl, sbase, u1 - u0, warp, lane);
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    softmax_rows<D>(p, ctl, base, sbase, tmem, (warp - 4) >> 2, warp, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 12) {
      issue_mmas<D>(p, ctl, sbase, tmem);
    } else if (warp == 13) {
      hand_out_pieces<D>(p, ctl, u0, u1, total, n_cta, lane);
    } else if (warp == 14) {
      pages_way<D>(p, maps, ctl, sbase, lane);
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
tp_status launch(int ctas, const AttendParams& p, const CodeMaps& maps, cudaStream_t stream) {
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
  e = launch_pdl(paged_tiles_kernel<D>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), M::SMEM, stream, p, maps);
  if (e == cudaSuccess)
    e = launch_pdl(paged_join_kernel<D, kRows, 1>, dim3(static_cast<unsigned>(ctas), kRows / kJoinRows<D, 1>), dim3(kJoinThreads), 0, stream, p);
  if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
  return TP_OK;
}

}  // namespace

size_t paged_tiles_part_floats(int head_dim) { return static_cast<size_t>(kRows) * (head_dim + 2); }

tp_status launch_paged_tiles(int head_dim, int ctas, const AttendParams& p, const CodeMaps& maps, cudaStream_t stream) {
  return head_dim == 128 ? launch<128>(ctas, p, maps, stream) : launch<64>(ctas, p, maps, stream);
}

}  // namespace tp
