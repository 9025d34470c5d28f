// Block-scaled 8-bit projections on the 5th-generation tensor cores.
//
//   colwise  Y_r = act(X . W_r^T + b_r),  rowwise  Z = sum_r X_r . W_r^T + b
//
// with e4m3 operands that carry one e8m0 scale per token and 128 features (X) and per 128 x 128
// block (W).  A scale is a power of two, so the tensor core applies it itself: tcgen05.mma
// kind::mxf8f6f4 takes a scale byte per operand row and 32 features from tensor memory, and the
// four K=32 steps of a group name the same byte.  Nothing is rescaled outside the MMA, the sum
// over K (and over the ranks of a rowwise call, in rank order) stays in one fp32 accumulator.
//
// Scale bytes reach tensor memory as 32-bit words of four consecutive groups (a "chunk", K = 512):
// operand row r's word lies in lane r % 32 of column r / 32, the same in each 32-lane quarter.
// Four warps load a chunk's words, a row to a lane, and leave them in shared memory in that order;
// the MMA thread copies them (tcgen05.cp) in front of the chunk's MMAs, which it stays in order
// with.
//
// fp8_tokens_kernel: the weight rows are the MMA's M (128 lanes), the tokens its N.  A launch is
// bound by the bytes of W, each read once: a ring of 128-byte-wide TMA boxes, and, when there are
// fewer 128-row tiles than SMs, the chunks of K split over the CTAs of a cluster.  Every CTA
// leaves its fp32 partial tile in its shared memory, and after a cluster barrier each CTA sums
// its share of the tokens over the CTAs in K order through distributed shared memory, applies
// bias and activation and stores (or quantises: a tile's 128 columns are one scale group).  One
// token's Q/K/V, 4 x 4608 x 6144, takes 21.4 us (5.3 TB/s; 16.7 us at the measured copy rate, the
// rest is a launch's start and join), gate/up of 23 tokens, 3 x 12288 x 6144, 39.3 us (5.8 TB/s).
// With 128 tokens a tile 144 CTAs take 32 KB each for a scale group, 227 MB from L2 in the 18 us of
// an out-projection of 300 tokens (4 x 6144 x 1536; some 12 us of them between start and join: 19 TB/s);
// the tensor pipe is 39 % busy, and without three quarters of the MMAs a launch is 10 % shorter.
//
// fp8_prompt_kernel: the tokens are M, 256 of them to a persistent CTA pair (cta_group::2), 256
// weight rows (SwiGLU: 128 gate and 128 up rows) are N.  Bound by the tensor core.  Two
// accumulators of 256 columns and the scale words do not fit tensor memory's 512 columns side by
// side, so the accumulators overlap by 32 columns: the epilogue reads those first and hands them
// back, and the next tile's MMAs start while it works through the rest.  Gate/up of 4608 tokens,
// 4 x 9216 x 6144 with SwiGLU to fp8, takes 649 us at the power limit (3220 TFLOP/s; 561 us in the
// first, unthrottled runs), the down projection 338 us (290).  A scale group's MMAs run 512 cycles; at
// the clocks sampled in 3 s of launches (1515 and 1400 MHz) gate/up takes 567 cycles a group of its
// 36 waves of 48, start and epilogues among them, down 548 of its 6 waves of 144.
//
// Every mbarrier wait is bounded (about 2 s); a CTA that gives up records it in the library's
// status word, lets its copies and MMAs drain, frees tensor memory and exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "tp_e4m3.cuh"
#include "tp_internal.h"
#include "tp_ptx.cuh"

namespace tp {
namespace {

constexpr int BM = 128;                // accumulator rows per CTA (TMEM lanes)
constexpr int KB = kFp8Group;          // K per stage: one 128-byte swizzled row, one scale group
constexpr int kChunk = 4;              // scale groups in one 32-bit word
constexpr uint32_t kBoxA = BM * KB;    // bytes of one operand box of 128 rows
constexpr int kMaxStages = 12;
constexpr int kMaxSplits = 8;          // CTAs of a cluster (portable limit)
constexpr uint64_t kWaitLimitNs = 2000000000ull;

struct Fp8Params {
  CUtensorMap map_x[TP_MAX_DEGREE];    // [0] only when the tokens are shared (colwise)
  CUtensorMap map_w[TP_MAX_DEGREE];
  const uint8_t* sx[TP_MAX_DEGREE];    // [T, k_groups], row stride ld_sx
  const uint8_t* sw[TP_MAX_DEGREE];    // [ceil(w_rows / 128), k_groups], dense
  const __nv_bfloat16* bias[TP_MAX_DEGREE];  // per output, nullable
  void* out[TP_MAX_DEGREE];                  // per output: bf16, or e4m3 when out_scales is set
  uint8_t* out_scales[TP_MAX_DEGREE];
  unsigned int* status;
  int64_t ld_sx, ldo, ld_os;
  int T;
  int w_rows;      // rows of each W
  int n_out;       // output columns of each output
  int up_row;      // SwiGLU: first row of the up block
  int n_groups;    // outputs (ranks of a colwise call; 1 for rowwise)
  int n_segs;      // K segments of an output (ranks of a rowwise call; 1 for colwise)
  int k_groups;    // scale groups (128 features) per segment
  int n_tiles, t_tiles;
  int splits;      // tokens kernel: cluster CTAs that share a tile's K
  int n_items;           // prompt kernel: n_tiles, or pairs of them (clusters of two CTA pairs)
  int group_m;           // prompt kernel: token tiles that sweep the weight tiles together
  bool x_words, w_words;  // scale chunks can be read as aligned 32-bit words
  int act;
};

// ---------------------------------------------------------------- instructions
// D[tmem] (+)= (A * 2^sfa)[smem] . (B * 2^sfb)[smem]^T, e4m3 operands, scale bytes in tensor memory.
__device__ __forceinline__ void umma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// The same over a CTA pair: 128 rows of A and half of B's rows from each CTA, issued by the leader.
__device__ __forceinline__ void umma_mx_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::mxf8f6f4: e4m3 A and B (both K-major), fp32 D, e8m0 scales, M x N tile.
__host__ __device__ constexpr uint32_t idesc_mx(int m, int n) {
  return (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(m >> 4) << 24);
}
// The byte of its scale words that an instruction uses, for A and B alike.
__device__ __forceinline__ uint32_t idesc_scale_byte(uint32_t k) { return (k << 4) | (k << 29); }

// Scale words of 128 rows from shared memory (32 x 16 bytes, dense) to four columns of tensor
// memory, the same in every 32-lane quarter; in order with the MMAs of the issuing thread.
// kPair: in both CTAs of a pair, each from its own shared memory.
template <bool kPair>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  const uint64_t desc = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu)     // start address
                        | (static_cast<uint64_t>(128 >> 4) << 32)         // stride of 8-row groups
                        | (static_cast<uint64_t>(1) << 46);               // descriptor version; no swizzle
  if constexpr (kPair)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Arrival on a barrier of the cluster without release semantics: what it announces is that tensor
// memory has been read, and tcgen05.wait::ld has seen to that.  (A release at cluster scope first
// waits for the thread's earlier memory operations: 1300 to 1700 cycles here, in which the tensor
// core had no work between two tiles.)
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Cluster barrier that orders no memory: for threads that have used all they read from other CTAs.
__device__ __forceinline__ void cluster_sync_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Bounded wait: true when the phase completed, false when this CTA is giving up.
// kCluster: the phase's arrivals may come from the other CTA of a pair.
template <bool kCluster>
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned int* status,
                                       bool ignore_abort) {
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (kCluster ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity)) return true;
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
template <bool kCluster = false>
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                             unsigned int* status, bool ignore_abort = false) {
  if (kCluster ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity)) return true;
  return wait_slow<kCluster>(bar, parity, abort_flag, status, ignore_abort);
}

// A box's bytes into L2.
__device__ __forceinline__ void prefetch_box(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

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

// ---------------------------------------------------------------- scale words
constexpr uint32_t kScaleOne = 0x7F7F7F7Fu;  // 2^0 for rows past the operand (their products are not stored)

// One row's word: scale bytes [kg, kg + n) of scale row (row >> kShift).  `words` (host: every
// row's chunks are aligned whole words) keeps the load free of branches, so that a thread's loads
// are in flight together.  (Not read-only loads: this CTA may have been resident while the kernel
// before wrote X's scales, and only ordinary loads are sure to see that after the grid wait.)
template <int kShift>
__device__ __forceinline__ uint32_t load_word(const uint8_t* s, int64_t ld, int rows, int row, int kg, int n,
                                              bool words) {
  const uint8_t* at = s + static_cast<int64_t>(row >> kShift) * ld + kg;
  if (words) return row < rows ? *reinterpret_cast<const uint32_t*>(at) : kScaleOne;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < kChunk; ++i)
    w |= (row < rows && i < n ? static_cast<uint32_t>(at[i]) : 0x7Fu) << (8 * i);
  return w;
}

constexpr int kSfBufs = 4;               // chunks of scale words in shared memory
constexpr uint32_t kSfRows = 32 * 16;    // bytes of 128 rows' words
__device__ __forceinline__ void store_word(uint32_t rows_at, int row, uint32_t w) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(rows_at + static_cast<uint32_t>((row & 31) * 16 + (row >> 5) * 4)), "r"(w)
               : "memory");
}

// The chunks of K in the order every role of a kernel walks them.
struct ChunkWalk {
  int seg, kg;  // segment and first scale group
  __device__ __forceinline__ void start(int chunk, int seg_chunks) {
    seg = chunk / seg_chunks;
    kg = (chunk - seg * seg_chunks) * kChunk;
  }
  __device__ __forceinline__ void next(int k_groups) {
    kg += kChunk;
    if (kg >= k_groups) kg = 0, ++seg;
  }
};

// ---------------------------------------------------------------- activation
// GELU(tanh) as x / (1 + e^(-2u)), u = sqrt(2/pi) (x + 0.044715 x^3); SiLU as x / (1 + e^(-x)).
__device__ __forceinline__ float gelu_tanh_f(float x) {
  const float u = 0.7978845608028654f * (x + 0.044715f * x * x * x);
  return __fdividef(x, 1.0f + __expf(-2.0f * u));
}
__device__ __forceinline__ float silu_f(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}

// ---------------------------------------------------------------- few tokens
template <int TN, bool kGlu>
struct TokensCfg {
  static constexpr int W_TILES = kGlu ? 2 : 1;                  // gate rows and up rows
  static constexpr uint32_t W_BYTES = W_TILES * kBoxA;
  static constexpr uint32_t X_BYTES = TN * KB;
  static constexpr uint32_t STAGE_BYTES = W_BYTES + X_BYTES;
  // Up to 32 tokens two CTAs fit an SM (so that a kernel's prologue runs beside its predecessor),
  // with 90 to 108 KB in flight each; more tokens take one CTA with up to 216 KB (SwiGLU of 64 tokens:
  // five stages 40.0 us, four 40.8).
  static constexpr bool SMALL = TN <= 32;
  static constexpr uint32_t RING_MAX = SMALL ? 110592 : 221184;
  static constexpr int STAGES = RING_MAX / STAGE_BYTES;
  static constexpr uint32_t RING = STAGES * STAGE_BYTES;
  static constexpr uint32_t PARTIAL = W_TILES * TN * BM * 4;    // fp32 [tile][token][128], over the ring
  static_assert(STAGES <= kMaxStages && PARTIAL <= RING, "the partial tile reuses the ring");
  static constexpr int ACC_COLS = W_TILES * TN;
  static constexpr int SF_COLS = 16;                            // per buffer: W (4 or 8), then tokens (4)
  static constexpr uint32_t TMEM_COLS = ACC_COLS + 2 * SF_COLS <= 64    ? 64
                                        : ACC_COLS + 2 * SF_COLS <= 128 ? 128
                                        : ACC_COLS + 2 * SF_COLS <= 256 ? 256
                                                                        : 512;
  static constexpr uint32_t SF_BYTES = (W_TILES + 1) * kSfRows;   // one chunk's words: W, then tokens
  static constexpr int SF_BUFS = 2;
  static constexpr size_t SMEM = 1024 + RING + SF_BUFS * SF_BYTES;
  // CTAs that can share an SM never ask for more tensor memory than it has, so that none waits for
  // another's: with clusters, whose CTAs wait for each other, that could close a circle.
  static constexpr int CTAS_PER_SM = static_cast<int>((228 * 1024) / (SMEM + 1024));
  static_assert(CTAS_PER_SM * TMEM_COLS <= 512, "tensor memory for every CTA an SM can hold");
};

struct alignas(8) TokensCtrl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t sf_full[2], sf_empty[2];
  uint64_t done;
  uint32_t tmem_base;
  int abort;
};

constexpr int kTokensThreads = 192;  // producer, MMA issuer, four scale / accumulator warps

template <int TN, bool kGlu>
__global__ void __launch_bounds__(kTokensThreads, TokensCfg<TN, kGlu>::SMALL ? 2 : 1)
    fp8_tokens_kernel(const __grid_constant__ Fp8Params p) {
  using C = TokensCfg<TN, kGlu>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ TokensCtrl ctl_mem;
  TokensCtrl* ctl = &ctl_mem;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort_flag = &ctl->abort;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform to the compiler
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    // The maps are launch parameters, so their descriptors can be fetched before the wait below.
    for (int r = 0; r < max(p.n_groups, p.n_segs); ++r) ptx::prefetch_tensormap(&p.map_w[r]);
    for (int r = 0; r < p.n_segs; ++r) ptx::prefetch_tensormap(&p.map_x[r]);
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(ptx::smem_addr(&ctl->full[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->empty[s]), 1);
    }
    for (int b = 0; b < C::SF_BUFS; ++b) {
      ptx::mbar_init(ptx::smem_addr(&ctl->sf_full[b]), 128);
      ptx::mbar_init(ptx::smem_addr(&ctl->sf_empty[b]), 1);
    }
    ptx::mbar_init(ptx::smem_addr(&ctl->done), 1);
    ctl->abort = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  // This CTA's tile and its share of the tile's chunks of K.
  const int splits = p.splits;
  const int part = static_cast<int>(blockIdx.x) % splits;
  const int tile = static_cast<int>(blockIdx.x) / splits;
  const int tt = tile % p.t_tiles;
  const int nt = tile / p.t_tiles % p.n_tiles;
  const int g = tile / p.t_tiles / p.n_tiles;
  const int seg_chunks = (p.k_groups + kChunk - 1) / kChunk;
  const int chunks = p.n_segs * seg_chunks;
  const int c0 = static_cast<int>(static_cast<int64_t>(chunks) * part / splits);
  const int c1 = static_cast<int>(static_cast<int64_t>(chunks) * (part + 1) / splits);
  const int t0 = tt * TN;
  const int w_row0 = nt * BM;
  // An output's operands: its rank's (colwise), or every rank's in turn (rowwise).
  auto w_of = [&](int seg) { return p.n_segs > 1 ? seg : g; };
  auto x_of = [&](int seg) { return p.n_segs > 1 ? seg : 0; };
  // The weights' first box is asked into L2 while the kernel before still ends.  (L2 is where all of
  // the GPU's writes meet: if that kernel writes it, the copy below reads what it wrote.  A token
  // of 2 x 2048 x 1024: 4.17 -> 3.80 us; more boxes than one slow long launches, the one before.)
  __syncwarp();
  if (warp == 0 && elect_one()) {
    ChunkWalk at;
    at.start(c0, seg_chunks);
    prefetch_box(&p.map_w[w_of(at.seg)], at.kg * (KB / 2), w_row0);
    if constexpr (kGlu) prefetch_box(&p.map_w[w_of(at.seg)], at.kg * (KB / 2), p.up_row + w_row0);
  }
  // Tensor memory is taken once the kernel before has ended, and only then may a dependent
  // kernel's CTAs be scheduled: CTAs of two kernels of a stream on one SM could otherwise wait for
  // each other's.
  pdl_wait();
  __syncwarp();  // (here and below: converged for the instructions that a whole warp has to run together)
  if (warp == 0) {
    ptx::tmem_alloc(ptx::smem_addr(&ctl->tmem_base), C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
  pdl_launch_dependents();

  const uint32_t sf_base = ptx::smem_addr(base) + C::RING;
  bool gave_up = false;

  // The producer and the MMA issuer spend a group's 16 KB, at an SM's share of the memory rate
  // some 350 ns, in loops that have to be shorter: addresses are carried along, and the whole
  // warp runs each loop, so that they stay in uniform registers; one lane issues.
  const uint32_t ring = ptx::smem_addr(base);
  const uint32_t full0 = ptx::smem_addr(&ctl->full[0]), empty0 = ptx::smem_addr(&ctl->empty[0]);
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, p.status));
  };
  if (warp == 0) {
    // -------------------------------------------------------------- producer
    const bool issuer = elect_one();
    uint32_t stage = 0, phase = 1, issued = 0;
    ChunkWalk at;
    at.start(c0, seg_chunks);
    bool ok = true;
    for (int c = c0; c < c1 && ok; ++c, at.next(p.k_groups)) {
      const int n = min(kChunk, p.k_groups - at.kg);
      const CUtensorMap* mw = &p.map_w[w_of(at.seg)];
      const CUtensorMap* mx = &p.map_x[x_of(at.seg)];
      const int kx = at.kg * (KB / 2);  // the maps count 2-byte elements
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        if (k < n) {
          if (!wait(empty0 + 8 * stage, phase)) {
            ok = false;
            break;
          }
          if (issuer) {
            const uint32_t full = full0 + 8 * stage, sw = ring + stage * C::STAGE_BYTES;
            ptx::mbar_arrive_expect_tx(full, C::STAGE_BYTES);
            ptx::tma_load_2d(sw, mw, full, kx + k * (KB / 2), w_row0);
            if constexpr (kGlu) ptx::tma_load_2d(sw + kBoxA, mw, full, kx + k * (KB / 2), p.up_row + w_row0);
            ptx::tma_load_2d(sw + C::W_BYTES, mx, full, kx + k * (KB / 2), t0);
          }
          ++issued;
          if (++stage == C::STAGES) stage = 0, phase ^= 1u;
        }
      }
    }
    // Every copy lands before the CTA can exit.
    const uint32_t first = issued > C::STAGES ? issued - C::STAGES : 0;
    for (uint32_t i = first; i < issued; ++i)
      wait_bounded(full0 + 8 * (i % C::STAGES), (i / C::STAGES) & 1u, abort_flag, p.status, true);
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc = idesc_mx(BM, TN);
    const bool issuer = elect_one();
    const uint64_t w0 = ptx::sw128_kmajor_desc(ring);
    const uint32_t sf_full0 = ptx::smem_addr(&ctl->sf_full[0]), sf_empty0 = ptx::smem_addr(&ctl->sf_empty[0]);
    uint64_t wdesc = w0;
    uint32_t stage = 0, phase = 0, accumulate = 0;
    ChunkWalk at;
    at.start(c0, seg_chunks);
    bool ok = true;
    for (int i = 0; i < c1 - c0 && ok; ++i, at.next(p.k_groups)) {
      const int n = min(kChunk, p.k_groups - at.kg);
      const uint32_t buf = i % C::SF_BUFS;
      if (!wait(sf_full0 + 8 * buf, (i / C::SF_BUFS) & 1u)) break;
      const uint32_t sf = tmem + C::ACC_COLS + (i & 1) * C::SF_COLS;
      if (issuer)
#pragma unroll
        for (int a = 0; a <= C::W_TILES; ++a)
          copy_scales<false>(sf + 4 * a, sf_base + buf * C::SF_BYTES + a * kSfRows);
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        if (k < n) {
          if (!wait(full0 + 8 * stage, phase)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          if (issuer) {
            const uint64_t xdesc = wdesc + (C::W_BYTES >> 4);
            const uint32_t id = idesc | idesc_scale_byte(static_cast<uint32_t>(k));
#pragma unroll
            for (int j = 0; j < KB / 32; ++j) {  // +32 bytes along K = +2 in the descriptor's 16-byte units
              umma_mx(tmem, wdesc + 2 * j, xdesc + 2 * j, id, sf, sf + 4 * C::W_TILES, j > 0 ? 1u : accumulate);
              if constexpr (kGlu)
                umma_mx(tmem + TN, wdesc + (kBoxA >> 4) + 2 * j, xdesc + 2 * j, id, sf + 4, sf + 4 * C::W_TILES,
                        j > 0 ? 1u : accumulate);
            }
            ptx::umma_commit(empty0 + 8 * stage);
          }
          accumulate = 1;
          wdesc += C::STAGE_BYTES >> 4;
          if (++stage == C::STAGES) stage = 0, phase ^= 1u, wdesc = w0;
        }
      }
      if (issuer && ok) ptx::umma_commit(sf_empty0 + 8 * buf);
    }
    if (issuer) ptx::umma_commit(ptx::smem_addr(&ctl->done));
    wait_bounded(ptx::smem_addr(&ctl->done), 0, abort_flag, p.status, true);
  } else {
    // -------------------------------------------------------------- scales, then the partial tile
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    const uint32_t quarter = static_cast<uint32_t>(q * 32) << 16;
    const int row = q * 32 + lane;
    uint32_t w_next, u_next = 0, x_next;
    auto load = [&](const ChunkWalk& at) {
      const int n = min(kChunk, p.k_groups - at.kg);
      const uint8_t* sw = p.sw[w_of(at.seg)];
      w_next = load_word<7>(sw, p.k_groups, p.w_rows, w_row0 + row, at.kg, n, p.w_words);
      if constexpr (kGlu) u_next = load_word<7>(sw, p.k_groups, p.w_rows, p.up_row + w_row0 + row, at.kg, n, p.w_words);
      x_next = load_word<0>(p.sx[x_of(at.seg)], p.ld_sx, row < TN ? p.T : 0, t0 + row, at.kg, n, p.x_words);
    };
    ChunkWalk at;
    at.start(c0, seg_chunks);
    load(at);
    for (int i = 0; i < c1 - c0; ++i) {
      const uint32_t buf = i % C::SF_BUFS;
      const uint32_t w = w_next, u = u_next, x = x_next;
      if (i + 1 < c1 - c0) {
        at.next(p.k_groups);
        load(at);
      }
      if (!__all_sync(0xffffffffu, wait_bounded(ptx::smem_addr(&ctl->sf_empty[buf]), ((i / C::SF_BUFS) & 1u) ^ 1u,
                                                abort_flag, p.status))) {
        gave_up = true;
        break;
      }
      const uint32_t words = sf_base + buf * C::SF_BYTES;
      store_word(words, row, w);
      if constexpr (kGlu) store_word(words + kSfRows, row, u);
      store_word(words + C::W_TILES * kSfRows, row, x);
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(ptx::smem_addr(&ctl->sf_full[buf]));
    }
    if (!gave_up)
      gave_up = !__all_sync(0xffffffffu, wait_bounded(ptx::smem_addr(&ctl->done), 0, abort_flag, p.status));
    if (!gave_up) {
      // Every MMA is done, so every copy has landed and the ring is free: it takes the partial
      // tile as [W tile][token][128 weight rows].
      __syncwarp();
      ptx::tc_fence_after();
      float* partial = reinterpret_cast<float*>(base);
#pragma unroll
      for (int j = 0; j < C::ACC_COLS; j += 16) {
        uint32_t v[16];
        ptx::tmem_ld_32x32b_x16(tmem + quarter + j, v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) partial[(j + e) * BM + q * 32 + lane] = __uint_as_float(v[e]);
      }
    }
    ptx::tc_fence_before();
  }
  __syncwarp();
  ptx::cluster_sync();  // every CTA's partial tile is in its shared memory

  // ---------------------------------------------------------------- join, activation, store
  // This CTA's share of the tile's tokens, a warp to a token, four columns to a lane.  A token's
  // reads, sums and store take half a microsecond one after the other, so what can be is in flight
  // together: the reads from all the CTAs that share K, or, with one or two, those of four tokens (with
  // one: gate/up of 256 tokens in this kernel 72 -> 64 us; with two: GELU of 333 tokens, 2 x 1096 x
  // 2000, 10.8 -> 10.1 us; two tokens with three or four: 0.1 to 0.3 us slower).
  if (!*abort_flag) {
    const int tokens = min(TN, p.T - t0);
    const int n0 = w_row0 + lane * 4;
    const bool on = n0 < p.n_out;  // n_out is a multiple of 8
    const bool fp8 = p.out_scales[g] != nullptr;
    float bias[C::W_TILES][4];
#pragma unroll
    for (int a = 0; a < C::W_TILES; ++a)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        bias[a][e] = p.bias[g] != nullptr && on ? __bfloat162float(p.bias[g][n0 + e + (a ? p.up_row : 0)]) : 0.0f;
    const uint32_t local = ptx::smem_addr(base) + static_cast<uint32_t>(lane) * 16;
    const int t_begin = tokens * part / splits, t_end = tokens * (part + 1) / splits;
    constexpr int kWarps = kTokensThreads / 32;
    auto join = [&](auto several, auto sources, int t) {
      constexpr int U = decltype(several)::value;      // tokens t, t + kWarps, ...
      constexpr int kFrom = decltype(sources)::value;  // at least `splits`
      float v[U][C::W_TILES][4];
      // What is not stored (a token past the share, a column past the output) is read from this CTA's own
      // partial tile, the share's first token in place of one past it.  A store waits for its reads, so
      // that none is on its way to another CTA when this one comes to the last barrier, behind which
      // the other's shared memory may be gone.
      auto at = [&](int j, int a, int s) {
        const bool inside = t + j * kWarps < t_end;
        const int tj = inside ? t + j * kWarps : t;
        return ptx::mapa_shared(local + static_cast<uint32_t>(a * TN + tj) * (BM * 4),
                                static_cast<uint32_t>(inside && on ? s : part));
      };
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int a = 0; a < C::W_TILES; ++a)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[j][a][e] = 0.0f;
      auto add = [](float (&to)[4], const float4& f) { to[0] += f.x, to[1] += f.y, to[2] += f.z, to[3] += f.w; };
      float4 f[U][C::W_TILES][kFrom];
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int a = 0; a < C::W_TILES; ++a)
#pragma unroll
          for (int s = 0; s < kFrom; ++s)
            if (s < splits) f[j][a][s] = ld_cluster_f4(at(j, a, s));
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int a = 0; a < C::W_TILES; ++a)
#pragma unroll
          for (int s = 0; s < kFrom; ++s)
            if (s < splits) add(v[j][a], f[j][a][s]);
      float y[U][4];
      uint32_t byte[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = v[j][0][e] + bias[0][e];
          if constexpr (kGlu)
            y[j][e] = silu_f(x) * (v[j][1][e] + bias[1][e]);
          else
            y[j][e] = p.act == TP_ACT_GELU_TANH ? gelu_tanh_f(x) : x;
        }
        if (fp8) {  // the tile's 128 columns are one group of the output
          const float m = max_abs(max_abs(y[j][0], y[j][1]), max_abs(y[j][2], y[j][3]));
          byte[j] = e8m0_of_amax(__reduce_max_sync(0xffffffffu, on ? abs_bits(m) : 0u));
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (t + j * kWarps >= t_end) break;
        const int64_t row = static_cast<int64_t>(t0 + t + j * kWarps);
        if (fp8) {
          const float inv = e8m0_inverse(byte[j]);
          if (on)
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out[g]) + row * p.ldo + n0) =
                e4m3x4(y[j][0] * inv, y[j][1] * inv, y[j][2] * inv, y[j][3] * inv);
          if (lane == 0) p.out_scales[g][row * p.ld_os + nt] = static_cast<uint8_t>(byte[j]);
        } else if (on) {
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out[g]) + row * p.ldo + n0) =
              make_uint2(pack_bf16(y[j][0], y[j][1]), pack_bf16(y[j][2], y[j][3]));
        }
      }
    };
    auto join_all = [&](auto several, auto sources) {
      for (int t = t_begin + warp; t < t_end; t += decltype(several)::value * kWarps) join(several, sources, t);
    };
    if (t_end - t_begin <= kWarps || splits > 2)
      join_all(std::integral_constant<int, 1>{}, std::integral_constant<int, kMaxSplits>{});
    else if (splits == 1)
      join_all(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
    else
      join_all(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
  }
  __syncwarp();            // the stores above are some lanes' only
  cluster_sync_relaxed();  // no CTA's shared memory goes away while another reads it
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- prompts
constexpr int PM = 256;                              // tokens per pair tile
constexpr int PN = 256;                              // accumulator columns (weight rows) per tile
constexpr int kPromptStages = 6;
constexpr uint32_t kPromptStage = 2 * kBoxA;         // a CTA's 128 tokens and its 128 weight rows
constexpr uint32_t kShared = 32;                     // columns the two accumulators share
constexpr uint32_t kPromptSf = 2 * PN - kShared;     // scale words: buffers of 16 columns (X 4, W 8)
constexpr uint32_t kSfTmem = 2;                      // of them, chunks that are in tensor memory at once
constexpr uint32_t kStagingWarp = 32 * 128;          // epilogue staging: 32 rows a warp, 128 codes or 32 bf16 each
constexpr uint32_t kPromptSfBytes = 3 * kSfRows;     // one chunk's words: X, W rows 0..127, W rows 128..255
constexpr int kPromptThreads = 320;                  // producer, MMA issuer, 4 epilogue and 4 scale warps
constexpr uint32_t kPromptBias = PN * 4;             // a tile's bias, in each epilogue warp's own copy
constexpr size_t kPromptSmem =
    1024 + kPromptStages * kPromptStage + 4 * kStagingWarp + kSfBufs * kPromptSfBytes + 4 * kPromptBias;
static_assert(kPromptSf + kSfTmem * 16 <= 512 && kSfTmem <= kSfBufs, "accumulators and scale words fill tensor memory");

struct alignas(8) PromptCtrl {
  uint64_t full[kPromptStages], empty[kPromptStages];
  uint64_t sf_full[kSfBufs], sf_empty[kSfBufs];
  uint64_t sf_peer[kSfBufs];  // the leader's: the other CTA's words are in its shared memory
  uint64_t tfull[2], tempty;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// A work item is a tile, or with clusters of two pairs two adjacent tiles.
__device__ __forceinline__ void decode_item(const Fp8Params& p, int t, int& g, int& mt, int& nt) {
  // group_m token tiles sweep the weight tiles together, so that CTAs that run at the same time
  // share both operands through L2.
  const int per_out = p.t_tiles * p.n_items;
  g = t / per_out;
  const int in_out = t - g * per_out;
  const int span = p.group_m * p.n_items;
  const int first = in_out / span * p.group_m;
  const int m = min(p.group_m, p.t_tiles - first);
  const int in_span = in_out % span;
  mt = first + in_span % m;
  nt = in_span / m;
}

// Copy a warp's 32 staged rows of kPieces 16-byte pieces out, so that a store instruction writes
// whole row segments.  `out` is row 0's first byte, `bytes` what the output has of a row.  A piece
// lies at a place of its 128-byte line that the row turns, so that neither the threads that wrote a
// row each nor these reads meet in a bank.
template <int kPieces>
__device__ __forceinline__ uint32_t staged(uint32_t staging, int row, int piece) {
  const int line = row * kPieces / 8, in_line = row % (8 / kPieces) * kPieces;
  return staging + static_cast<uint32_t>(line * 128 + ((in_line + (piece ^ (line & (kPieces - 1)))) << 4));
}
template <int kPieces>
__device__ __forceinline__ void store_rows(uint8_t* out, int64_t row_bytes, uint32_t staging, int rows, int bytes,
                                           int lane) {
  __syncwarp();
  const int c = lane % kPieces;
#pragma unroll
  for (int i = 0; i < 32; i += 32 / kPieces) {
    const int r = i + lane / kPieces;
    uint32_t w[4];
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(staged<kPieces>(staging, r, c)));
    if (r < rows && 16 * c < bytes)
      *reinterpret_cast<uint4*>(out + r * row_bytes + 16 * c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncwarp();  // the buffer may be written again
}

// A tile's bias as fp32 in a warp's own shared memory, eight columns to a lane (SwiGLU: gate, then
// up); read before the tile's MMAs are done, so that its latency is not the epilogue's.
template <bool kGlu>
__device__ __forceinline__ void stage_bias(const Fp8Params& p, const __nv_bfloat16* bias, int nt, uint32_t bias_at,
                                           int lane) {
  const bool up = kGlu && lane >= 16;
  const int col = kGlu ? nt * BM + (lane & 15) * 8 : nt * PN + lane * 8;
  const __nv_bfloat16* from = bias + (up ? p.up_row : 0) + col;
  float b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) b[e] = col + e < p.n_out ? __bfloat162float(from[e]) : 0.0f;
#pragma unroll
  for (int e = 0; e < 8; e += 4)
    ptx::st_shared_v4(bias_at + static_cast<uint32_t>(lane * 8 + e) * 4, __float_as_uint(b[e]), __float_as_uint(b[e + 1]),
                      __float_as_uint(b[e + 2]), __float_as_uint(b[e + 3]));
  __syncwarp();
}
__device__ __forceinline__ void add_bias(float (&v)[32], uint32_t at) {
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    float b[4];
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(b[0]), "=f"(b[1]), "=f"(b[2]), "=f"(b[3])
                 : "r"(at + 4 * e));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[e + i] += b[i];
  }
}

// One accumulator tile: this thread's row of it, in groups of 128 output columns (SwiGLU: one, from
// 128 gate and 128 up columns; else two), each in four chunks of 32.  The accumulator's columns that
// the other one shares come first (accumulator 0: its last 32, accumulator 1: its first): once they
// are in registers, the next tile's MMAs may start.  A group that leaves as codes needs its largest
// value before the first of them: its activated chunks wait in the accumulator's own columns (the
// first one, whose columns may be gone, in registers).  The loops stay rolled: unrolled over 128
// columns and both accumulators, the code was fetched from memory once per tile (SwiGLU, K 1024:
// 11 us a tile).
template <bool kGlu>
__device__ __forceinline__ void epilogue_tile(const Fp8Params& p, int g, int acc, uint32_t taddr, int nt, int row0,
                                              uint32_t staging, uint32_t bias_at, uint32_t tempty, int lane) {
  uint32_t v[32], keep[32];
  ptx::tmem_ld_32x32b_x32(taddr + (acc == 0 ? PN - kShared : 0), keep);
  ptx::tmem_ld_wait();
  ptx::tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive_cluster_relaxed(tempty);
  __syncwarp();

  const bool biased = p.bias[g] != nullptr, fp8 = p.out_scales[g] != nullptr;
  const int rows = p.T - row0;
#pragma unroll 1
  for (int i = 0; i < (kGlu ? 1 : 2); ++i) {
    const int half = kGlu ? 0 : (acc == 0 ? 1 - i : i);
    const int col0 = kGlu ? nt * BM : nt * PN + 128 * half;
    const uint32_t columns = taddr + 128 * half;
    const uint32_t stash = columns + (kGlu && acc == 1 ? 128 : 0);  // not the shared columns
    const int first = acc == 0 ? 3 : 0;
    if (col0 >= p.n_out) continue;  // uniform
    float largest = 0.0f;
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const int c = (first + k) & 3;
      const int col = col0 + 32 * c;
      float y[32];
      ptx::tmem_ld_32x32b_x32(columns + 32 * c, v);
      if constexpr (kGlu) {
        uint32_t u[32];
        ptx::tmem_ld_32x32b_x32(columns + 128 + 32 * c, u);
        ptx::tmem_ld_wait();
        if (k == 0) {  // one of the two is what was read before
          if (acc == 0)
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = keep[e];
          else
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = keep[e];
        }
        float up[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(v[e]), up[e] = __uint_as_float(u[e]);
        if (biased) {  // uniform
          add_bias(y, bias_at + 4 * (32 * c));
          add_bias(up, bias_at + 4 * (128 + 32 * c));
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = silu_f(y[e]) * up[e];
      } else {
        ptx::tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(i == 0 && k == 0 ? keep[e] : v[e]);
        if (biased) add_bias(y, bias_at + 4 * (128 * half + 32 * c));
        if (p.act == TP_ACT_GELU_TANH)
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = gelu_tanh_f(y[e]);
      }
      if (!fp8) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          ptx::st_shared_v4(staged<4>(staging, lane, e), pack_bf16(y[8 * e], y[8 * e + 1]),
                            pack_bf16(y[8 * e + 2], y[8 * e + 3]), pack_bf16(y[8 * e + 4], y[8 * e + 5]),
                            pack_bf16(y[8 * e + 6], y[8 * e + 7]));
        store_rows<4>(static_cast<uint8_t*>(p.out[g]) + 2 * (row0 * p.ldo + col), 2 * p.ldo, staging, rows,
                      2 * (p.n_out - col), lane);
        continue;
      }
#pragma unroll
      for (int h = 0; h < 32; h += 16)
        if (col + h < p.n_out)  // n_out is a multiple of 16
#pragma unroll
          for (int e = h; e < h + 16; ++e) largest = max_abs(largest, y[e]);
      if (k == 0) {
#pragma unroll
        for (int e = 0; e < 32; ++e) keep[e] = __float_as_uint(y[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(y[e]);
        ptx::tmem_st_32x32b_x32(stash + 32 * c, v);
      }
    }
    if (!fp8) continue;
    ptx::tmem_st_wait();
    const uint32_t byte = e8m0_of_amax(abs_bits(largest));
    const float inv = e8m0_inverse(byte);
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const int c = (first + k) & 3;
      if (k > 0) {
        ptx::tmem_ld_32x32b_x32(stash + 32 * c, v);
        ptx::tmem_ld_wait();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = keep[e];
      }
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e] = e4m3x4(__uint_as_float(v[4 * e]) * inv, __uint_as_float(v[4 * e + 1]) * inv,
                      __uint_as_float(v[4 * e + 2]) * inv, __uint_as_float(v[4 * e + 3]) * inv);
      ptx::st_shared_v4(staged<8>(staging, lane, 2 * c), w[0], w[1], w[2], w[3]);
      ptx::st_shared_v4(staged<8>(staging, lane, 2 * c + 1), w[4], w[5], w[6], w[7]);
    }
    store_rows<8>(static_cast<uint8_t*>(p.out[g]) + row0 * p.ldo + col0, p.ldo, staging, rows, p.n_out - col0, lane);
    if (lane < rows) p.out_scales[g][(row0 + lane) * p.ld_os + col0 / kFp8Group] = static_cast<uint8_t>(byte);
    __syncwarp();
  }
}

// kQuad: clusters of two pairs on n-adjacent tiles, which share X.  Each CTA loads half of its
// tokens and multicasts them to the CTA in its place in the other pair: a quarter less is read
// from L2.  A stage is then free once both pairs' MMAs are done with it.
template <bool kGlu, bool kQuad>
__global__ void __launch_bounds__(kPromptThreads, 1) fp8_prompt_kernel(const __grid_constant__ Fp8Params p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ PromptCtrl ctl_mem;
  PromptCtrl* ctl = &ctl_mem;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort_flag = &ctl->abort;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform to the compiler
  const int lane = threadIdx.x & 31;
  const uint32_t crank = ptx::cluster_ctarank();
  const uint32_t cta = crank & 1u;                  // 0 = the pair's leader
  const uint32_t leader = crank & ~1u;              // its cluster rank
  const uint32_t pair = kQuad ? crank >> 1 : 0u;
  const uint16_t pair_mask = static_cast<uint16_t>(0x3u << (2 * pair));
  constexpr int kCtas = kQuad ? 4 : 2;
  const int unit = static_cast<int>(blockIdx.x) / kCtas;
  const int units = static_cast<int>(gridDim.x) / kCtas;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPromptStages; ++s) {
      ptx::mbar_init(ptx::smem_addr(&ctl->full[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->empty[s]), kQuad ? 2 : 1);
    }
    for (int b = 0; b < kSfBufs; ++b) {
      ptx::mbar_init(ptx::smem_addr(&ctl->sf_full[b]), 128);
      ptx::mbar_init(ptx::smem_addr(&ctl->sf_empty[b]), 1);
      ptx::mbar_init(ptx::smem_addr(&ctl->sf_peer[b]), 1);
    }
    ptx::mbar_init(ptx::smem_addr(&ctl->tfull[0]), 1);
    ptx::mbar_init(ptx::smem_addr(&ctl->tfull[1]), 1);
    ptx::mbar_init(ptx::smem_addr(&ctl->tempty), 8);  // four epilogue warps of each CTA
    ptx::mbar_init(ptx::smem_addr(&ctl->drain), 1);
    ctl->abort = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  __syncwarp();  // (here and below: converged for the instructions that a whole warp has to run together)
  if (warp == 0) {
    ptx::tmem_alloc_pair(ptx::smem_addr(&ctl->tmem_base), 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
  pdl_launch_dependents();
  pdl_wait();

  const uint32_t sf_base = ptx::smem_addr(base) + kPromptStages * kPromptStage + 4 * kStagingWarp;
  const int total = p.n_groups * p.t_tiles * p.n_items;
  // Work item t's output and this pair's tile.
  auto tile_of = [&](int t, int& g, int& mt, int& nt) {
    decode_item(p, t, g, mt, nt);
    if (kQuad) nt = 2 * nt + static_cast<int>(pair);
  };

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      const uint32_t full0 = ptx::smem_addr(&ctl->full[0]), empty0 = ptx::smem_addr(&ctl->empty[0]);
      uint32_t it = 0;  // copies issued
      const uint32_t full0_leader = ptx::mapa_shared(full0, leader);  // both CTAs' copies complete there
      const uint32_t ring = ptx::smem_addr(base);
      const uint32_t half = pair * (kBoxA / 2);                       // the part of a shared box this CTA loads
      const int half_row = static_cast<int>(pair) * (BM / 2);
      const uint16_t both = static_cast<uint16_t>(0x5u << cta);       // this CTA's place in both pairs
      uint32_t stage = 0, phase = 1;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        int g, mt, nt;
        tile_of(t, g, mt, nt);
        const int x_row = mt * PM + static_cast<int>(cta) * BM + half_row;
        const int w_row = kGlu ? (cta == 0 ? 0 : p.up_row) + nt * BM : nt * PN + static_cast<int>(cta) * BM;
        for (int seg = 0; seg < p.n_segs && ok; ++seg) {
          const CUtensorMap* mx = &p.map_x[p.n_segs > 1 ? seg : 0];
          const CUtensorMap* mw = &p.map_w[p.n_segs > 1 ? seg : g];
          int kx = 0;
          for (int k = p.k_groups; k > 0; --k, kx += KB / 2, ++it) {
            if (!wait_bounded(empty0 + 8 * stage, phase, abort_flag, p.status)) {
              ok = false;
              break;
            }
            const uint32_t full = full0_leader + 8 * stage;
            const uint32_t sx = ring + stage * kPromptStage;
            if (cta == 0) ptx::mbar_arrive_expect_tx(full0 + 8 * stage, 2 * kPromptStage);
            if constexpr (kQuad)
              ptx::tma_load_2d_pair_mc(sx + half, mx, full, kx, x_row, both);
            else
              ptx::tma_load_2d_pair(sx, mx, full, kx, x_row);
            ptx::tma_load_2d_pair(sx + kBoxA, mw, full, kx, w_row);
            if (++stage == kPromptStages) stage = 0, phase ^= 1u;
          }
        }
      }
      // Every copy lands before the CTAs can exit; the leader's barriers count both CTAs' copies.
      const uint32_t first = it > kPromptStages ? it - kPromptStages : 0;
      if (cta == 0) {
        for (uint32_t j = first; j < it; ++j)
          wait_bounded(ptx::smem_addr(&ctl->full[j % kPromptStages]), (j / kPromptStages) & 1u, abort_flag, p.status,
                       true);
      } else if (*abort_flag) {
        // The peer cannot observe its own copies; give any in flight time to land (give-up path only).
        const uint64_t t0 = ptx::globaltimer_ns();
        while (ptx::globaltimer_ns() - t0 < 100000ull) {
        }
      }
      // And so does every arrival that hands a stage back (from another CTA's MMA thread, kQuad: from both
      // pairs'): none is on its way here when this CTA's shared memory goes.
      for (uint32_t j = first; j < it; ++j)
        if (!wait_bounded<true>(empty0 + 8 * (j % kPromptStages), (j / kPromptStages) & 1u, abort_flag, p.status)) break;
    }
  } else if (warp == 1) {
    if (cta == 0) {
      // ------------------------------------------------------------ MMA issuer (leader)
      // A group's four MMAs run in 512 cycles, and the loop has to issue them in less: it carries
      // its addresses along (computed from the stage number, the loop took 690 cycles a group and
      // bounded the kernel), and the whole warp runs it, so that they stay in uniform registers;
      // one lane issues.
      const bool issuer = elect_one();
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, p.status));
      };
      constexpr uint32_t idesc = idesc_mx(PM, PN);
      const uint64_t x0 = ptx::sw128_kmajor_desc(ptx::smem_addr(base));
      const uint32_t full0 = ptx::smem_addr(&ctl->full[0]), empty0 = ptx::smem_addr(&ctl->empty[0]);
      const uint32_t sf_full0 = ptx::smem_addr(&ctl->sf_full[0]), sf_empty0 = ptx::smem_addr(&ctl->sf_empty[0]);
      const uint32_t sf_peer0 = ptx::smem_addr(&ctl->sf_peer[0]);
      uint32_t stage = 0, phase = 0, chunk = 0, tile = 0;
      uint64_t xdesc = x0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units, ++tile) {
        // The shared columns are back from the tile before; the rest of this accumulator was read
        // before that, by the same threads.
        if (tile > 0 && !__all_sync(0xffffffffu, wait_bounded<true>(ptx::smem_addr(&ctl->tempty), (tile - 1) & 1u,
                                                                    abort_flag, p.status)))
          break;
        ptx::tc_fence_after();
        const uint32_t acc = tmem + (tile & 1u) * (PN - kShared);
        uint32_t accumulate = 0;
        for (int seg = 0; seg < p.n_segs && ok; ++seg) {
          for (int left = p.k_groups; left > 0; left -= kChunk, ++chunk) {
            const uint32_t buf = chunk % kSfBufs;
            if (!wait(sf_full0 + 8 * buf, (chunk / kSfBufs) & 1u) ||
                !__all_sync(0xffffffffu, wait_bounded<true>(sf_peer0 + 8 * buf, (chunk / kSfBufs) & 1u, abort_flag,
                                                            p.status))) {
              ok = false;
              break;
            }
            // Copies are in order with the MMAs behind them, but nothing orders them with those before: the
            // chunk whose words these replace has to be done (one chunk's MMAs are queued meanwhile).
            if (chunk >= kSfTmem &&
                !wait(sf_empty0 + 8 * ((chunk - kSfTmem) % kSfBufs), ((chunk - kSfTmem) / kSfBufs) & 1u)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            const uint32_t sf = tmem + kPromptSf + chunk % kSfTmem * 16;
            if (issuer)
#pragma unroll
              for (int a = 0; a < 3; ++a)
                copy_scales<true>(sf + 4 * a, sf_base + buf * kPromptSfBytes + a * kSfRows);
#pragma unroll
            for (int k = 0; k < kChunk; ++k) {
              if (k < left) {
                if (!wait(full0 + 8 * stage, phase)) {
                  ok = false;
                  break;
                }
                ptx::tc_fence_after();
                if (issuer) {
#pragma unroll
                  for (int j = 0; j < KB / 32; ++j)
                    umma_mx_pair(acc, xdesc + 2 * j, xdesc + (kBoxA >> 4) + 2 * j,
                                 idesc | idesc_scale_byte(static_cast<uint32_t>(k)), sf, sf + 4, j > 0 ? 1u : accumulate);
                  ptx::umma_commit_pair(empty0 + 8 * stage, kQuad ? 0xF : 0x3);
                }
                accumulate = 1;
                xdesc += kPromptStage >> 4;
                if (++stage == kPromptStages) stage = 0, phase ^= 1u, xdesc = x0;
              }
            }
            if (!ok) break;
            if (issuer) ptx::umma_commit_pair(sf_empty0 + 8 * buf, pair_mask);
          }
        }
        if (!ok) break;
        if (issuer) ptx::umma_commit_pair(ptx::smem_addr(&ctl->tfull[tile & 1u]), pair_mask);
      }
      if (issuer) ptx::umma_commit_pair(ptx::smem_addr(&ctl->drain), pair_mask);
      wait_bounded<true>(ptx::smem_addr(&ctl->drain), 0, abort_flag, p.status, true);
    } else if (lane == 0) {
      // The peer tells the leader when its own scale words are there.  The threads that store them
      // release them to this lane in their own CTA, and this lane, which has seen that, releases
      // them at cluster scope.  (From the threads themselves such a release first waits for their loads of
      // the next words, 1.5 us, longer than a chunk's MMAs: down of 256 tokens 63 us, by way of this
      // lane, which loads nothing, 48.  An asynchronous store whose bytes complete on the leader's
      // barrier took 45, but releases no more than its own word.)
      const uint32_t to = ptx::mapa_shared(ptx::smem_addr(&ctl->sf_peer[0]), leader);
      const int tile_chunks = p.n_segs * ((p.k_groups + kChunk - 1) / kChunk);
      uint32_t buf = 0, phase = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        for (int i = 0; i < tile_chunks; ++i) {
          if (!wait_bounded(ptx::smem_addr(&ctl->sf_full[buf]), phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          ptx::mbar_arrive_cluster(to + 8 * buf);
          if (++buf == kSfBufs) buf = 0, phase ^= 1u;
        }
      }
      // Its shared memory feeds the leader's MMAs until the drain arrives.
      wait_bounded<true>(ptx::smem_addr(&ctl->drain), 0, abort_flag, p.status, true);
    }
  } else if (warp < 6) {
    // -------------------------------------------------------------- epilogue: a row to a thread
    const int q = warp & 3;
    const uint32_t quarter = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t staging = ptx::smem_addr(base) + kPromptStages * kPromptStage +
                             static_cast<uint32_t>(warp - 2) * kStagingWarp;
    const uint32_t bias_at = sf_base + kSfBufs * kPromptSfBytes + static_cast<uint32_t>(warp - 2) * kPromptBias;
    const uint32_t tempty = ptx::mapa_shared(ptx::smem_addr(&ctl->tempty), leader);
    uint32_t tile = 0;
    for (int t = unit; t < total; t += units, ++tile) {
      int g, mt, nt;
      tile_of(t, g, mt, nt);
      if (p.bias[g] != nullptr) stage_bias<kGlu>(p, p.bias[g], nt, bias_at, lane);
      if (!__all_sync(0xffffffffu, wait_bounded<true>(ptx::smem_addr(&ctl->tfull[tile & 1u]), (tile >> 1) & 1u,
                                                      abort_flag, p.status)))
        break;
      __syncwarp();
      ptx::tc_fence_after();
      const int row0 = mt * PM + static_cast<int>(cta) * BM + q * 32;
      const int acc = static_cast<int>(tile & 1u);
      epilogue_tile<kGlu>(p, g, acc, tmem + quarter + static_cast<uint32_t>(acc) * (PN - kShared), nt, row0, staging,
                          bias_at, tempty, lane);
    }
  } else {
    // -------------------------------------------------------------- scale words
    const int row = (warp & 3) * 32 + lane;
    uint32_t x_next = 0, w0_next = 0, w1_next = 0;
    int t = unit, g = 0, mt = 0, nt = 0;
    auto load = [&](const ChunkWalk& at) {
      const int n = min(kChunk, p.k_groups - at.kg);
      const uint8_t* sw = p.sw[p.n_segs > 1 ? at.seg : g];
      const int w_row = kGlu ? nt * BM : nt * PN;
      x_next = load_word<0>(p.sx[p.n_segs > 1 ? at.seg : 0], p.ld_sx, p.T, mt * PM + static_cast<int>(cta) * BM + row,
                            at.kg, n, p.x_words);
      w0_next = load_word<7>(sw, p.k_groups, p.w_rows, w_row + row, at.kg, n, p.w_words);
      w1_next = load_word<7>(sw, p.k_groups, p.w_rows, w_row + (kGlu ? p.up_row : BM) + row, at.kg, n, p.w_words);
    };
    ChunkWalk at{0, 0};
    if (t < total) {
      tile_of(t, g, mt, nt);
      load(at);
    }
    uint32_t chunk = 0;
    bool ok = true;
    for (; t < total; ++chunk) {
      const uint32_t buf = chunk % kSfBufs;
      const uint32_t x = x_next, w0 = w0_next, w1 = w1_next;
      at.next(p.k_groups);
      if (at.seg == p.n_segs) {  // on to the next tile
        at = ChunkWalk{0, 0};
        t += units;
        if (t < total) tile_of(t, g, mt, nt);
      }
      if (t < total) load(at);
      if (!__all_sync(0xffffffffu, wait_bounded<true>(ptx::smem_addr(&ctl->sf_empty[buf]),
                                                      ((chunk / kSfBufs) & 1u) ^ 1u, abort_flag, p.status))) {
        ok = false;
        break;
      }
      const uint32_t words = sf_base + buf * kPromptSfBytes;
      store_word(words, row, x);
      store_word(words + kSfRows, row, w0);
      store_word(words + 2 * kSfRows, row, w1);
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(ptx::smem_addr(&ctl->sf_full[buf]));
    }
    // The arrivals that hand the last buffers back, as the stages' above.
    for (uint32_t j = chunk > kSfBufs ? chunk - kSfBufs : 0; j < chunk && ok; ++j)
      ok = wait_bounded<true>(ptx::smem_addr(&ctl->sf_empty[j % kSfBufs]), (j / kSfBufs) & 1u, abort_flag, p.status);
  }
  __syncwarp();
  ptx::tc_fence_before();
  ptx::cluster_sync();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

inline int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// Operand map over a row-major [rows, K] matrix of bytes: boxes of 128 bytes x box_rows, 128-byte
// swizzle, zeros outside.  Encoded as 2-byte elements (K and the stride are multiples of 16).
tp_status operand_map(CUtensorMap* m, const void* ptr, int64_t K, int64_t rows, int64_t ld, int box_rows) {
  return encode_bf16_2d_now(m, ptr, K / 2, rows, ld / 2, KB / 2, static_cast<uint32_t>(box_rows));
}

// The operands of a call, checked.
struct Fp8Call {
  const void* const* x;         // one (shared) or tp_degree
  const void* const* sx;
  bool x_shared;
  int64_t ldx, ld_sx;
  const void* const* w;
  const void* const* sw;
  int p;
  int64_t T, K, w_rows, n_out;
};

// The maps of X and W in boxes of x_box and w_box rows.
tp_status set_maps(const Fp8Call& c, Fp8Params& p, int x_box, int w_box) {
  for (int r = 0; r < c.p; ++r) {
    tp_status st = operand_map(&p.map_w[r], c.w[r], c.K, c.w_rows, c.K, w_box);
    if (st == TP_OK && (r == 0 || !c.x_shared)) st = operand_map(&p.map_x[r], c.x[r], c.K, c.T, c.ldx, x_box);
    if (st != TP_OK) return st;
  }
  return TP_OK;
}

// Clusters of `size` CTAs of a kernel that can be resident at once, as the runtime counts them (0: no such
// cluster on this device).  It counts one CTA an SM for the small tokens kernels too, of which two fit:
// 152 / 76 / 46 / 36 / 28 / 23 / 15 / 15 clusters of 1 to 8.
template <typename Kernel>
int resident_clusters(Kernel kernel, int size, int threads, size_t smem) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(size) * 64, 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(size);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 0) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

// What a kernel's first call on a device finds out, for the later ones.
struct Residency {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  int clusters[kMaxSplits + 1] = {0};  // by cluster size
};
tp_status current_device_index(int* dev) {
  const cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (*dev < 0 || *dev >= 64) return fail(TP_ERR_UNSUPPORTED, "device index %d", *dev);
  return TP_OK;
}

// The tokens kernel's resident clusters by size.
template <int TN, bool kGlu>
tp_status tokens_residency(const int** clusters) {
  static Residency found[64];
  int dev = 0;
  tp_status st = current_device_index(&dev);
  if (st != TP_OK) return st;
  Residency& r = found[dev];
  std::call_once(r.once, [&] {
    r.err = cudaFuncSetAttribute(fp8_tokens_kernel<TN, kGlu>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(TokensCfg<TN, kGlu>::SMEM));
    for (int s = 1; s <= kMaxSplits && r.err == cudaSuccess; ++s)
      r.clusters[s] =
          resident_clusters(fp8_tokens_kernel<TN, kGlu>, s, kTokensThreads, TokensCfg<TN, kGlu>::SMEM);
  });
  if (r.err != cudaSuccess) return cuda_fail(r.err, "cudaFuncSetAttribute(max dynamic shared memory)");
  *clusters = r.clusters;
  return TP_OK;
}

template <int TN, bool kGlu>
tp_status launch_tokens(const Fp8Call& c, Fp8Params& p, cudaStream_t stream) {
  const int chunks = p.n_segs * ceil_div(p.k_groups, kChunk);
  p.n_tiles = ceil_div(p.n_out, BM);
  const int64_t tiles = static_cast<int64_t>(p.n_groups) * p.n_tiles * p.t_tiles;
  // The split of K whose longest SM is shortest: waves x (a CTA's chunks + the fixed part of its
  // life, about 4 us or three chunks; with 128 tokens to join, six).  Ties go to the smaller
  // cluster.  Measured, down projection of one token (4 x 6144 x 4608, 36 chunks, 48 tiles): splits
  // 1 / 2 / 3 / 4 / 5 / 6 / 8 take 29.9 / 22.0 / 21.2 / 20.6 / 20.7 / 26.3 / 24.7 us (from 6 on the
  // clusters need a second wave; the rule, which counts one CTA an SM, takes 2); of 256 tokens (96
  // tiles): 36.4 / 43.7 / 50.1 / 44.1 / 52.0 / 56.4 / 72.0, of 512 (192 tiles): 70.1 / 64.8 / 81.8 / 81.9
  // and more.
  constexpr int kFixed = TN > 64 ? 6 : 3;
  const int* resident = nullptr;
  tp_status st = tokens_residency<TN, kGlu>(&resident);
  if (st != TP_OK) return st;
  int best = 0;
  int64_t best_cost = 0;
  for (int s = 1; s <= kMaxSplits && s <= chunks; ++s) {
    const int n = resident[s];
    if (n < 1) continue;
    const int64_t cost = ((tiles + n - 1) / n) * (ceil_div(chunks, s) + kFixed);
    if (best == 0 || cost < best_cost) best = s, best_cost = cost;
  }
  if (best == 0) return fail(TP_ERR_UNSUPPORTED, "the kernel does not fit on this device");
  if (tiles * best > 0x7FFFFFFF) return fail(TP_ERR_UNSUPPORTED, "too many tiles (%lld)", (long long)tiles);
  p.splits = best;
  st = set_maps(c, p, TN, BM);
  if (st != TP_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * best), 1, 1);
  cfg.blockDim = dim3(kTokensThreads, 1, 1);
  cfg.dynamicSmemBytes = TokensCfg<TN, kGlu>::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(best);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_tokens_kernel<TN, kGlu>, p);
  if (e != cudaSuccess) return cuda_fail(e, "fp8 projection launch");
  return TP_OK;
}

// The prompt kernel's resident pairs, or clusters of two pairs.
template <bool kGlu, bool kQuad>
tp_status resident_prompt(int* n) {
  static Residency found[64];
  int dev = 0;
  tp_status st = current_device_index(&dev);
  if (st != TP_OK) return st;
  Residency& r = found[dev];
  std::call_once(r.once, [&] {
    r.err = cudaFuncSetAttribute(fp8_prompt_kernel<kGlu, kQuad>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kPromptSmem));
    if (r.err == cudaSuccess)
      r.clusters[0] = resident_clusters(fp8_prompt_kernel<kGlu, kQuad>, kQuad ? 4 : 2, kPromptThreads, kPromptSmem);
  });
  if (r.err != cudaSuccess) return cuda_fail(r.err, "cudaFuncSetAttribute(max dynamic shared memory)");
  *n = r.clusters[0];
  return TP_OK;
}

template <bool kGlu, bool kQuad>
tp_status launch_prompt(Fp8Params& p, int clusters, cudaStream_t stream) {
  const int64_t items = static_cast<int64_t>(p.n_groups) * p.t_tiles * p.n_items;
  if (items > 0x7FFFFFFF) return fail(TP_ERR_UNSUPPORTED, "too many tiles (%lld)", (long long)items);
  if (items < clusters) clusters = static_cast<int>(items);
  constexpr unsigned kCtas = kQuad ? 4 : 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kCtas * static_cast<unsigned>(clusters), 1, 1);
  cfg.blockDim = dim3(kPromptThreads, 1, 1);
  cfg.dynamicSmemBytes = kPromptSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_prompt_kernel<kGlu, kQuad>, p);
  if (e != cudaSuccess) return cuda_fail(e, "fp8 projection launch");
  return TP_OK;
}

// Token tiles that sweep the weight tiles together: all of them while their operand fits L2
// comfortably (each weight tile is then read from HBM once), else groups of about 16, evenly sized.
int choose_group_m(int t_tiles, int64_t x_bytes) {
  if (x_bytes <= (64ll << 20)) return t_tiles;
  const int groups = ceil_div(t_tiles, 16);
  return ceil_div(t_tiles, groups);
}

template <bool kGlu>
tp_status run_prompt(const Fp8Call& c, Fp8Params& p, cudaStream_t stream) {
  p.n_tiles = ceil_div(c.n_out, kGlu ? BM : PN);
  p.t_tiles = ceil_div(c.T, PM);
  int pairs = 0, quads = 0;
  tp_status st = resident_prompt<kGlu, false>(&pairs);
  if (st == TP_OK) st = resident_prompt<kGlu, true>(&quads);
  if (st != TP_OK) return st;
  if (pairs < 1) return fail(TP_ERR_UNSUPPORTED, "no CTA pair of the kernel fits on this device");
  // Clusters of two pairs, on n-adjacent tiles that share X, where the tiles pair up and the
  // clusters' waves, each about 3 % shorter, take no longer than the pairs' (fewer clusters of
  // four CTAs than pairs fit: 36 x 4 against 76 x 2).  Measured in 3 s each at the power limit:
  // gate/up of 4608 tokens 647 us against 655 (36 waves, 35 of pairs), down 338 against 343.5 (6
  // waves either way), of 2048 tokens 158 against 161.5 (3 either way).
  const int64_t tiles = static_cast<int64_t>(p.n_groups) * p.n_tiles * p.t_tiles;
  bool quad = quads > 0 && p.n_tiles % 2 == 0;
  if (quad) {
    const int64_t waves_quad = (tiles / 2 + quads - 1) / quads, waves_pair = (tiles + pairs - 1) / pairs;
    quad = waves_quad * 32 <= waves_pair * 33;
  }
  p.n_items = quad ? p.n_tiles / 2 : p.n_tiles;
  p.group_m = choose_group_m(p.t_tiles, c.T * c.K * p.n_segs);
  st = set_maps(c, p, quad ? BM / 2 : BM, BM);
  if (st != TP_OK) return st;
  return quad ? launch_prompt<kGlu, true>(p, quads, stream) : launch_prompt<kGlu, false>(p, pairs, stream);
}

template <int TN>
tp_status run_tokens(const Fp8Call& c, Fp8Params& p, cudaStream_t stream) {
  p.t_tiles = ceil_div(c.T, TN);
  return p.act == TP_ACT_SWIGLU ? launch_tokens<TN, true>(c, p, stream) : launch_tokens<TN, false>(c, p, stream);
}

// Whether 256 x 256 tiles on CTA pairs beat 128 x 128 tiles on single CTAs, by what both took (ns): a
// wave of single CTAs 6000 and 230 a scale group of the CTAs' share (SwiGLU 28 more a token of the
// tile, and 400), a launch of pairs 6500 and 260 a group and wave.  Measured (us, single against
// pairs): Q/K/V of 128 / 192 / 384 tokens 25.1 / 36.2 / 52.6 against 26.2 / 26.7 / 38.5; down of 256 /
// 384 / 512 tokens 36.4 / 37.9 / 63.4 against 48.0 / 47.6 / 48.2; 2 x 2048 x 1024 of 256 / 512 / 768
// tokens 7.1 / 8.8 / 16.4 against 8.6 / 8.7 / 9.2; SwiGLU 4096 x 512 of 65 / 128 tokens 8.5 / 11.5
// against 8.2 / 8.1, 2 x 2048 x 2048 of 96 / 300 tokens 9.1 / 12.1 against 11.5 / 11.7.
bool prompt_is_faster(const Fp8Params& p, const Fp8Call& c) {
  const bool glu = p.act == TP_ACT_SWIGLU;
  const int64_t sms = sm_count(), groups = static_cast<int64_t>(p.n_segs) * p.k_groups;
  if (sms < 2) return false;
  const int64_t single = static_cast<int64_t>(p.n_groups) * ceil_div(c.n_out, BM) * ceil_div(c.T, 128);
  const int64_t paired = static_cast<int64_t>(p.n_groups) * ceil_div(c.n_out, glu ? BM : PN) * ceil_div(c.T, PM);
  const int64_t chunks = (groups + kChunk - 1) / kChunk;
  const int64_t splits = std::max<int64_t>(1, std::min<int64_t>({kMaxSplits, chunks, sms / single}));
  const int64_t share = (groups + splits - 1) / splits;
  const int64_t wave = 6000 + (glu ? 28 * std::min<int64_t>(c.T, 128) + share * 400 : share * 230);
  const int64_t t_single = (single + sms - 1) / sms * wave;
  const int64_t t_paired = 6500 + (paired + sms / 2 - 1) / (sms / 2) * groups * 260;
  return t_paired < t_single;
}

tp_status run_fp8(const Fp8Call& c, Fp8Params& p, cudaStream_t stream) {
  p.status = status_word();
  if (p.status == nullptr) return fail(TP_ERR_CUDA, "cannot locate the kernel status word");
  p.ld_sx = c.ld_sx;
  p.T = static_cast<int>(c.T);
  p.w_rows = static_cast<int>(c.w_rows);
  p.n_out = static_cast<int>(c.n_out);
  p.up_row = static_cast<int>(c.w_rows / 2);
  p.k_groups = ceil_div(c.K, KB);
  auto word_rows = [](const void* q, int64_t ld) { return (reinterpret_cast<uintptr_t>(q) & 3u) == 0 && ld % 4 == 0; };
  p.x_words = p.w_words = p.k_groups % kChunk == 0;
  for (int r = 0; r < c.p; ++r) {
    p.sw[r] = static_cast<const uint8_t*>(c.sw[r]);
    p.w_words = p.w_words && word_rows(p.sw[r], p.k_groups);
    if (r == 0 || !c.x_shared) {
      p.sx[r] = static_cast<const uint8_t*>(c.sx[r]);
      p.x_words = p.x_words && word_rows(p.sx[r], c.ld_sx);
    }
  }
  if (c.T > 64 && prompt_is_faster(p, c))
    return p.act == TP_ACT_SWIGLU ? run_prompt<true>(c, p, stream) : run_prompt<false>(c, p, stream);
  if (c.T <= 16) return run_tokens<16>(c, p, stream);
  if (c.T <= 32) return run_tokens<32>(c, p, stream);
  if (c.T <= 64) return run_tokens<64>(c, p, stream);
  return run_tokens<128>(c, p, stream);
}

// What both entry points check of their operands.
tp_status check_fp8(const Fp8Call& c) {
  if (c.x == nullptr || c.sx == nullptr || c.w == nullptr || c.sw == nullptr)
    return fail(TP_ERR_INVALID_ARG, "an operand array or its scales is NULL");
  if (c.K % 16 != 0 || c.ldx % 16 != 0)
    return fail(TP_ERR_ALIGNMENT, "in_features (%lld) and the input's row stride (%lld) must be multiples of 16",
                (long long)c.K, (long long)c.ldx);
  for (int r = 0; r < c.p; ++r) {
    const int xr = c.x_shared ? 0 : r;
    if (c.x[xr] == nullptr || c.sx[xr] == nullptr || c.w[r] == nullptr || c.sw[r] == nullptr)
      return fail(TP_ERR_INVALID_ARG, "rank %d: an operand or its scales is NULL", r);
    if (!aligned16(c.x[xr]) || !aligned16(c.w[r]))
      return fail(TP_ERR_ALIGNMENT, "rank %d: the input or the weight is not 16-byte aligned", r);
  }
  return TP_OK;
}

// bf16 elements one at a time, so that a bias may start at any of them (but not inside one).
tp_status check_bias(const void* bias, int r) {
  if ((reinterpret_cast<uintptr_t>(bias) & 1u) != 0)
    return fail(TP_ERR_ALIGNMENT, "bias %d is not 2-byte aligned", r);
  return TP_OK;
}

tp_status check_sizes(int tp_degree, int64_t T, int64_t K, int64_t N) {
  if (tp_degree < 1) return fail(TP_ERR_INVALID_ARG, "tp_degree must be >= 1, got %d", tp_degree);
  if (tp_degree > TP_MAX_DEGREE)
    return fail(TP_ERR_UNSUPPORTED, "tp_degree=%d above TP_MAX_DEGREE=%d", tp_degree, TP_MAX_DEGREE);
  if (T < 0 || K < 0 || N < 0) return fail(TP_ERR_INVALID_ARG, "negative size");
  if (T > 0x7FFFFF00 || N > 0x7FFFFF00 || K > 0x7FFFFF00)
    return fail(TP_ERR_UNSUPPORTED, "sizes above 2^31-256 are not supported");
  return TP_OK;
}

}  // namespace
}  // namespace tp

extern "C" {

tp_status tp_linear_colwise_fp8(const void* x, int64_t ldx, const void* x_scales, int64_t ld_xs,
                                const void* const* w_shards, const void* const* w_scales,
                                const void* const* bias_shards, tp_act act, int tp_degree, int64_t T, int64_t K,
                                int64_t N_r, void* const* y_shards, int64_t ldy, void* const* y_scales, int64_t ld_ys,
                                tp_stream_t stream) {
  using namespace tp;
  return guarded([&]() -> tp_status {
    clear_error();
    tp_status st = check_sizes(tp_degree, T, K, N_r);
    if (st != TP_OK) return st;
    if (act != TP_ACT_NONE && act != TP_ACT_GELU_TANH && act != TP_ACT_SWIGLU)
      return fail(TP_ERR_INVALID_ARG, "unknown activation %d", (int)act);
    if (act == TP_ACT_SWIGLU && (N_r % 2) != 0)
      return fail(TP_ERR_INVALID_ARG, "SwiGLU needs an even shard width ([gate_r; up_r]), got N_r=%lld", (long long)N_r);
    const int64_t n_out = (act == TP_ACT_SWIGLU) ? N_r / 2 : N_r;
    const int64_t k_groups = ceil_div(K, KB), out_groups = ceil_div(n_out, KB);
    if (ldx == 0) ldx = K;
    if (ld_xs == 0) ld_xs = k_groups;
    if (ldy == 0) ldy = n_out;
    if (ld_ys == 0) ld_ys = out_groups;
    if (ldx < K || ld_xs < k_groups || ldy < n_out || ld_ys < out_groups)
      return fail(TP_ERR_INVALID_ARG, "a row stride (ldx %lld, ld_xs %lld, ldy %lld, ld_ys %lld) is smaller than its row",
                  (long long)ldx, (long long)ld_xs, (long long)ldy, (long long)ld_ys);
    if (T == 0 || N_r == 0) return TP_OK;
    if (K == 0) return fail(TP_ERR_INVALID_ARG, "K (in_features) must be positive");
    const void* xs[1] = {x};
    const void* sxs[1] = {x_scales};
    Fp8Call c{xs, sxs, true, ldx, ld_xs, w_shards, w_scales, tp_degree, T, K, N_r, n_out};
    st = check_fp8(c);
    if (st != TP_OK) return st;
    if (y_shards == nullptr) return fail(TP_ERR_INVALID_ARG, "y_shards is NULL");
    const int64_t step = y_scales != nullptr ? 16 : 8;
    if (n_out % step != 0 || ldy % step != 0)
      return fail(TP_ERR_ALIGNMENT, "output width (%lld) and ldy (%lld) must be multiples of %lld", (long long)n_out,
                  (long long)ldy, (long long)step);
    Fp8Params p{};
    for (int r = 0; r < tp_degree; ++r) {
      if (y_shards[r] == nullptr || (y_scales != nullptr && y_scales[r] == nullptr))
        return fail(TP_ERR_INVALID_ARG, "y_shards[%d] or y_scales[%d] is NULL", r, r);
      if (!aligned16(y_shards[r])) return fail(TP_ERR_ALIGNMENT, "y_shards[%d] is not 16-byte aligned", r);
      p.out[r] = y_shards[r];
      p.out_scales[r] = y_scales != nullptr ? static_cast<uint8_t*>(y_scales[r]) : nullptr;
      p.bias[r] = bias_shards != nullptr ? static_cast<const __nv_bfloat16*>(bias_shards[r]) : nullptr;
      st = check_bias(p.bias[r], r);
      if (st != TP_OK) return st;
    }
    p.act = act;
    p.n_groups = tp_degree;
    p.n_segs = 1;
    p.ldo = ldy;
    p.ld_os = ld_ys;
    return run_fp8(c, p, reinterpret_cast<cudaStream_t>(stream));
  });
}

tp_status tp_linear_rowwise_fp8(const void* const* x_shards, int64_t ldx, const void* const* x_scales, int64_t ld_xs,
                                const void* const* w_shards, const void* const* w_scales, const void* bias,
                                int tp_degree, int64_t T, int64_t K_r, int64_t N, void* out, int64_t ldo,
                                tp_stream_t stream) {
  using namespace tp;
  return guarded([&]() -> tp_status {
    clear_error();
    tp_status st = check_sizes(tp_degree, T, K_r, N);
    if (st != TP_OK) return st;
    const int64_t k_groups = ceil_div(K_r, KB);
    if (ldx == 0) ldx = K_r;
    if (ld_xs == 0) ld_xs = k_groups;
    if (ldo == 0) ldo = N;
    if (ldx < K_r || ld_xs < k_groups || ldo < N)
      return fail(TP_ERR_INVALID_ARG, "a row stride (ldx %lld, ld_xs %lld, ldo %lld) is smaller than its row",
                  (long long)ldx, (long long)ld_xs, (long long)ldo);
    if (T == 0 || N == 0) return TP_OK;
    if (K_r == 0) return fail(TP_ERR_INVALID_ARG, "K_r (in_features per rank) must be positive");
    if (static_cast<int64_t>(tp_degree) * k_groups > 0x7FFFFFFF)
      return fail(TP_ERR_UNSUPPORTED, "too many K groups (%d ranks of %lld)", tp_degree, (long long)k_groups);
    Fp8Call c{x_shards, x_scales, false, ldx, ld_xs, w_shards, w_scales, tp_degree, T, K_r, N, N};
    st = check_fp8(c);
    if (st != TP_OK) return st;
    if (out == nullptr) return fail(TP_ERR_INVALID_ARG, "out is NULL");
    if (N % 8 != 0 || ldo % 8 != 0)
      return fail(TP_ERR_ALIGNMENT, "N (%lld) and ldo (%lld) must be multiples of 8", (long long)N, (long long)ldo);
    if (!aligned16(out)) return fail(TP_ERR_ALIGNMENT, "out is not 16-byte aligned");
    st = check_bias(bias, 0);
    if (st != TP_OK) return st;
    Fp8Params p{};
    p.out[0] = out;
    p.bias[0] = static_cast<const __nv_bfloat16*>(bias);
    p.act = TP_ACT_NONE;
    p.n_groups = 1;
    p.n_segs = tp_degree;
    p.ldo = ldo;
    return run_fp8(c, p, reinterpret_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
