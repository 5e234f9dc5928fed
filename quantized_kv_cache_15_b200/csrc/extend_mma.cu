// Attention of several new tokens per sequence on the 5th-generation tensor cores
// (block codecs, F16 pages and the raw tail).
//
// A unit's rows (queries x query heads of one kv head, N = 16, 32 or 64 of them) meet a
// tile of 128 positions in two products with the positions or the channels on the
// M = 128 side, so that few rows cost little:
//
//   S^T = K Q^T    [128 positions x N]    A = K (tensor memory), B = Q (shared memory)
//   O^T += V^T P^T [128 channels x 2N]    A = V^T, B = P^T (shared memory)
//
// Keys enter as their integer codes, exact in fp16: a block's 32 channels have their own
// accumulators, and the block scales are applied to the four partial scores in fp32,
//   s = f sum_b (d_b S_b + m_b sum_{c in b} q_c)     (m_b: the _1 codecs' minimum),
// so dequantizing a key value costs an unpack and one subtraction.  The query
// q' = R (s_k * q) is scaled by a power of two into fp16's range and split into two fp16
// halves (22 bits; f undoes the power and applies the softmax scale in log2 units).
// Values enter as d c (+ m) rounded once to fp16, the largest rounding of the kernel
// (2^-11 of a value); the softmax weights as two fp16 halves side by side in N (22 bits),
// which costs the tensor cores nothing where a product is bound by reading its A operand.
// Raw rows (tail, F16 pages) enter as they are, with the raw query.
//
// Roles (32 (4 SW + 6) threads; SW = N / 16 score warpgroups of 16 rows each):
//   score warps   thread = position: unpack that position's key codes into tensor memory,
//                 read its scores, 2^(s - m) into the P image; per-thread sums.  The running
//                 maximum moves only when a score passes it by 8 (log2 units), found by
//                 one barrier vote a tile; then the group's O columns are rescaled.
//   value warps   dequantize value rows into the V image (128-byte swizzle);
//   producer      one bulk copy per page-head into a ring of page stages, running ahead
//                 over tiles and units;
//   MMA warp      one thread issues both products, S of the next tile before P V.
#include "extend.h"

#include "ptx.cuh"
#include "quant.cuh"
#include "tensor.cuh"

namespace kvq {

namespace {

constexpr float EXM_RESCALE = 8.0f;
constexpr int EXM_SMEM_MAX = 232448;                     // 227 KiB opt-in per CTA

template <int N>
struct Shape {
  static constexpr int SW = N / 16;                      // score warpgroups
  static constexpr int SCORE_WARPS = 4 * SW;
  static constexpr int THREADS = 32 * (SCORE_WARPS + 4 + 2);
  static constexpr int CTAS = N == 16 ? 2 : 1;           // per SM
  static constexpr int VB = N == 16 ? 1 : 2;             // V images
  static constexpr int PB = N == 32 ? 2 : 1;             // P images
  static constexpr int SB = N == 32 ? 2 : 1;             // S accumulators
  // tensor memory columns: keys (two buffers of 64), S, O
  static constexpr uint32_t K_COL = 0, S_COL = 128, O_COL = S_COL + SB * 4 * N, COLS = N == 16 ? 256 : 512;
  static constexpr int Q_BYTES = N * D * 2;              // one half of the query image
  static constexpr int V_BYTES = EX_TILE * D * 2;
  static constexpr int P_BYTES = EX_TILE * 2 * N * 2;    // [2N / 8][128 positions][8 rows]
  static constexpr int OFF_V = 2 * Q_BYTES;
  static constexpr int OFF_P = OFF_V + VB * V_BYTES;
  static constexpr int OFF_ROWS = OFF_P + PB * P_BYTES;
  // per-row words: threshold, factor, maximum used, maximum, rescale factor, 4 query sums,
  // mask (2 words), query index, 4 warps' maxima
  static constexpr int ROW_WORDS = 16;
  static constexpr int OFF_BARS = OFF_ROWS + ROW_WORDS * N * 4;
  static constexpr int OFF_RAW = (OFF_BARS + 512 + 127) / 128 * 128;
  static_assert(O_COL + 2 * N <= COLS, "tensor memory");
};

// kind::f16 instruction descriptor: D fp32; A and B fp16 or both bf16; M = 128.
__device__ __forceinline__ uint32_t exm_idesc(int n, bool bf16, bool mn_major) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (mn_major ? (1u << 15) | (1u << 16) : 0u) |
         ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
// A and B from shared memory.
__device__ __forceinline__ void umma_f16_ss(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of an MN-major operand without swizzle: bricks of 8 (M or N) x 8 (K)
// elements, 128 contiguous bytes each (16 bytes per K); `kstep` bytes to the next 8
// along K, `mnstep` to the next 8 along M or N.
__device__ __forceinline__ uint64_t umma_desc_bricks(uint32_t saddr, uint32_t kstep, uint32_t mnstep) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((kstep >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((mnstep >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}

// Tensor memory to registers, waited for inside the statement so that no use can move above.
__device__ __forceinline__ void tmem_ld16_wait(uint32_t a, uint32_t r[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a)
      : "memory");
}
// Four groups of 8 columns, waited for in the same statement.
__device__ __forceinline__ void tmem_ld8x4_wait(uint32_t a, uint32_t step, uint32_t r[4][8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%32];\n"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%33];\n"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%34];\n"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%24,%25,%26,%27,%28,%29,%30,%31}, [%35];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0][0]), "=r"(r[0][1]), "=r"(r[0][2]), "=r"(r[0][3]), "=r"(r[0][4]), "=r"(r[0][5]), "=r"(r[0][6]),
        "=r"(r[0][7]), "=r"(r[1][0]), "=r"(r[1][1]), "=r"(r[1][2]), "=r"(r[1][3]), "=r"(r[1][4]), "=r"(r[1][5]),
        "=r"(r[1][6]), "=r"(r[1][7]), "=r"(r[2][0]), "=r"(r[2][1]), "=r"(r[2][2]), "=r"(r[2][3]), "=r"(r[2][4]),
        "=r"(r[2][5]), "=r"(r[2][6]), "=r"(r[2][7]), "=r"(r[3][0]), "=r"(r[3][1]), "=r"(r[3][2]), "=r"(r[3][3]),
        "=r"(r[3][4]), "=r"(r[3][5]), "=r"(r[3][6]), "=r"(r[3][7])
      : "r"(a), "r"(a + step), "r"(a + 2 * step), "r"(a + 3 * step)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8_wait(uint32_t a, uint32_t r[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t r[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ float exm_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Barrier of one score warpgroup; the second form also tells whether any thread of it
// passed a true predicate.
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(group + 1) : "memory");
}
__device__ __forceinline__ bool group_any(int group, bool v) {
  uint32_t any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.or.pred q, %1, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(any)
      : "r"(group + 1), "r"((uint32_t)v)
      : "memory");
  return any != 0;
}

// Bounded wait of every role.  A timeout latches the error and sets the abort flag, after
// which no wait of the CTA waits any more: the roles run through their remaining tiles on
// whatever is there (all accesses stay inside the CTA's own memory), so they still meet at
// their barriers and the CTA ends; the MMA thread issues nothing more.
// exm_wait1: one thread; exm_wait: a whole warp, converged afterwards.
__device__ __forceinline__ bool exm_wait1(uint64_t* bar, uint32_t parity, const ExtendParams& p, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*abort) return false;
  if (mbar_wait(bar, parity, p.wait_ns)) return true;
  *abort = 1;
  atomicOr(p.err, ERR_TIMEOUT);
  return false;
}
__device__ __forceinline__ void exm_wait(uint64_t* bar, uint32_t parity, const ExtendParams& p, volatile int* abort) {
  exm_wait1(bar, parity, p, abort);
  __syncwarp();
}

// ---- codes to fp16 pairs
//
// 4-bit words take a short way: nibbles i and i + 4 of a word of 8 share a register, so
// one masked OR with 0x6400 makes a pair 1024 + u (or 1024 + 16 u, brought back by a
// multiply-add), and positions 0 .. 7 of a group of 8 channels hold channels
// 0 4 1 5 2 6 3 7.  The query image and the output use the same order.  Other widths keep
// the channel order.
__device__ __forceinline__ int group_channel(int pos, bool nibbles) {   // channel at a position of its group of 8
  return nibbles ? (pos >> 1) | ((pos & 1) << 2) : pos;
}

// Block b of token t -> 16 words of fp16 pairs: u - 2^(BITS-1) (_0) or u (_1), exact.
template <int BITS, bool ASYM, bool KPLANE>
__device__ __forceinline__ void block_codes(const uint8_t* codes, int cb, int t, int b, uint32_t W[16]) {
  uint32_t lo[8], hi[2];
  block_planes<BITS, KPLANE>(codes, cb, t, b, lo, hi);
  if (BITS == 4) {
    const __half2 c0 = as_h2(ASYM ? 0x64006400u : 0x64086408u);          // 1024, 1032
    const __half2 c1 = as_h2(ASYM ? 0xD400D400u : 0xD480D480u);          // -64, -72
    const __half2 sixteenth = as_h2(0x2C002C00u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = lo[j], v = w >> 8;
      W[4 * j + 0] = as_u32(__hsub2(as_h2((w & 0x000F000Fu) | 0x64006400u), c0));
      W[4 * j + 1] = as_u32(__hfma2(as_h2((w & 0x00F000F0u) | 0x64006400u), sixteenth, c1));
      W[4 * j + 2] = as_u32(__hsub2(as_h2((v & 0x000F000Fu) | 0x64006400u), c0));
      W[4 * j + 3] = as_u32(__hfma2(as_h2((v & 0x00F000F0u) | 0x64006400u), sixteenth, c1));
    }
  } else {
    const __half2 c0 = as_h2(ASYM ? 0x64006400u : (0x6400u + (1u << (BITS - 1))) * 0x10001u);
#define KVQ_EXM_GROUP(J)                                                                  \
  {                                                                                       \
    uint32_t w[4];                                                                        \
    chunk_pairs<BITS, J>(lo, hi, w);                                                      \
    _Pragma("unroll") for (int e = 0; e < 4; ++e) W[4 * J + e] = as_u32(__hsub2(as_h2(w[e]), c0)); \
  }
    KVQ_EXM_GROUP(0)
    KVQ_EXM_GROUP(1)
    KVQ_EXM_GROUP(2)
    KVQ_EXM_GROUP(3)
#undef KVQ_EXM_GROUP
  }
}

// The key codes of `blocks` blocks from b0 of token t into tensor memory columns.
template <int BITS, bool ASYM>
__device__ __forceinline__ void key_blocks(const uint8_t* codes, int cb, int t, int b0, int blocks, uint32_t col) {
#pragma unroll 1
  for (int k = 0; k < blocks; ++k) {
    uint32_t W[16];
    block_codes<BITS, ASYM, true>(codes, cb, t, b0 + k, W);
    __syncwarp();
    tmem_st16(col + 16 * (b0 + k), W);
  }
}
// Value block b of token t (or zeros) into the V image.
template <int BITS, bool ASYM>
__device__ __forceinline__ void value_block(const uint8_t* codes, const uint8_t* scales, int cb, int sb, int t, int b,
                                            bool valid, uint8_t* img, int row) {
  uint32_t W[16];
  if (valid) {
    block_codes<BITS, ASYM, false>(codes, cb, t, b, W);
    __half2 d2, m2;
    if (ASYM) {
      const __half2 dm = *reinterpret_cast<const __half2*>(scales + t * sb + 4 * b);
      d2 = __low2half2(dm);
      m2 = __high2half2(dm);
    } else {
      // a scale whose largest product would leave fp16's range is clamped: an infinite value
      // would reach every row as 0 * inf
      d2 = __half2half2(*reinterpret_cast<const __half*>(scales + t * sb + 2 * b));
      d2 = __hmin2(d2, __float2half2_rn(65504.f / (float)(1 << (BITS - 1))));
    }
#pragma unroll
    for (int e = 0; e < 16; ++e)
      W[e] = as_u32(ASYM ? __hmax2(__hmin2(__hfma2(as_h2(W[e]), d2, m2), as_h2(0x7BFF7BFFu)), as_h2(0xFBFFFBFFu))
                         : __hmul2(as_h2(W[e]), d2));
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) W[e] = 0u;
  }
  // chunks 4b .. 4b+3 of the row, in an order that differs between the two 64-channel
  // halves: the 8 lanes of a store phase (2 tokens x 4 blocks) then fill all banks
  uint8_t* base = img + (b >> 1) * (EX_TILE * 128) + row * 128;
  const bool swap = b >= 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = i ^ 2;
    const uint4 v = make_uint4(swap ? W[4 * j] : W[4 * i], swap ? W[4 * j + 1] : W[4 * i + 1],
                               swap ? W[4 * j + 2] : W[4 * i + 2], swap ? W[4 * j + 3] : W[4 * i + 3]);
    const int c = 4 * (b & 1) + (swap ? j : i);
    *reinterpret_cast<uint4*>(base + ((c ^ (row & 7)) << 4)) = v;
  }
}

#define KVQ_EXM_CODECS(CASE)                                                              \
  CASE(KVQ_Q8_0, 8, false) CASE(KVQ_Q6_0, 6, false) CASE(KVQ_Q5_0, 5, false)              \
  CASE(KVQ_Q4_0, 4, false) CASE(KVQ_Q3_0, 3, false) CASE(KVQ_Q2_0, 2, false)              \
  CASE(KVQ_Q8_1, 8, true) CASE(KVQ_Q6_1, 6, true) CASE(KVQ_Q5_1, 5, true)                 \
  CASE(KVQ_Q4_1, 4, true) CASE(KVQ_Q3_1, 3, true) CASE(KVQ_Q2_1, 2, true)

__device__ __forceinline__ bool finite_words(const uint4& v, bool bf16) {   // no NaN or infinity among 8 raw values
  const uint32_t e = bf16 ? 0x7F80u : 0x7C00u;
  bool ok = true;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t w = k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
    ok &= (w & e) != e && ((w >> 16) & e) != e;
  }
  return ok;
}
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w, bool bf16) {
  const uint32_t e = bf16 ? 0x7F80u : 0x7C00u;
  if ((w & e) == e) w &= 0xFFFF0000u;
  if (((w >> 16) & e) == e) w &= 0x0000FFFFu;
  return w;
}

}  // namespace

template <int N>
__global__ void __launch_bounds__(Shape<N>::THREADS, Shape<N>::CTAS)
    extend_mma_kernel(const __grid_constant__ ExtendParams p) {
  using C = Shape<N>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first_tile = blockIdx.x * p.per, last_tile = min(first_tile + p.per, p.total_tiles);
  const int NR = p.n_raw;

  uint8_t* sQ = smem;
  uint8_t* sV = smem + C::OFF_V;
  uint8_t* sP = smem + C::OFF_P;
  float* rows = reinterpret_cast<float*>(smem + C::OFF_ROWS);
  float* r_thr = rows;                   // scores above this move the maximum (accumulator units)
  float* r_f = rows + N;                 // accumulator -> log2 units
  float* r_use = rows + 2 * N;           // the maximum that weights are taken against (0 while there is none)
  float* r_max = rows + 3 * N;
  float* r_alpha = rows + 4 * N;
  float* r_qsum = rows + 5 * N;          // [4][N] sums of the scaled query over a block's channels
  unsigned long long* r_mask = reinterpret_cast<unsigned long long*>(rows + 9 * N);
  int* r_query = reinterpret_cast<int*>(rows + 11 * N);   // query index in its entry, -1 for padding
  float* r_part = rows + 12 * N;         // [4][N] per-warp results of a row
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  uint64_t* k_full = bars;               // [2] keys of a tile in tensor memory
  uint64_t* s_full = bars + 2;           // [2] S of a tile complete (its keys are read)
  uint64_t* s_empty = bars + 4;          // [2] S of a tile read
  uint64_t* p_full = bars + 6;           // [2]
  uint64_t* v_full = bars + 8;           // [2]
  uint64_t* pv_done = bars + 10;         // [2] P V of a tile complete (its P and V images are free)
  uint64_t* q_full = bars + 12;          // a unit's query image is written and its O columns are free
  uint64_t* done = bars + 13;
  uint64_t* raw_full = bars + 14;        // [8] page stages
  uint64_t* raw_empty = bars + 22;       // [8]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 30);
  volatile int* abort = reinterpret_cast<volatile int*>(bars + 31);
  uint8_t* sRaw = smem + C::OFF_RAW;

  if (warp == C::SCORE_WARPS + 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                 "r"(C::COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&k_full[i], C::SCORE_WARPS);
        mbar_init(&s_full[i], 1);
        mbar_init(&s_empty[i], C::SCORE_WARPS);
        mbar_init(&p_full[i], C::SCORE_WARPS);
        mbar_init(&v_full[i], 4);
        mbar_init(&pv_done[i], 1);
      }
      mbar_init(q_full, C::SCORE_WARPS);
      mbar_init(done, 1);
      for (int i = 0; i < NR; ++i) {
        mbar_init(&raw_full[i], 1);
        mbar_init(&raw_empty[i], C::SCORE_WARPS + 4);
      }
      *abort = 0;
      fence_mbar_init();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  // pages that a tile of [begin, end) positions has, 0 for tail tiles
  auto tile_pages = [&](const ExtendUnit& u, int pos0, int end) -> int {
    return u.kind == EX_TAIL ? 0 : (end - pos0 > PAGE ? 2 : 1);
  };

  if (warp == C::SCORE_WARPS + 4) {
    // ---------------------------------------------------------------- producer
    int pg = 0, issued = 0;
    bool open = true;                                    // lane 0: no wait has run out
    for (int t = first_tile; t < last_tile;) {
      const ExtendUnit u = ex_find(p, t);
      const int stop = min(last_tile, u.first + u.tiles);
      if (u.kind != EX_TAIL) {
        int begin, end;
        ex_range(p, u, &begin, &end);
        const HeadInfo& h = p.heads[u.head];
        const int seq = u.kind == EX_SHARED ? p.seq[p.order[p.g_first[u.index]]] : p.seq[u.index];
        const int* table = p.table + (size_t)seq * p.mpps;
        const int j0 = (begin + (t - u.first) * EX_TILE) / PAGE;
        const int j1 = (min(end, begin + (stop - u.first) * EX_TILE) + PAGE - 1) / PAGE;
        int ids = 0;
        for (int j = j0; j < j1; ++j, ++pg) {
          if (((j - j0) & 31) == 0 && j + lane < j1) {
            ids = table[j + lane];
            if (ids < 0) { atomicOr(p.err, ERR_NO_PAGE); ids = 0; }
          }
          const int id = __shfl_sync(0xffffffffu, ids, (j - j0) & 31);
          const int st = pg % NR;
          if (lane == 0 && open) {
            open = pg < NR || exm_wait1(&raw_empty[st], ((pg / NR) - 1) & 1, p, abort);
            if (open) {
              mbar_arrive_expect_tx(&raw_full[st], h.bytes);
              bulk_g2s(sRaw + (size_t)st * p.stage_bytes, p.pool + (size_t)id * p.page_bytes + h.off, h.bytes,
                       &raw_full[st]);
              issued = pg + 1;
            }
          }
          __syncwarp();
        }
      }
      t = stop;
    }
    // no copy may still be landing when the CTA exits
    if (lane == 0)
      for (int i = max(0, issued - NR); i < issued; ++i)
        if (!mbar_wait(&raw_full[i % NR], (i / NR) & 1, p.wait_ns)) atomicOr(p.err, ERR_TIMEOUT);
    __syncwarp();
  } else if (warp == C::SCORE_WARPS + 5) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      const uint32_t aQ = smem_u32(sQ), aV = smem_u32(sV), aP = smem_u32(sP);
      const uint64_t dQ = umma_desc_sw128(aQ, 16, 1024);
      const uint64_t dV = umma_desc_sw128(aV, EX_TILE * 128, 1024);
      const uint64_t dP = umma_desc_bricks(aP, 128, EX_TILE * 16);
      int tg = 0, units = 0;
      bool ok = true;
      for (int t = first_tile; t < last_tile && ok; ++units) {
        const ExtendUnit u = ex_find(p, t);
        const int n = min(last_tile, u.first + u.tiles) - t;
        const bool raw_k = ex_raw_k(p, u), bf16 = p.bf16 && u.kind == EX_TAIL;
        const uint32_t idS = exm_idesc(N, bf16, false);
        const uint32_t idPV = exm_idesc(N == 64 ? 64 : 2 * N, bf16, true);
        ok = exm_wait1(q_full, units & 1, p, abort);
        tc_fence_after();
        auto issue_pv = [&](int i, int g) {
          ok = ok && exm_wait1(&p_full[g & 1], (g >> 1) & 1, p, abort) &&
               exm_wait1(&v_full[g & 1], (g >> 1) & 1, p, abort);
          if (!ok) return;
          tc_fence_after();
          const uint64_t v = dV + (uint64_t)((g % C::VB) * C::V_BYTES / 16);
          const uint64_t q = dP + (uint64_t)((g % C::PB) * C::P_BYTES / 16);
#pragma unroll
          for (int s = 0; s < EX_TILE / 16; ++s) {
            umma_f16_ss(tmem + C::O_COL, v + s * 128, q + s * 16, idPV, (i > 0 || s > 0) ? 1u : 0u);
            if (N == 64)                                 // the weights' low halves
              umma_f16_ss(tmem + C::O_COL + 64, v + s * 128, q + 8 * (EX_TILE * 16) / 16 + s * 16, idPV,
                          (i > 0 || s > 0) ? 1u : 0u);
          }
          umma_commit(&pv_done[g & 1]);
        };
        for (int i = 0; i < n && ok; ++i, ++tg) {
          ok = exm_wait1(&k_full[tg & 1], (tg >> 1) & 1, p, abort);
          if (ok && tg >= C::SB) ok = exm_wait1(&s_empty[(tg - C::SB) & 1], ((tg - C::SB) >> 1) & 1, p, abort);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = tmem + C::K_COL + (tg & 1) * 64, s = tmem + C::S_COL + (tg % C::SB) * 4 * N;
          if (raw_k) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              umma_f16_tmem_a(s, a + 8 * k, dQ + (k >> 2) * (N * 128 / 16) + (k & 3) * 2, idS, k > 0 ? 1u : 0u);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint64_t q = dQ + (k >> 2) * (N * 128 / 16) + (k & 3) * 2;
              umma_f16_tmem_a(s + (k >> 1) * N, a + 8 * k, q, idS, (k & 1) ? 1u : 0u);
              umma_f16_tmem_a(s + (k >> 1) * N, a + 8 * k, q + C::Q_BYTES / 16, idS, 1u);
            }
          }
          umma_commit(&s_full[tg & 1]);
          if (i > 0) issue_pv(i - 1, tg - 1);
        }
        if (ok) issue_pv(n - 1, tg - 1);
        t += n;
      }
      // nothing of this CTA may still run on the tensor cores when it exits
      umma_commit(done);
      if (!mbar_wait(done, 0, p.wait_ns)) atomicOr(p.err, ERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp >= C::SCORE_WARPS) {
    // ---------------------------------------------------------------- values
    const int vt = threadIdx.x - 32 * C::SCORE_WARPS;    // 0 .. 127
    int tg = 0, pg = 0;
    for (int t = first_tile; t < last_tile;) {
      const ExtendUnit u = ex_find(p, t);
      const int stop = min(last_tile, u.first + u.tiles);
      int begin, end;
      ex_range(p, u, &begin, &end);
      const HeadInfo& h = p.heads[u.head];
      const bool raw = ex_raw_v(p, u);
      const int base = u.kind == EX_SHARED ? 0x7fffffff : p.len[u.index] - p.nq[u.index];
      const uint8_t* ring = u.kind == EX_TAIL ? p.tail + (((size_t)p.seq[u.index] * p.L + p.layer) * p.Hkv + u.head) *
                                                             (size_t)p.T * (D * 2 * 2)
                                              : nullptr;
      for (; t < stop; ++t, ++tg) {
        const int pos0 = begin + (t - u.first) * EX_TILE;
        const int np = tile_pages(u, pos0, end);
        for (int k = 0; k < np; ++k) exm_wait(&raw_full[(pg + k) % NR], ((pg + k) / NR) & 1, p, abort);
        if (tg >= C::VB) exm_wait(&pv_done[(tg - C::VB) & 1], ((tg - C::VB) >> 1) & 1, p, abort);
        uint8_t* img = sV + (size_t)(tg % C::VB) * C::V_BYTES;
        if (raw) {
          // thread = position: its 256-byte row, 16 chunks
          const int pos = pos0 + vt;
          const bool valid = pos < end;
          const uint8_t* src = nullptr;
          if (valid && u.kind == EX_TAIL) {
            const int slot = pos % p.T;
            src = ring + (size_t)(slot / TAIL_TOK) * TAIL_PAGE_BYTES + TAIL_TOK * D * 2 + (slot % TAIL_TOK) * (D * 2);
          } else if (valid) {
            src = sRaw + (size_t)((pg + vt / PAGE) % NR) * p.stage_bytes + PAGE * (h.cbK + h.sbK) + (vt % PAGE) * h.cbV;
          }
          const bool clean = pos >= base;                // rows may mask this position: nothing non-finite may reach them
#pragma unroll 4
          for (int c = 0; c < 16; ++c) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (valid) v = *reinterpret_cast<const uint4*>(src + 16 * c);
            if (clean) {
              v.x = finite_or_zero(v.x, p.bf16);
              v.y = finite_or_zero(v.y, p.bf16);
              v.z = finite_or_zero(v.z, p.bf16);
              v.w = finite_or_zero(v.w, p.bf16);
            }
            *reinterpret_cast<uint4*>(img + (c >> 3) * (EX_TILE * 128) + vt * 128 + (((c & 7) ^ (vt & 7)) << 4)) = v;
          }
        } else {
          const int half = vt >> 6, th = vt & 63;        // page of the tile
          const uint8_t* region = sRaw + (size_t)((pg + half) % NR) * p.stage_bytes;
          const uint8_t* codes = region + PAGE * (h.cbK + h.sbK);
          const uint8_t* scales = codes + PAGE * h.cbV;
#define KVQ_EXM_CASE(CODEC, B, A)                                                                             \
  case CODEC:                                                                                                 \
    _Pragma("unroll 1") for (int k = 0; k < 4; ++k) {                                                         \
      const int i = k * 64 + th, tok = i >> 2;                                                                \
      value_block<B, A>(codes, scales, h.cbV, h.sbV, tok, i & 3, pos0 + half * PAGE + tok < end, img,          \
                        half * PAGE + tok);                                                                   \
    }                                                                                                         \
    break;
          switch (h.vcodec) {
            KVQ_EXM_CODECS(KVQ_EXM_CASE)
            default: break;
          }
#undef KVQ_EXM_CASE
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          for (int k = 0; k < np; ++k) mbar_arrive(&raw_empty[(pg + k) % NR]);
          mbar_arrive(&v_full[tg & 1]);
        }
        pg += np;
      }
    }
  } else {
    // ---------------------------------------------------------------- scores
    const int group = warp >> 2, w4 = warp & 3;          // 16 rows from row0; lanes 32 w4 .. of tensor memory
    const int row0 = 16 * group, tok = 32 * w4 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * w4) << 16);
    constexpr int KBLOCKS = 4 / C::SW;                   // key blocks this thread unpacks
    int tg = 0, pg = 0;
    for (int t = first_tile; t < last_tile;) {
      const ExtendUnit u = ex_find(p, t);
      const int n = min(last_tile, u.first + u.tiles) - t;
      int begin, end;
      ex_range(p, u, &begin, &end);
      const HeadInfo& h = p.heads[u.head];
      const bool raw_k = ex_raw_k(p, u), raw_v = ex_raw_v(p, u), tail = u.kind == EX_TAIL;
      const bool asym = !raw_k && codec_is_asym(h.kcodec), bf16_pv = p.bf16 && tail;
      const int base = u.kind == EX_SHARED ? 0x7fffffff : p.len[u.index] - p.nq[u.index];
      const int pos_first = begin + (t - u.first) * EX_TILE;
      const uint8_t* ring =
          tail ? p.tail + (((size_t)p.seq[u.index] * p.L + p.layer) * p.Hkv + u.head) * (size_t)p.T * (D * 2 * 2) : nullptr;
      // ---- the group's 16 query rows, four per warp
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const int r = row0 + 4 * w4 + k;
        const ExtendRow w = ex_row(p, u, r);
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        uint2 bits = make_uint2(0u, 0u);
        float f = p.qscale;
        if (w.entry >= 0) {
          const __half* src = p.q + ((size_t)(p.q0[w.entry] + w.query) * p.Hq + w.head) * D;
          bits = *reinterpret_cast<const uint2*>(src + 4 * lane);
          load_row_raw(src, x, p.bf16);
        }
        const int c = lane >> 1;                         // the lane's 16-byte chunk (8 channels)
        uint8_t* at = sQ + (c >> 3) * (N * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4) + 8 * (lane & 1);
        if (raw_k) {
          *reinterpret_cast<uint2*>(at) = bits;
        } else {
          if (p.rot != KVQ_ROT_NONE) {
            if (p.s_k) {
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] *= p.s_k[(size_t)u.head * D + 4 * lane + i];
            }
            fwht_row(x);
          }
          float big = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
          for (int m = 16; m; m >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, m));
          if (big > 0.f && big < INFINITY) {             // largest element in [2^11, 2^12)
            int e;
            frexpf(big, &e);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = ldexpf(x[i], 12 - e);
            f = ldexpf(f, e - 12);
          }
          float s = (x[0] + x[1]) + (x[2] + x[3]);
#pragma unroll
          for (int m = 1; m < 8; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
          if ((lane & 7) == 0) r_qsum[(lane >> 3) * N + r] = s;
          if (h.kbits == 4) {
            // positions 0 4 1 5 | 2 6 3 7: the even lane of a pair takes channels 0 4 1 5
            const bool odd = lane & 1;
            const float ra = __shfl_xor_sync(0xffffffffu, odd ? x[0] : x[2], 1);
            const float rb = __shfl_xor_sync(0xffffffffu, odd ? x[1] : x[3], 1);
            const float y0 = odd ? ra : x[0], y1 = odd ? x[2] : ra, y2 = odd ? rb : x[1], y3 = odd ? x[3] : rb;
            x[0] = y0; x[1] = y1; x[2] = y2; x[3] = y3;
          }
          const __half2 h0 = __floats2half2_rn(x[0], x[1]), h1 = __floats2half2_rn(x[2], x[3]);
          const float2 g0 = __half22float2(h0), g1 = __half22float2(h1);
          *reinterpret_cast<uint2*>(at) = make_uint2(as_u32(h0), as_u32(h1));
          *reinterpret_cast<uint2*>(at + C::Q_BYTES) =
              make_uint2(as_u32(__floats2half2_rn(x[0] - g0.x, x[1] - g0.y)), as_u32(__floats2half2_rn(x[2] - g1.x, x[3] - g1.y)));
        }
        if (lane == 0) {
          r_thr[r] = -INFINITY;
          r_f[r] = f;
          r_use[r] = 0.f;
          r_max[r] = -INFINITY;
          r_query[r] = w.entry < 0 ? -1 : w.query;
          r_mask[r] = (w.entry >= 0 && p.mask) ? p.mask[p.q0[w.entry] + w.query] : 0ull;
        }
      }
      fence_proxy_async_shared();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      group_sync(group);                                 // the group's row words are written

      float d_next[4] = {0.f, 0.f, 0.f, 0.f}, m_next[4] = {0.f, 0.f, 0.f, 0.f};
      // Keys of tile i of the run into the buffer of tile g, their scales into *_next.
      auto load_keys = [&](int i, int g) {
        const int pos0 = pos_first + i * EX_TILE, pos = pos0 + tok;
        const int np = tile_pages(u, pos0, end);
        const uint32_t col = lanes + C::K_COL + (g & 1) * 64;
        for (int k = 0; k < np; ++k) exm_wait(&raw_full[(pg + k) % NR], ((pg + k) / NR) & 1, p, abort);
        const uint8_t* region = sRaw + (size_t)((pg + tok / PAGE) % NR) * p.stage_bytes;
        if (raw_k) {
          const uint8_t* src = region;
          int step = PAGE * 16;
          if (tail) {
            const int slot = pos % p.T;
            src = ring + (size_t)(slot / TAIL_TOK) * TAIL_PAGE_BYTES + (slot % TAIL_TOK) * 16;
            step = TAIL_TOK * 16;
          } else {
            src += (tok % PAGE) * 16;
          }
          const bool valid = pos < end;
#pragma unroll 1
          for (int k = 0; k < KBLOCKS; ++k) {
            const int b = group * KBLOCKS + k;
            uint32_t W[16];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint4 v = make_uint4(0u, 0u, 0u, 0u);
              if (valid) v = *reinterpret_cast<const uint4*>(src + (size_t)(4 * b + c) * step);
              W[4 * c] = v.x; W[4 * c + 1] = v.y; W[4 * c + 2] = v.z; W[4 * c + 3] = v.w;
            }
            __syncwarp();
            tmem_st16(col + 16 * b, W);
          }
        } else {
          const uint8_t* scales = region + PAGE * h.cbK + (tok % PAGE) * h.sbK;
          if (asym) {
            const uint4 s = *reinterpret_cast<const uint4*>(scales);
            const uint32_t w[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const float2 dm = __half22float2(as_h2(w[b]));
              d_next[b] = dm.x;
              m_next[b] = dm.y;
            }
          } else {
            const uint2 s = *reinterpret_cast<const uint2*>(scales);
            const float2 a = __half22float2(as_h2(s.x)), b = __half22float2(as_h2(s.y));
            d_next[0] = a.x; d_next[1] = a.y; d_next[2] = b.x; d_next[3] = b.y;
          }
#define KVQ_EXM_CASE(CODEC, B, A) \
  case CODEC: key_blocks<B, A>(region, h.cbK, tok % PAGE, group * KBLOCKS, KBLOCKS, col); break;
          switch (h.kcodec) {
            KVQ_EXM_CODECS(KVQ_EXM_CASE)
            default: break;
          }
#undef KVQ_EXM_CASE
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          for (int k = 0; k < np; ++k) mbar_arrive(&raw_empty[(pg + k) % NR]);
          mbar_arrive(&k_full[g & 1]);
        }
        pg += np;
      };

      float l[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) l[r] = 0.f;
      load_keys(0, tg);
#pragma unroll 1
      for (int i = 0; i < n; ++i, ++tg) {
        float dk[4], mk[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) { dk[b] = d_next[b]; mk[b] = m_next[b]; }
        if (i + 1 < n) load_keys(i + 1, tg + 1);
        exm_wait(&s_full[tg & 1], (tg >> 1) & 1, p, abort);
        tc_fence_after();
        // ---- scores of this position, accumulator units
        float a[16];
        const uint32_t s_col = lanes + C::S_COL + (tg % C::SB) * 4 * N + row0;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (raw_k) {
            uint32_t v[8];
            tmem_ld8_wait(s_col + 8 * c, v);
#pragma unroll
            for (int r = 0; r < 8; ++r) a[8 * c + r] = __uint_as_float(v[r]);
          } else {
            uint32_t v[4][8];
            tmem_ld8x4_wait(s_col + 8 * c, N, v);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              float s = dk[0] * __uint_as_float(v[0][r]);
              s = fmaf(dk[1], __uint_as_float(v[1][r]), s);
              s = fmaf(dk[2], __uint_as_float(v[2][r]), s);
              s = fmaf(dk[3], __uint_as_float(v[3][r]), s);
              a[8 * c + r] = s;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[tg & 1]);
        if (asym) {
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
              const float4 s = *reinterpret_cast<const float4*>(&r_qsum[b * N + row0 + r]);
              a[r] = fmaf(mk[b], s.x, a[r]);
              a[r + 1] = fmaf(mk[b], s.y, a[r + 1]);
              a[r + 2] = fmaf(mk[b], s.z, a[r + 2]);
              a[r + 3] = fmaf(mk[b], s.w, a[r + 3]);
            }
        }
        const int pos = pos_first + i * EX_TILE + tok;
        if (pos >= min(end, base)) {
          // outside the range, or one of the entry's new tokens
          bool spoils = false;                           // a raw value row with NaN or infinity
          if (raw_v && pos < end) {
            const int slot = tail ? pos % p.T : 0;
            // an F16 page's stage may be gone by now: read the row from the page itself
            const uint8_t* src;
            if (tail) {
              src = ring + (size_t)(slot / TAIL_TOK) * TAIL_PAGE_BYTES + TAIL_TOK * D * 2 + (slot % TAIL_TOK) * (D * 2);
            } else {
              const int id = max(0, p.table[(size_t)p.seq[u.index] * p.mpps + pos / PAGE]);
              src = p.pool + (size_t)id * p.page_bytes + h.off + PAGE * (h.cbK + h.sbK) + (pos % PAGE) * h.cbV;
            }
#pragma unroll 1
            for (int c = 0; c < 16; ++c) spoils |= !finite_words(*reinterpret_cast<const uint4*>(src + 16 * c), p.bf16);
          }
          const int j = pos - base;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const bool sees = pos < end && (j < 0 || (p.mask ? (r_mask[row0 + r] >> j) & 1ull : j <= r_query[row0 + r]));
            a[r] = !sees ? -INFINITY : spoils ? __uint_as_float(0x7fc00000u) : a[r];
          }
        }
        // ---- the running maximum
        bool high = false;
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const float4 th = *reinterpret_cast<const float4*>(&r_thr[row0 + r]);
          high |= a[r] > th.x || a[r + 1] > th.y || a[r + 2] > th.z || a[r + 3] > th.w;
        }
        if (group_any(group, high)) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            float m = a[r];
#pragma unroll
            for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
            if (lane == 0) r_part[w4 * N + row0 + r] = m;
          }
          group_sync(group);
          if (w4 == 0 && lane < 16) {
            const int r = row0 + lane;
            const float f = r_f[r], old = r_max[r];
            const float top = fmaxf(fmaxf(r_part[r], r_part[N + r]), fmaxf(r_part[2 * N + r], r_part[3 * N + r])) * f;
            const float m = fmaxf(old, top);
            r_alpha[r] = m == old ? 1.f : exm_ex2(old - m);
            r_max[r] = m;
            r_use[r] = m == -INFINITY ? 0.f : m;
            r_thr[r] = m == -INFINITY ? -INFINITY : (m + EXM_RESCALE) / f;
          }
          group_sync(group);
          float al[16];
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            al[r] = r_alpha[row0 + r];
            l[r] *= al[r];
          }
          if (i > 0) {                                   // O holds the tiles before this one
            exm_wait(&pv_done[(tg - 1) & 1], ((tg - 1) >> 1) & 1, p, abort);
            tc_fence_after();
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {
              uint32_t v[16];
              const uint32_t o = lanes + C::O_COL + part * N + row0;
              tmem_ld16_wait(o, v);
#pragma unroll
              for (int r = 0; r < 16; ++r) v[r] = __float_as_uint(__uint_as_float(v[r]) * al[r]);
              tmem_st16(o, v);
            }
            tmem_wait_st();
          }
        }
        // ---- weights: fp32 sums, and two halves into the P image
        if (i >= C::PB) exm_wait(&pv_done[(tg - C::PB) & 1], ((tg - C::PB) >> 1) & 1, p, abort);
        uint8_t* img = sP + (size_t)(tg % C::PB) * C::P_BYTES + tok * 16;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * c + 4 * e;
            const float4 f = *reinterpret_cast<const float4*>(&r_f[row0 + r]);
            const float4 m = *reinterpret_cast<const float4*>(&r_use[row0 + r]);
            const float x0 = exm_ex2(fmaf(a[r], f.x, -m.x)), x1 = exm_ex2(fmaf(a[r + 1], f.y, -m.y));
            const float x2 = exm_ex2(fmaf(a[r + 2], f.z, -m.z)), x3 = exm_ex2(fmaf(a[r + 3], f.w, -m.w));
            l[r] += x0;
            l[r + 1] += x1;
            l[r + 2] += x2;
            l[r + 3] += x3;
            if (bf16_pv) {
              const __nv_bfloat162 b0 = __floats2bfloat162_rn(x0, x1), b1 = __floats2bfloat162_rn(x2, x3);
              const float2 g0 = __bfloat1622float2(b0), g1 = __bfloat1622float2(b1);
              hi[2 * e] = float2_to_raw2(x0, x1, true);
              hi[2 * e + 1] = float2_to_raw2(x2, x3, true);
              lo[2 * e] = float2_to_raw2(x0 - g0.x, x1 - g0.y, true);
              lo[2 * e + 1] = float2_to_raw2(x2 - g1.x, x3 - g1.y, true);
            } else {
              const __half2 b0 = __floats2half2_rn(x0, x1), b1 = __floats2half2_rn(x2, x3);
              const float2 g0 = __half22float2(b0), g1 = __half22float2(b1);
              hi[2 * e] = as_u32(b0);
              hi[2 * e + 1] = as_u32(b1);
              lo[2 * e] = as_u32(__floats2half2_rn(x0 - g0.x, x1 - g0.y));
              lo[2 * e + 1] = as_u32(__floats2half2_rn(x2 - g1.x, x3 - g1.y));
            }
          }
          const int brick = (row0 >> 3) + c;
          *reinterpret_cast<uint4*>(img + (size_t)brick * (EX_TILE * 16)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(img + (size_t)(N / 8 + brick) * (EX_TILE * 16)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[tg & 1]);
      }
      // ---- the unit's partial result: O^T (lane = channel position), sums, maximum
      const size_t slot = (size_t)blockIdx.x + u.unit;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float s = l[r];
#pragma unroll
        for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
        if (lane == 0) r_part[w4 * N + row0 + r] = s;
      }
      exm_wait(&pv_done[(tg - 1) & 1], ((tg - 1) >> 1) & 1, p, abort);
      tc_fence_after();
      {
        uint32_t o[16], q[16];
        tmem_ld16_wait(lanes + C::O_COL + row0, o);
        tmem_ld16_wait(lanes + C::O_COL + N + row0, q);
        const int channel = (tok & ~7) | group_channel(tok & 7, !raw_v && h.vbits == 4);
        float* dst = p.part_o + (slot * N + row0) * D + channel;
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (r_query[row0 + r] >= 0) dst[(size_t)r * D] = __uint_as_float(o[r]) + __uint_as_float(q[r]);
      }
      group_sync(group);
      if (w4 == 0 && lane < 16) {
        const int r = row0 + lane;
        const float s = (r_part[r] + r_part[N + r]) + (r_part[2 * N + r] + r_part[3 * N + r]);
        if (r_query[r] >= 0) p.part_ml[slot * N + r] = make_float2(r_max[r], s);
      }
      tc_fence_before();
      group_sync(group);                                 // the row words may be overwritten
      t += n;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::SCORE_WARPS + 5) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::COLS) : "memory");
  }
}

template <int N>
static cudaError_t launch(const ExtendParams& p, cudaStream_t s) {
  const cudaError_t e =
      cudaFuncSetAttribute(extend_mma_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, EXM_SMEM_MAX);
  if (e != cudaSuccess) return e;
  const size_t smem = (size_t)Shape<N>::OFF_RAW + (size_t)p.n_raw * p.stage_bytes;
  extend_mma_kernel<N><<<p.n_ctas, Shape<N>::THREADS, smem, s>>>(p);
  note_launches(1);
  return cudaGetLastError();
}

ExtendShape extend_mma_shape(int N, int stage_bytes) {
  const int off = N == 16 ? Shape<16>::OFF_RAW : N == 32 ? Shape<32>::OFF_RAW : Shape<64>::OFF_RAW;
  const int ctas = N == 16 ? Shape<16>::CTAS : 1;
  ExtendShape x;
  // two CTAs share an SM's 228 KiB (1 KiB of each is reserved)
  x.ctas_per_sm = ctas;
  x.n_raw = (std::min(EXM_SMEM_MAX, 228 * 1024 / ctas - 1024) - off) / stage_bytes;
  if (x.n_raw < 4 && ctas > 1) {                         // large page-heads: one CTA with the whole SM's ring
    x.ctas_per_sm = 1;
    x.n_raw = (EXM_SMEM_MAX - off) / stage_bytes;
  }
  x.n_raw = std::min(x.n_raw, 8);
  return x;
}

cudaError_t launch_extend_mma(const ExtendParams& p, cudaStream_t s) {
  return p.N == 16 ? launch<16>(p, s) : p.N == 32 ? launch<32>(p, s) : launch<64>(p, s);
}

}  // namespace kvq
