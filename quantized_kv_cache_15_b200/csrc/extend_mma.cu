// Attention of several new tokens per sequence on the 5th-generation tensor cores
// (every codec, F16 pages and the raw tail).
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
// (2^-11 of a value; see exm_again for those that fp16 cannot hold); the softmax weights as two halves side by side in N (fp16: 22 bits, see
// EXM_BIAS; bf16 next to bf16 rows: 16 bits),
// which costs the tensor cores nothing where a product is bound by reading its A operand.
// Raw rows (tail, F16 pages) enter as they are, with the raw query.  Rank rows have the codes
// 2 u - (2^b - 1) of half their scales, in the head's projected space (q' = M_h q).
//
// Roles (32 (4 SW + 2) threads; SW warpgroups of RW = 8 or 16 rows each):
//   workers   every warp does a share of each step of a tile: its positions' key codes into
//             tensor memory (for the next tile), value rows into the V image (128-byte
//             swizzle), then scores -> weights 2^(s - m + EXM_BIAS) into the P image, with
//             sums per thread.  The running maximum m moves only when a score passes it by 8
//             (log2 units), found by one barrier vote a tile; then the group's O is rescaled.
//   producer  one bulk copy per page-head into a ring of tile stages, running ahead over
//             tiles and units;
//   MMA warp  one elected thread issues both products, S of the next tile before P V.
// The arithmetic around the products decides the speed (an unpack of 1.1 instructions a key
// value, 1.6 a value value, 12 a score), and after it instruction fetch: with separate score
// and value warps the three loops together overflow the instruction caches next to the
// schedulers (64 ragged sequences of 1024 to 16384 tokens x 4 drafts, 32 query heads over 8,
// 4 bits: 525 us so, 437 with workers that all run one loop, 301 now: 2.3 TB/s of packed rows,
// issue slots 60 % busy, the tensor pipe 11 %).
#include "extend.h"

#include "dequant_row.cuh"
#include "ptx.cuh"
#include "quant.cuh"
#include "tensor.cuh"

namespace kvq {

namespace {

constexpr float EXM_RESCALE = 8.0f;
// fp16 weights are taken against the row's maximum less EXM_BIAS, so the largest is 2^7, 2^15
// before the maximum moves, and what the upper half leaves goes into the lower one EXM_LOW
// times as large (its columns of O are brought back with the partial result).  Together they
// have 22 bits down to 2^-21 of the largest weight, and below that an error of at most 2^-43
// of it: tokens next to one with nearly all of the weight keep theirs (halves of 2^(s - max)
// without both: 6 bits at 2^-20 and nothing below 2^-25, which the sums still count).  bf16
// halves have the range of fp32 and need neither.
constexpr float EXM_BIAS = 7.0f;
constexpr float EXM_LOW = 2048.0f;
constexpr float EXM_NONE = -1e30f;       // "maximum used" of a row without one: any score is far above it
constexpr int EXM_SMEM_MAX = 232448;                     // 227 KiB opt-in per CTA

// N rows a unit, CT CTAs on an SM.
template <int N, int CT>
struct Shape {
  static constexpr int RW = N == 64 ? 16 : 8;            // rows of a warpgroup
  static constexpr int SW = N / RW;                      // warpgroups
  static constexpr int WORKERS = 4 * SW;                 // warps
  static constexpr int THREADS = 32 * (WORKERS + 2);
  // With one CTA an SM the keys of the next tile come first in a turn, into a second buffer,
  // so that the products of the tile in hand have time; with two CTAs the scores come first,
  // which gives P V of the tile before more time (the other way round: 131072 tokens x 8 drafts
  // 110 us instead of 105; 64 sequences x 4 drafts 329 instead of 301).
  static constexpr bool KEYS_FIRST = CT == 1;
  // tensor memory columns: keys, S, O
  static constexpr int KB = KEYS_FIRST ? 2 : 1;
  static constexpr uint32_t K_COL = 0, S_COL = 64 * KB, O_COL = S_COL + 4 * N, COLS = O_COL + 2 * N <= 256 ? 256 : 512;
  static constexpr int Q_BYTES = N * D * 2;              // one half of the query image
  static constexpr int V_BYTES = EX_TILE * D * 2;
  static constexpr int P_BYTES = EX_TILE * 2 * N * 2;    // [2N / 8][128 positions][8 rows]
  static constexpr int OFF_V = 2 * Q_BYTES;
  static constexpr int OFF_P = OFF_V + V_BYTES;
  static constexpr int OFF_ROWS = OFF_P + P_BYTES;
  // per-row words: factor, maximum used, maximum, rescale factor, 4 query sums, mask (2
  // words), query index, 4 warps' results
  static constexpr int ROW_WORDS = 16;
  static constexpr int OFF_BARS = OFF_ROWS + ROW_WORDS * N * 4;
  static constexpr int OFF_RAW = (OFF_BARS + 256 + 127) / 128 * 128;
  static_assert(O_COL + 2 * N <= COLS, "tensor memory");
};
constexpr int EXM_MIN_STAGES = 2;        // a tile's pages are held while the next tile's are waited for

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
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t r[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
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
// (a - b) f of two pairs, f a power of two: two packed instructions.
__device__ __forceinline__ float2 sub_scale2(float2 a, float2 b, float f) {
  float2 r;
  asm("{\n .reg .b64 x, y, m, k;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 m, {%6, %6};\n mov.b64 k, {%7, %7};\n"
      " fma.rn.f32x2 x, y, m, x;\n mul.rn.f32x2 x, x, k;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(-1.f), "f"(f));
  return r;
}
// True in one thread of the (converged) warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
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

// Bounded wait of every role: exm_wait1 in one thread, exm_wait in a whole warp (converged
// afterwards).  A timeout latches the error and sets the abort flag.  From then on the producer
// and the MMA warp load and issue nothing but arrive at once where their copies and products
// would have, and the waits that stay open end after one round of 64 tries: the roles run
// through their remaining tiles on whatever is there (all accesses stay inside the buffers),
// meet at their barriers, and the CTA ends.
// Tries come four in a row, two instructions each: what the waiting warps issue is taken
// from the others, and so is what longer code takes of the instruction cache (a look at the
// flag before the first try or after every four: 64 sequences x 4 drafts 2 to 3 % slower).
// The flag and the timer are read after a round; a try that waits in vain takes some 8 us, so
// a limit is kept to within half a millisecond (with a limit of 1 ms the call ends after 1.6).
static __device__ __noinline__ void exm_wait_late(uint64_t t0, const ExtendParams& p, volatile int* abort) {
  if (globaltimer_ns() - t0 > p.wait_ns && !*abort) {
    *abort = 1;
    atomicOr(p.err, ERR_TIMEOUT);
  }
}
__device__ __forceinline__ void exm_wait1(uint64_t* bar, uint32_t parity, const ExtendParams& p, volatile int* abort) {
  uint64_t t0 = 0;
  while (true) {
    uint32_t ok;
#define KVQ_TRY4                                                                    \
  " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra EXM_OUT;\n"     \
  " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra EXM_OUT;\n"     \
  " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra EXM_OUT;\n"     \
  " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra EXM_OUT;\n"
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, 16;\n"
        "EXM_TRY:\n" KVQ_TRY4
        " sub.u32 n, n, 1;\n setp.ne.u32 q, n, 0;\n @q bra EXM_TRY;\n"
        "EXM_OUT:\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
#undef KVQ_TRY4
    if (ok || *abort) return;
    if (t0 == 0) t0 = globaltimer_ns();
    exm_wait_late(t0, p, abort);
  }
}
__device__ __forceinline__ void exm_wait(uint64_t* bar, uint32_t parity, const ExtendParams& p, volatile int* abort) {
  exm_wait1(bar, parity, p, abort);
  __syncwarp();
}

// Non-blocking first look at a barrier, taken some work before the wait that needs it: the
// look itself takes a few hundred cycles, and mostly finds the phase complete.
__device__ __forceinline__ bool exm_look(uint64_t* bar, uint32_t parity) { return mbar_test_wait(bar, parity); }
__device__ __forceinline__ void exm_wait_if(bool seen, uint64_t* bar, uint32_t parity, const ExtendParams& p,
                                            volatile int* abort) {
  if (!seen) exm_wait1(bar, parity, p, abort);
  __syncwarp();
}

// Position in the ring of page stages.
struct Stage {
  int i;
  uint32_t phase;
  int at;                                                // bytes from the ring's start
  __device__ __forceinline__ void next(int n, int bytes) {
    at += bytes;
    if (++i == n) { i = 0; at = 0; phase ^= 1u; }
  }
};

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

__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {   // one instruction
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
  return r;
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
      W[4 * j + 0] = as_u32(__hsub2(as_h2(and_or(w, 0x000F000Fu, 0x64006400u)), c0));
      W[4 * j + 1] = as_u32(__hfma2(as_h2(and_or(w, 0x00F000F0u, 0x64006400u)), sixteenth, c1));
      W[4 * j + 2] = as_u32(__hsub2(as_h2(and_or(v, 0x000F000Fu, 0x64006400u)), c0));
      W[4 * j + 3] = as_u32(__hfma2(as_h2(and_or(v, 0x00F000F0u, 0x64006400u)), sixteenth, c1));
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

// Key codes of BLOCKS blocks from b0 of the token whose first 16-byte piece is at `codes`,
// into tensor memory columns.
template <int BITS, bool ASYM, int BLOCKS>
__device__ __forceinline__ void key_blocks(const uint8_t* codes, int cb, int b0, uint32_t col) {
#pragma unroll 2
  for (int b = b0; b < b0 + BLOCKS; ++b) {
    uint32_t W[16];
    block_codes<BITS, ASYM, true>(codes, cb, 0, b, W);
    __syncwarp();
    tmem_st16(col + 16 * b, W);
  }
}
// Value block b of the token whose codes and scales are at `codes`, `scales` (zeros unless
// valid) into four chunks of the V image.  A value above fp16's range becomes an infinity,
// which makes its channel of every partial result of the unit infinite or NaN: the CTA finds
// that and takes those rows again (exm_again).
template <int BITS, bool ASYM>
__device__ __forceinline__ void value_block(const uint8_t* codes, const uint8_t* scales, int cb, int b, bool valid,
                                            uint8_t* img, const uint32_t off[4]) {
  uint32_t W[16];
  __half2 d2, m2;
  if (ASYM) {
    uint32_t dm = *reinterpret_cast<const uint32_t*>(scales + 4 * b);
    dm = valid ? dm : 0u;
    d2 = __low2half2(as_h2(dm));
    m2 = __high2half2(as_h2(dm));
  } else {
    uint32_t d = *reinterpret_cast<const uint16_t*>(scales + 2 * b);
    d = valid ? d : 0u;
    d2 = as_h2(d * 0x10001u);
    m2 = d2;
  }
  block_codes<BITS, ASYM, false>(codes, cb, 0, b, W);
#pragma unroll
  for (int e = 0; e < 16; ++e) W[e] = as_u32(ASYM ? __hfma2(as_h2(W[e]), d2, m2) : __hmul2(as_h2(W[e]), d2));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(img + off[i]) = make_uint4(W[4 * i], W[4 * i + 1], W[4 * i + 2], W[4 * i + 3]);
}

// Block b of token t's row of n rank values -> 16 words of fp16 pairs: 2 u - (2^BITS - 1),
// exact, in channel order; zeros behind n.  Rank rows are as short as 2 bytes, so their
// words are read by halves.
template <int BITS>
__device__ __forceinline__ void rank_block(const uint8_t* codes, int cb, int t, bool kplane, int n, int b, uint32_t W[16]) {
  constexpr int P = BITS == 3 ? 2 : BITS;                // bits of the first plane; 3 bits: 1 more in the second
  const int nb = min(n, 32);
  uint32_t lo[P], hi = 0;
  auto half = [&](int o) { return (uint32_t)*reinterpret_cast<const uint16_t*>(codes + (kplane ? kplane_off(cb, t, o) : t * cb + o)); };
#pragma unroll
  for (int i = 0; i < P; ++i) lo[i] = 0;
  if (32 * b < n) {
#pragma unroll
    for (int i = 0; i < 2 * P; ++i)
      if (16 * i < nb * P) lo[i / 2] |= half(b * nb * P / 8 + 2 * i) << (16 * (i % 2));
    if (BITS == 3) {
      hi = half(n * 2 / 8 + b * nb / 8);
      if (nb > 16) hi |= half(n * 2 / 8 + b * nb / 8 + 2) << 16;
    }
  }
  const __half2 two = as_h2(0x40004000u), off = __float2half2_rn(-(float)((1 << BITS) - 1)), c = as_h2(0x64006400u);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    uint32_t w = 0x64006400u;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int v = 2 * e + k, at = v * P;
      uint32_t u = (lo[at / 32] >> (at % 32)) & ((1u << P) - 1u);
      if (BITS == 3) u |= ((hi >> v) & 1u) << 2;
      w |= u << (16 * k);
    }
    W[e] = 32 * b + 2 * e < n ? as_u32(__hfma2(__hsub2(as_h2(w), c), two, off)) : 0u;
  }
}
// Half a rank block's scale: its values are 2 u - (2^b - 1) of these.
__device__ __forceinline__ float rank_scale(const uint8_t* scales, int n, int b) {
  return 32 * b < n ? 0.5f * __half2float(*reinterpret_cast<const __half*>(scales + 2 * b)) : 0.f;
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

// The CTA's partial results that a value above fp16's range has spoilt, again in fp32 on the
// CUDA cores: sums against the same maximum, a warp a row, position after position (every page
// with such a value: 131072 tokens x 8 drafts 24 ms instead of 108 us, 16 x 8192 tokens x 4
// drafts 12 ms instead of 79 us).  Stored values get there where a rotation gathers a row into
// one channel (sqrt(128) times a value of 5790 or more), or from bf16 rows.  A factor for such
// tokens in the loops themselves, values down and weights up by 2^8, cost all other calls 6 to
// 10 %; looking for what is not finite where a unit ends costs 0 to 1 %.
static __device__ __noinline__ void exm_again(const ExtendParams& p, int warp, int warps, float* scratch) {
  const int lane = threadIdx.x & 31;
  float* zs = scratch + warp * D;
  ExtendWalk walk = ex_walk(p, blockIdx.x);
  ExtendUnit u;
  int k0, k1;
  while (ex_next(p, walk, u, k0, k1)) {
    if (ex_raw_v(p, u)) continue;
    const size_t slot = (size_t)blockIdx.x + u.unit;
    const HeadInfo& h = p.heads[u.head];
    int begin, end;
    ex_range(p, u, &begin, &end);
    end = min(end, begin + k1 * EX_TILE);
    for (int r = warp; r < p.N; r += warps) {
      const ExtendRow w = ex_row(p, u, r);
      if (w.entry < 0) continue;
      float4* dst = reinterpret_cast<float4*>(p.part_o + (slot * p.N + r) * D) + lane;
      const float2 ml = p.part_ml[slot * p.N + r];
      float4 o = *dst;
      const bool fits = isfinite(o.x) && isfinite(o.y) && isfinite(o.z) && isfinite(o.w);
      if (__all_sync(0xffffffffu, fits) || !isfinite(ml.y)) continue;
      const int index = p.q0[w.entry] + w.query, base = u.kind == EX_SHARED ? 0x7fffffff : p.len[w.entry] - p.nq[w.entry];
      const unsigned long long mask = p.mask ? p.mask[index] : 0ull;
      const uint2 bits = *reinterpret_cast<const uint2*>(p.q + ((size_t)index * p.Hq + w.head) * D + 4 * lane);
      const float2 q01 = raw2_to_float2(bits.x, p.bf16), q23 = raw2_to_float2(bits.y, p.bf16);
      float q[4] = {q01.x, q01.y, q23.x, q23.y};
      if (h.kcodec == KVQ_RANK) {                        // M_h q
        __syncwarp();
        for (int i = 0; i < D; ++i) {
          float s = 0.f;
          if (i < h.r) {
            const float4 m = *reinterpret_cast<const float4*>(p.M + h.m_off + (size_t)i * D + 4 * lane);
            s = fmaf(m.x, q[0], fmaf(m.y, q[1], fmaf(m.z, q[2], m.w * q[3])));
          }
#pragma unroll
          for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
          if (lane == 0) zs[i] = s;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = zs[4 * lane + i];
      } else if (h.kcodec != KVQ_F16 && p.rot != KVQ_ROT_NONE) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (p.s_k) q[i] *= p.s_k[(size_t)u.head * D + 4 * lane + i];
        fwht_row(q);
      }
      const int* table = p.table + (size_t)p.seq[w.entry] * p.mpps;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int t = begin + k0 * EX_TILE; t < end; ++t) {
        if (t >= base && !(p.mask ? (mask >> (t - base)) & 1ull : t - base <= w.query)) continue;
        const uint8_t* region = p.pool + (size_t)max(0, table[t / PAGE]) * p.page_bytes + h.off;
        float k[4], v[4];
        page_row_stored(region, h, 0, t % PAGE, p.bf16, k);
        page_row_stored(region, h, 1, t % PAGE, p.bf16, v);
        float s = fmaf(q[0], k[0], fmaf(q[1], k[1], fmaf(q[2], k[2], q[3] * k[3])));
#pragma unroll
        for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
        const float e = exm_ex2(fmaf(s, p.qscale, -ml.x));
        o.x = fmaf(e, v[0], o.x); o.y = fmaf(e, v[1], o.y); o.z = fmaf(e, v[2], o.z); o.w = fmaf(e, v[3], o.w);
      }
      *dst = o;
    }
  }
}

}  // namespace

// KC, VC: the codec of every head's keys and values, or -1: read per head.  KVQ_RANK: plans
// with a projection, whose heads hold rank rows (or F16 pages).  A rank head's products are
// in its projected space, zeros behind the rank: q' = M_h q, and the merge takes M_h^T.
template <int N, int CT, int KC, int VC>
__global__ void __launch_bounds__(Shape<N, CT>::THREADS, CT)
    extend_mma_kernel(const __grid_constant__ ExtendParams p) {
  using C = Shape<N, CT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  // The thread's index is held in a register (the compiler would read the special register
  // again at every use), the warp's in a uniform one: 64 sequences x 4 drafts 327 -> 305 us.
  int tid;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int NR = p.n_raw;

  uint8_t* sQ = smem;
  uint8_t* sV = smem + C::OFF_V;
  uint8_t* sP = smem + C::OFF_P;
  float* rows = reinterpret_cast<float*>(smem + C::OFF_ROWS);
  float* r_f = rows;                     // accumulator -> log2 units
  float* r_use = rows + N;               // what weights are taken against: the maximum in use less the bias
  float* r_max = rows + 2 * N;
  float* r_alpha = rows + 3 * N;
  float* r_qsum = rows + 5 * N;          // [4][N] sums of the scaled query over a block's channels
  unsigned long long* r_mask = reinterpret_cast<unsigned long long*>(rows + 9 * N);
  int* r_query = reinterpret_cast<int*>(rows + 11 * N);   // query index in its entry, -1 for padding
  float* r_part = rows + 12 * N;         // [4][N] per-warp results of a row
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  uint64_t* k_full = bars;               // [2] keys of a tile in tensor memory
  uint64_t* s_full = bars + 2;           // [2] S of a tile complete (its keys are read)
  uint64_t* s_empty = bars + 4;          // [2] S of a tile read
  uint64_t* p_full = bars + 6;           // [2] P and V of a tile written
  uint64_t* pv_done = bars + 8;          // [2] P V of a tile complete (the P and V images are free)
  uint64_t* q_full = bars + 10;          // a unit's query image is written and its O columns are free
  uint64_t* done = bars + 11;
  uint64_t* raw_full = bars + 12;        // [8] stages of a tile's two pages
  uint64_t* raw_empty = bars + 20;       // [8]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 28);
  volatile int* abort = reinterpret_cast<volatile int*>(bars + 29);
  volatile int* again = abort + 1;       // a partial result is not finite
  uint8_t* sRaw = smem + C::OFF_RAW;

  if (warp == C::WORKERS + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                 "r"(C::COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&k_full[i], C::WORKERS);
        mbar_init(&s_full[i], 1);
        mbar_init(&s_empty[i], C::WORKERS);
        mbar_init(&p_full[i], C::WORKERS);
        mbar_init(&pv_done[i], 1);
      }
      mbar_init(q_full, C::WORKERS);
      mbar_init(done, 1);
      for (int i = 0; i < NR; ++i) {
        mbar_init(&raw_full[i], 1);
        mbar_init(&raw_empty[i], C::WORKERS);
      }
      *abort = 0;
      *again = 0;
      fence_mbar_init();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  // Launched as a programmatic dependent: nothing global is touched before the wait.  The
  // second of two launches starts when every CTA of the first has passed it, and waits for
  // the first at its own end.
  if (p.chain != EX_ENTRIES) griddep_wait();
  if (p.chain == EX_GROUPS) griddep_launch_dependents();
  ExtendWalk walk = ex_walk(p, blockIdx.x);
  ExtendUnit u;
  int k0, k1;                            // the CTA's tiles of unit u

  if (warp == C::WORKERS) {
    // ---------------------------------------------------------------- producer
    Stage st{0, 1u, 0};                                  // the first round finds the stages empty
    int issued = 0, drop = -1;
    if (p.drop_last_tile) {                              // test-only: the CTA's last tile of pages is not loaded
      for (ExtendWalk w = walk; ex_next(p, w, u, k0, k1);)
        if (u.kind != EX_TAIL) drop += k1 - k0;
    }
    while (ex_next(p, walk, u, k0, k1)) {
      int begin, end;
      ex_range(p, u, &begin, &end);
      if (u.kind == EX_TAIL) {
        // the workers read raw rows straight from the ring: have them in L2 by then
        const uint8_t* ring = p.tail + (((size_t)p.seq[u.index] * p.L + p.layer) * p.Hkv + u.head) * (size_t)p.T * (D * 2 * 2);
        const int used = min(p.T, p.len[u.index]);
        for (int i = lane; i * TAIL_TOK < used; i += 32)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(ring + (size_t)i * TAIL_PAGE_BYTES),
                       "r"((uint32_t)TAIL_PAGE_BYTES)
                       : "memory");
      } else {
        const HeadInfo& h = p.heads[u.head];
        const int seq = u.kind == EX_SHARED ? p.seq[p.order[p.g_first[u.index]]] : p.seq[u.index];
        const int* table = p.table + (size_t)seq * p.mpps;
        const int j0 = (begin + k0 * EX_TILE) / PAGE;
        const int j1 = (min(end, begin + k1 * EX_TILE) + PAGE - 1) / PAGE;
        int ids = 0;
        for (int j = j0; j < j1; j += 2) {
          if (((j - j0) & 31) == 0 && j + lane < j1) {
            ids = table[j + lane];
            if (ids < 0) { atomicOr(p.err, ERR_NO_PAGE); ids = 0; }
          }
          const int id0 = __shfl_sync(0xffffffffu, ids, (j - j0) & 31), id1 = __shfl_sync(0xffffffffu, ids, (j + 1 - j0) & 31);
          if (lane == 0 && issued != drop) {
            exm_wait1(&raw_empty[st.i], st.phase, p, abort);
            if (*abort) {
              mbar_arrive(&raw_full[st.i]);
            } else {
              uint8_t* dst = sRaw + st.at;
              const uint8_t* src = p.pool + h.off;
              mbar_arrive_expect_tx(&raw_full[st.i], j + 1 < j1 ? 2 * h.bytes : h.bytes);
              bulk_g2s(dst, src + (size_t)id0 * p.page_bytes, h.bytes, &raw_full[st.i]);
              if (j + 1 < j1) bulk_g2s(dst + p.page_stage, src + (size_t)id1 * p.page_bytes, h.bytes, &raw_full[st.i]);
            }
            ++issued;
            st.next(NR, 2 * p.page_stage);
          }
          __syncwarp();
        }
      }
    }
    // no copy may still be landing when the CTA exits
    if (lane == 0)
      for (int i = max(0, issued - NR); i < issued; ++i)
        if (!mbar_wait(&raw_full[i % NR], (i / NR) & 1, p.wait_ns)) atomicOr(p.err, ERR_TIMEOUT);
    __syncwarp();
  } else if (warp == C::WORKERS + 1) {
    // ---------------------------------------------------------------- MMA issue
    // The whole warp walks the tiles and waits; one elected thread issues.  (With a single
    // thread in the loop every descriptor word went through a vector register first, and
    // issuing took 3000 cycles a tile.)
    const uint64_t dQ = umma_desc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dV = umma_desc_sw128(smem_u32(sV), EX_TILE * 128, 1024);
    const uint64_t dP = umma_desc_bricks(smem_u32(sP), 128, EX_TILE * 16);
    const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
    int tg = 0, units = 0;
    for (; ex_next(p, walk, u, k0, k1); ++units) {
      const int n = k1 - k0;
      const bool raw_k = ex_raw_k(p, u), bf16 = p.bf16 && u.kind == EX_TAIL;
      const uint32_t idS = exm_idesc(N, bf16, false);
      const uint32_t idPV = exm_idesc(N == 64 ? 64 : 2 * N, bf16, true);
      exm_wait(q_full, units & 1, p, abort);
      // turn i issues S of tile i and P V of tile i - 1
      for (int i = 0; i <= n; ++i) {
        if (i < n) {
          exm_wait(&k_full[tg & 1], (tg >> 1) & 1, p, abort);
          if (tg > 0) exm_wait(&s_empty[(tg - 1) & 1], ((tg - 1) >> 1) & 1, p, abort);
          tc_fence_after();
          const uint32_t a = base + C::K_COL + (tg % C::KB) * 64, d = base + C::S_COL;
          const bool stop = *abort != 0;
          if (stop && lane == 0) mbar_arrive(&s_full[tg & 1]);
          if (!stop && elect_one()) {
            if (raw_k) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                umma_f16_tmem_a(d, a + 8 * k, dQ + (k >> 2) * (N * 128 / 16) + (k & 3) * 2, idS, k > 0 ? 1u : 0u);
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint64_t q = dQ + (k >> 2) * (N * 128 / 16) + (k & 3) * 2;
                umma_f16_tmem_a(d + (k >> 1) * N, a + 8 * k, q, idS, (k & 1) ? 1u : 0u);
                umma_f16_tmem_a(d + (k >> 1) * N, a + 8 * k, q + C::Q_BYTES / 16, idS, 1u);
              }
            }
            umma_commit(&s_full[tg & 1]);
          }
          __syncwarp();
        }
        if (i > 0) {
          const int g = tg - 1;
          exm_wait(&p_full[g & 1], (g >> 1) & 1, p, abort);
          tc_fence_after();
          const bool stop = *abort != 0;
          if (stop && lane == 0) mbar_arrive(&pv_done[g & 1]);
          if (!stop && elect_one()) {
#pragma unroll
            for (int k = 0; k < EX_TILE / 16; ++k) {
              umma_f16_ss(base + C::O_COL, dV + k * 128, dP + k * 16, idPV, (i > 1 || k > 0) ? 1u : 0u);
              if (N == 64)                               // the weights' low halves
                umma_f16_ss(base + C::O_COL + 64, dV + k * 128, dP + 8 * (EX_TILE * 16) / 16 + k * 16, idPV,
                            (i > 1 || k > 0) ? 1u : 0u);
            }
            umma_commit(&pv_done[g & 1]);
          }
          __syncwarp();
        }
        if (i < n) ++tg;
      }
    }
    // nothing of this CTA may still run on the tensor cores when it exits
    if (elect_one()) {
      umma_commit(done);
      if (!mbar_wait(done, 0, p.wait_ns)) atomicOr(p.err, ERR_TIMEOUT);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- workers
    constexpr int RW = C::RW;
    constexpr int KBLOCKS = 4 / C::SW;                   // key blocks a thread unpacks
    constexpr int VROUND = 8 * C::WORKERS;               // positions of one round of value rows: 64 or 128
    const int group = warp >> 2, w4 = warp & 3;          // RW rows from row0; lanes 32 w4 .. of tensor memory
    const int row0 = RW * group, tok = 32 * w4 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * w4) << 16);
    // Value rows: a warp takes 8 positions x 4 blocks a round.  A phase of 8 lanes takes two
    // positions' blocks 0 1 and two positions' blocks 2 3 (or the other way round): its loads
    // and its stores both touch all banks once.
    const int vtok = 8 * warp + (lane >> 4) * 4 + ((lane & 7) >> 1);
    const int vblk = (lane & 1) | ((((lane >> 2) ^ (lane >> 3)) & 1) << 1);
    uint32_t voff[4];                                    // chunks 4 vblk .. of the thread's rows (all equal mod 8)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      voff[i] = (uint32_t)((vblk >> 1) * (EX_TILE * 128) + vtok * 128 + (((4 * (vblk & 1) + i) ^ (vtok & 7)) << 4));
    int tg = 0;
    Stage st{0, 0u, 0};
    const int page_stage = p.page_stage;
    while (ex_next(p, walk, u, k0, k1)) {
      const int n = k1 - k0;
      int begin, end;
      ex_range(p, u, &begin, &end);
      const HeadInfo& h = p.heads[u.head];
      const bool raw_k = ex_raw_k(p, u), raw_v = ex_raw_v(p, u), tail = u.kind == EX_TAIL;
      const int kcodec = KC >= 0 ? KC : h.kcodec, vcodec = VC >= 0 ? VC : h.vcodec;
      int cbK, sbK, cbV, sbV;                            // constants where the codecs are
      if (KC >= 0 && KC != KVQ_RANK) row_bytes(KC, D, 0, &cbK, &sbK); else { cbK = h.cbK; sbK = h.sbK; }
      if (VC >= 0 && VC != KVQ_RANK) row_bytes(VC, D, 0, &cbV, &sbV); else { cbV = h.cbV; sbV = h.sbV; }
      const int v_at = PAGE * (cbK + sbK);
      const bool asym = !raw_k && codec_is_asym(kcodec), bf16_pv = p.bf16 && tail;
      const float bias = bf16_pv ? 0.f : EXM_BIAS;
      const int base = u.kind == EX_SHARED ? 0x7fffffff : p.len[u.index] - p.nq[u.index];
      const int pos_first = begin + k0 * EX_TILE;
      // a group whose rows are all padding only unpacks
      const int blocks = u.block * p.QB, queries = (u.kind == EX_SHARED ? p.g_nq[u.index] : p.nq[u.index]) - blocks;
      const bool active = row0 < min(queries, p.QB) * p.G;
      const int edge = min(end, base) - tok;             // tiles from here on hold a position outside or masked
      const uint8_t* ring =
          tail ? p.tail + (((size_t)p.seq[u.index] * p.L + p.layer) * p.Hkv + u.head) * (size_t)p.T * (D * 2 * 2) : nullptr;
      // ---- the group's query rows, RW / 4 per warp: all loads first, then the rows in step
      // (row after row every shuffle's latency counted)
      constexpr int QR = RW / 4;
      if (active) {
        uint2 bits[QR];
        int query[QR];                                   // of its entry (-1: padding)
        unsigned long long mask[QR];
        float4 sk = make_float4(1.f, 1.f, 1.f, 1.f);
        if (KC != KVQ_RANK && !raw_k && p.rot != KVQ_ROT_NONE && p.s_k) sk = *reinterpret_cast<const float4*>(p.s_k + (size_t)u.head * D + 4 * lane);
#pragma unroll
        for (int k = 0; k < QR; ++k) {
          const ExtendRow w = ex_row(p, u, row0 + QR * w4 + k);
          const int index = w.entry < 0 ? 0 : p.q0[w.entry] + w.query;
          query[k] = w.entry < 0 ? -1 : w.query;
          bits[k] = make_uint2(0u, 0u);
          mask[k] = 0ull;
          if (w.entry >= 0) {
            bits[k] = *reinterpret_cast<const uint2*>(p.q + ((size_t)index * p.Hq + w.head) * D + 4 * lane);
            if (p.mask) mask[k] = p.mask[index];
          }
        }
        const int c = lane >> 1;                         // the lane's 16-byte chunk (8 channels)
        uint8_t* at[QR];
        float f[QR];
#pragma unroll
        for (int k = 0; k < QR; ++k) {
          const int r = row0 + QR * w4 + k;
          at[k] = sQ + (c >> 3) * (N * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4) + 8 * (lane & 1);
          f[k] = p.qscale;
        }
        if (raw_k) {
#pragma unroll
          for (int k = 0; k < QR; ++k) *reinterpret_cast<uint2*>(at[k]) = bits[k];
        } else {
          float x[QR][4], big[QR], sum[QR];
#pragma unroll
          for (int k = 0; k < QR; ++k) {
            const float2 x01 = raw2_to_float2(bits[k].x, p.bf16), x23 = raw2_to_float2(bits[k].y, p.bf16);
            x[k][0] = x01.x * sk.x; x[k][1] = x01.y * sk.y; x[k][2] = x23.x * sk.z; x[k][3] = x23.y * sk.w;
          }
          if (KC == KVQ_RANK) {
            // the warp's rows at once: eight rows of M_h a step, 32 / (8 QR) lanes end with each sum
            float* z = reinterpret_cast<float*>(sV) + (row0 + QR * w4) * D;   // the V image is free between units
            const float* M = p.M + h.m_off + 4 * lane;
#pragma unroll 1
            for (int i = 0; i < D; i += 8) {
              float s[8 * QR];                           // [row][8]
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < h.r) m = *reinterpret_cast<const float4*>(M + (size_t)(i + e) * D);
#pragma unroll
                for (int k = 0; k < QR; ++k)
                  s[8 * k + e] = fmaf(m.x, x[k][0], fmaf(m.y, x[k][1], fmaf(m.z, x[k][2], m.w * x[k][3])));
              }
              int at = 0;
#pragma unroll
              for (int m = 16, n = 8 * QR; m; m >>= 1) {
                if (n > 1) {
                  n >>= 1;
                  const bool up = lane & m;
                  at += up ? n : 0;
#pragma unroll
                  for (int e = 0; e < n; ++e) {
                    const float keep = up ? s[n + e] : s[e], give = up ? s[e] : s[n + e];
                    s[e] = keep + __shfl_xor_sync(0xffffffffu, give, m);
                  }
                } else {
                  s[0] += __shfl_xor_sync(0xffffffffu, s[0], m);
                }
              }
              z[(at >> 3) * D + i + (at & 7)] = s[0];    // lanes with the same sum write it twice
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < QR; ++k) {
              const float4 y = *reinterpret_cast<const float4*>(z + k * D + 4 * lane);
              x[k][0] = y.x; x[k][1] = y.y; x[k][2] = y.z; x[k][3] = y.w;
            }
          } else if (p.rot != KVQ_ROT_NONE) {
#pragma unroll
            for (int k = 0; k < QR; ++k) fwht_row(x[k]);
          }
#pragma unroll
          for (int k = 0; k < QR; ++k) big[k] = fmaxf(fmaxf(fabsf(x[k][0]), fabsf(x[k][1])), fmaxf(fabsf(x[k][2]), fabsf(x[k][3])));
#pragma unroll
          for (int m = 16; m; m >>= 1)
#pragma unroll
            for (int k = 0; k < QR; ++k) big[k] = fmaxf(big[k], __shfl_xor_sync(0xffffffffu, big[k], m));
#pragma unroll
          for (int k = 0; k < QR; ++k) {
            // a power of two that brings the largest element into [2^11, 2^12); f takes it back
            const int e = (int)(__float_as_uint(big[k]) >> 23) - 127;
            const bool in = e > -100 && e < 100;
            const float up = in ? __uint_as_float((uint32_t)(127 + 11 - e) << 23) : 1.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[k][i] *= up;
            f[k] *= in ? __uint_as_float((uint32_t)(127 - 11 + e) << 23) : 1.f;
            sum[k] = (x[k][0] + x[k][1]) + (x[k][2] + x[k][3]);
          }
#pragma unroll
          for (int m = 1; m < 8; m <<= 1)
#pragma unroll
            for (int k = 0; k < QR; ++k) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], m);
          if ((lane & 7) == 0)
#pragma unroll
            for (int k = 0; k < QR; ++k) r_qsum[(lane >> 3) * N + row0 + QR * w4 + k] = sum[k];
          if (KC != KVQ_RANK && h.kbits == 4) {
            // positions 0 4 1 5 | 2 6 3 7: the even lane of a pair takes channels 0 4 1 5
            const bool odd = lane & 1;
#pragma unroll
            for (int k = 0; k < QR; ++k) {
              const float ra = __shfl_xor_sync(0xffffffffu, odd ? x[k][0] : x[k][2], 1);
              const float rb = __shfl_xor_sync(0xffffffffu, odd ? x[k][1] : x[k][3], 1);
              const float y0 = odd ? ra : x[k][0], y1 = odd ? x[k][2] : ra, y2 = odd ? rb : x[k][1], y3 = odd ? x[k][3] : rb;
              x[k][0] = y0; x[k][1] = y1; x[k][2] = y2; x[k][3] = y3;
            }
          }
#pragma unroll
          for (int k = 0; k < QR; ++k) {
            const __half2 h0 = __floats2half2_rn(x[k][0], x[k][1]), h1 = __floats2half2_rn(x[k][2], x[k][3]);
            const float2 g0 = __half22float2(h0), g1 = __half22float2(h1);
            *reinterpret_cast<uint2*>(at[k]) = make_uint2(as_u32(h0), as_u32(h1));
            *reinterpret_cast<uint2*>(at[k] + C::Q_BYTES) =
                make_uint2(as_u32(__floats2half2_rn(x[k][0] - g0.x, x[k][1] - g0.y)),
                           as_u32(__floats2half2_rn(x[k][2] - g1.x, x[k][3] - g1.y)));
          }
        }
        if (lane == 0)
#pragma unroll
          for (int k = 0; k < QR; ++k) {
            const int r = row0 + QR * w4 + k;
            r_f[r] = f[k];
            r_use[r] = EXM_NONE;
            r_max[r] = -INFINITY;
            r_query[r] = query[k];
            r_mask[r] = mask[k];
          }
      }
      fence_proxy_async_shared();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      group_sync(group);                                 // the group's row words are written

      // the position's key scales and minima, of the tile in hand and of the next
      float dk[4] = {0.f, 0.f, 0.f, 0.f}, mk[4] = {0.f, 0.f, 0.f, 0.f};
      float d_next[4] = {0.f, 0.f, 0.f, 0.f}, m_next[4] = {0.f, 0.f, 0.f, 0.f};
      float l[RW];
#pragma unroll
      for (int r = 0; r < RW; ++r) l[r] = 0.f;
      Stage held = st;                                   // of the tile in hand
      bool raw_seen = !tail && exm_look(&raw_full[st.i], st.phase);
      // Turn i takes the scores of tile i, unpacks the keys of tile i + 1 (or the other way
      // round) and finishes tile i.
#pragma unroll 1
      for (int i = -1; i < n; ++i) {
        const int pos0 = pos_first + i * EX_TILE;        // of tile i
        float x[RW];                                     // log2 of the weights of tile i
        const bool s_seen = i >= 0 && exm_look(&s_full[tg & 1], (tg >> 1) & 1);
        const Stage next = st;
        auto take_scores = [&]() {
          // ---- scores of this position, accumulator units
          exm_wait_if(s_seen, &s_full[tg & 1], (tg >> 1) & 1, p, abort);
          if (!active) {
            if (lane == 0) mbar_arrive(&s_empty[tg & 1]);
            return;
          }
          tc_fence_after();
          float a[RW];
          const uint32_t s_col = lanes + C::S_COL + row0;
          if (raw_k) {
#pragma unroll
            for (int c = 0; c < RW / 8; ++c) {
              uint32_t v[8];
              tmem_ld8_wait(s_col + 8 * c, v);
#pragma unroll
              for (int r = 0; r < 8; ++r) a[8 * c + r] = __uint_as_float(v[r]);
            }
          } else {
#pragma unroll
            for (int c = 0; c < RW / 8; ++c) {
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
              for (int r = 0; r < RW; r += 4) {
                const float4 s = *reinterpret_cast<const float4*>(&r_qsum[b * N + row0 + r]);
                a[r] = fmaf(mk[b], s.x, a[r]);
                a[r + 1] = fmaf(mk[b], s.y, a[r + 1]);
                a[r + 2] = fmaf(mk[b], s.z, a[r + 2]);
                a[r + 3] = fmaf(mk[b], s.w, a[r + 3]);
              }
          }
          if (pos0 >= edge) {
            const int pos = pos0 + tok;
            // outside the range, or one of the entry's new tokens
            bool spoils = false;                         // a raw value row with NaN or infinity
            if (raw_v && pos < end) {
              const uint8_t* src;
              if (tail) {
                const int slot = pos % p.T;
                src = ring + (size_t)(slot / TAIL_TOK) * TAIL_PAGE_BYTES + TAIL_TOK * D * 2 + (slot % TAIL_TOK) * (D * 2);
              } else {
                // the page's stage may be gone by now: read the row from the page itself
                const int id = max(0, p.table[(size_t)p.seq[u.index] * p.mpps + pos / PAGE]);
                src = p.pool + (size_t)id * p.page_bytes + h.off + v_at + (pos % PAGE) * cbV;
              }
#pragma unroll 1
              for (int c = 0; c < 16; c += 8) {          // eight loads in flight
                uint4 v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = *reinterpret_cast<const uint4*>(src + 16 * (c + e));
#pragma unroll
                for (int e = 0; e < 8; ++e) spoils |= !finite_words(v[e], p.bf16);
              }
            }
            const int j = pos - base;
#pragma unroll
            for (int r = 0; r < RW; ++r) {
              const bool sees = pos < end && (j < 0 || (p.mask ? (r_mask[row0 + r] >> j) & 1ull : j <= r_query[row0 + r]));
              a[r] = !sees ? -INFINITY : spoils ? __uint_as_float(0x7fc00000u) : a[r];
            }
          }
          // ---- log2 of the weights, against the maximum in use
          float top = -INFINITY;
          auto against_max = [&]() {
#pragma unroll
            for (int r = 0; r < RW; r += 4) {
              const float4 f = *reinterpret_cast<const float4*>(&r_f[row0 + r]);
              const float4 m = *reinterpret_cast<const float4*>(&r_use[row0 + r]);
              x[r] = fmaf(a[r], f.x, -m.x);
              x[r + 1] = fmaf(a[r + 1], f.y, -m.y);
              x[r + 2] = fmaf(a[r + 2], f.z, -m.z);
              x[r + 3] = fmaf(a[r + 3], f.w, -m.w);
            }
          };
          against_max();
#pragma unroll
          for (int r = 0; r < RW; ++r) top = fmaxf(top, x[r]);
          if (group_any(group, top > EXM_RESCALE + bias)) {
#pragma unroll
            for (int r = 0; r < RW; ++r) {
              float m = a[r];
#pragma unroll
              for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
              if (lane == 0) r_part[w4 * N + row0 + r] = m;
            }
            group_sync(group);
            if (w4 == 0 && lane < RW) {
              const int r = row0 + lane;
              const float old = r_max[r];
              const float most = fmaxf(fmaxf(r_part[r], r_part[N + r]), fmaxf(r_part[2 * N + r], r_part[3 * N + r])) * r_f[r];
              const float m = fmaxf(old, most);
              r_alpha[r] = m == old ? 1.f : exm_ex2(old - m);
              r_max[r] = m;
              r_use[r] = m == -INFINITY ? EXM_NONE : m - bias;
            }
            group_sync(group);
            against_max();
#pragma unroll
            for (int r = 0; r < RW; ++r) l[r] *= r_alpha[row0 + r];
            if (i > 0) {                                 // O holds the tiles before this one
              exm_wait(&pv_done[(tg - 1) & 1], ((tg - 1) >> 1) & 1, p, abort);
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < RW / 4; ++c) {         // both halves of O
                const uint32_t o = lanes + C::O_COL + (c / (RW / 8)) * N + row0 + 8 * (c % (RW / 8));
                const float* al = &r_alpha[row0 + 8 * (c % (RW / 8))];
                uint32_t v[8];
                tmem_ld8_wait(o, v);
#pragma unroll
                for (int r = 0; r < 8; ++r) v[r] = __float_as_uint(__uint_as_float(v[r]) * al[r]);
                tmem_st8(o, v);
              }
              tmem_wait_st();
            }
          }
        };
        auto unpack_keys = [&]() {
          // ---- keys of tile i + 1
          const int g = i < 0 ? tg : tg + 1, kpos0 = pos0 + EX_TILE;
          const uint32_t col = lanes + C::K_COL + (g % C::KB) * 64;
          if (!tail) {
            exm_wait_if(raw_seen, &raw_full[st.i], st.phase, p, abort);
            st.next(NR, 2 * page_stage);
          }
          const uint8_t* region = sRaw + next.at + (w4 < 2 ? 0 : page_stage);
          if (raw_k) {
            const uint8_t* src = region + (tok % PAGE) * 16;
            int step = PAGE * 16;
            if (tail) {
              const int slot = (kpos0 + tok) % p.T;
              src = ring + (size_t)(slot / TAIL_TOK) * TAIL_PAGE_BYTES + (slot % TAIL_TOK) * 16;
              step = TAIL_TOK * 16;
            }
            const bool valid = kpos0 + tok < end;
#pragma unroll
            for (int k = 0; k < KBLOCKS; k += 2) {       // the loads of two blocks go out together
              uint32_t W[2][16];
#pragma unroll
              for (int e = 0; e < (KBLOCKS < 2 ? 1 : 2); ++e)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  uint4 v = make_uint4(0u, 0u, 0u, 0u);
                  if (valid) v = *reinterpret_cast<const uint4*>(src + (size_t)(4 * (group * KBLOCKS + k + e) + c) * step);
                  W[e][4 * c] = v.x; W[e][4 * c + 1] = v.y; W[e][4 * c + 2] = v.z; W[e][4 * c + 3] = v.w;
                }
              __syncwarp();
#pragma unroll
              for (int e = 0; e < (KBLOCKS < 2 ? 1 : 2); ++e) tmem_st16(col + 16 * (group * KBLOCKS + k + e), W[e]);
            }
          } else {
            const uint8_t* scales = region + PAGE * cbK + (tok % PAGE) * sbK;
            if (KC == KVQ_RANK) {
#pragma unroll
              for (int b = 0; b < 4; ++b) d_next[b] = rank_scale(scales, h.r, b);
            } else if (asym) {
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
  case CODEC: key_blocks<B, A, KBLOCKS>(region + (tok % PAGE) * 16, cbK, group * KBLOCKS, col); break;
            if (KC == KVQ_RANK) {
#pragma unroll 1
              for (int b = group * KBLOCKS; b < (group + 1) * KBLOCKS; ++b) {
                uint32_t W[16];
                switch (h.kbits) {
                  case 1: rank_block<1>(region, cbK, tok % PAGE, true, h.r, b, W); break;
                  case 2: rank_block<2>(region, cbK, tok % PAGE, true, h.r, b, W); break;
                  case 3: rank_block<3>(region, cbK, tok % PAGE, true, h.r, b, W); break;
                  default: rank_block<4>(region, cbK, tok % PAGE, true, h.r, b, W);
                }
                __syncwarp();
                tmem_st16(col + 16 * b, W);
              }
            } else {
              switch (kcodec) {
                KVQ_EXM_CODECS(KVQ_EXM_CASE)
                default: break;
              }
            }
#undef KVQ_EXM_CASE
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&k_full[g & 1]);
        };
        if (C::KEYS_FIRST && i + 1 < n) unpack_keys();
        if (i >= 0) take_scores();
        if (!C::KEYS_FIRST && i + 1 < n) unpack_keys();
        if (i >= 0) {
          const bool pv_seen = i > 0 && exm_look(&pv_done[(tg - 1) & 1], ((tg - 1) >> 1) & 1);
          // ---- values of tile i (its V and P images are free once P V of the tile before is done)
          if (i > 0) exm_wait_if(pv_seen, &pv_done[(tg - 1) & 1], ((tg - 1) >> 1) & 1, p, abort);
          if (raw_v) {
            // 16 neighbouring threads read one 256-byte row; the loads of four rows go out
            // together (their latency is all this path takes)
            constexpr int STEP = 2 * C::WORKERS;
            const int c = lane & 15;
            int row = 2 * warp + (lane >> 4);
            int slot = tail ? (pos0 + row) % p.T : 0;
#pragma unroll 1
            for (int k = 0; k < EX_TILE / STEP; k += 4) {
              uint4 v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint8_t* src =
                    tail ? ring + (size_t)(slot / TAIL_TOK) * TAIL_PAGE_BYTES + TAIL_TOK * D * 2 + (slot % TAIL_TOK) * (D * 2)
                         : sRaw + held.at + (row + e * STEP < PAGE ? 0 : page_stage) + v_at + ((row + e * STEP) % PAGE) * cbV;
                v[e] = make_uint4(0u, 0u, 0u, 0u);
                if (pos0 + row + e * STEP < end) v[e] = *reinterpret_cast<const uint4*>(src + 16 * c);
                slot += STEP;
                if (slot >= p.T) slot -= p.T;            // T is at least 64
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (pos0 + row >= base) {                // rows may mask this position: nothing non-finite may reach them
                  v[e].x = finite_or_zero(v[e].x, p.bf16);
                  v[e].y = finite_or_zero(v[e].y, p.bf16);
                  v[e].z = finite_or_zero(v[e].z, p.bf16);
                  v[e].w = finite_or_zero(v[e].w, p.bf16);
                }
                *reinterpret_cast<uint4*>(sV + (c >> 3) * (EX_TILE * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = v[e];
                row += STEP;
              }
            }
          } else if (VC == KVQ_RANK) {
#pragma unroll 1
            for (int k = 0; k < EX_TILE; k += VROUND) {
              const uint8_t* page = sRaw + held.at + (VROUND == PAGE ? k / PAGE : vtok / PAGE) * page_stage + v_at;
              const int t = vtok % PAGE;
              uint32_t W[16];
              switch (h.vbits) {
                case 1: rank_block<1>(page, cbV, t, false, h.r, vblk, W); break;
                case 2: rank_block<2>(page, cbV, t, false, h.r, vblk, W); break;
                case 3: rank_block<3>(page, cbV, t, false, h.r, vblk, W); break;
                default: rank_block<4>(page, cbV, t, false, h.r, vblk, W);
              }
              const float d = pos0 + k + vtok < end ? rank_scale(page + PAGE * cbV + t * sbV, h.r, vblk) : 0.f;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float2 c = __half22float2(as_h2(W[4 * e + j]));
                  w[j] = as_u32(__floats2half2_rn(c.x * d, c.y * d));
                }
                *reinterpret_cast<uint4*>(sV + k * 128 + voff[e]) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          } else {
#define KVQ_EXM_CASE(CODEC, B, A)                                                                             \
  case CODEC:                                                                                                 \
    _Pragma("unroll") for (int k = 0; k < EX_TILE; k += VROUND) {                                             \
      const uint8_t* page = sRaw + held.at + (VROUND == PAGE ? k / PAGE : vtok / PAGE) * page_stage + v_at;   \
      const int t = vtok % PAGE;                                                                              \
      value_block<B, A>(page + t * cbV, page + PAGE * cbV + t * sbV, cbV, vblk, pos0 + k + vtok < end,        \
                        sV + k * 128, voff);                                                                  \
    }                                                                                                         \
    break;
            switch (vcodec) {
              KVQ_EXM_CODECS(KVQ_EXM_CASE)
              default: break;
            }
#undef KVQ_EXM_CASE
          }
          if (!tail) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&raw_empty[held.i]);
          }
          // ---- weights: fp32 sums, and two halves into the P image
          uint8_t* img = sP + (size_t)(row0 >> 3) * (EX_TILE * 16) + tok * 16;
          if (active)
#pragma unroll
          for (int c = 0; c < RW / 8; ++c) {
            uint32_t hi[4], lo[4];
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              w[e] = exm_ex2(x[8 * c + e]);
              l[8 * c + e] += w[e];
            }
            if (bf16_pv) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 g = __bfloat1622float2(__floats2bfloat162_rn(w[2 * e], w[2 * e + 1]));
                hi[e] = float2_to_raw2(g.x, g.y, true);
                lo[e] = float2_to_raw2(w[2 * e] - g.x, w[2 * e + 1] - g.y, true);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __half2 h2 = __floats2half2_rn(w[2 * e], w[2 * e + 1]);
                const float2 g = __half22float2(h2);
                hi[e] = as_u32(h2);
                const float2 r = sub_scale2(make_float2(w[2 * e], w[2 * e + 1]), g, EXM_LOW);
                lo[e] = as_u32(__floats2half2_rn(r.x, r.y));
              }
            }
            *reinterpret_cast<uint4*>(img + (size_t)c * (EX_TILE * 16)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(img + (size_t)(N / 8 + c) * (EX_TILE * 16)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
          fence_proxy_async_shared();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[tg & 1]);
          ++tg;
        }
        held = next;
#pragma unroll
        for (int b = 0; b < 4; ++b) { dk[b] = d_next[b]; mk[b] = m_next[b]; }
        raw_seen = !tail && exm_look(&raw_full[st.i], st.phase);   // of the tile after the next
      }
      // ---- the unit's partial result: O^T (lane = channel position), sums, maximum
      const size_t slot = (size_t)blockIdx.x + u.unit;
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        float s = l[r];
#pragma unroll
        for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
        if (lane == 0) r_part[w4 * N + row0 + r] = s;
      }
      exm_wait(&pv_done[(tg - 1) & 1], ((tg - 1) >> 1) & 1, p, abort);
      tc_fence_after();
      const int channel = (tok & ~7) | group_channel(tok & 7, VC != KVQ_RANK && !raw_v && h.vbits == 4);
      float* dst = p.part_o + (slot * N + row0) * D + channel;
      const float low = bf16_pv ? 1.f : 1.f / EXM_LOW;
      float spoilt = 0.f;                                // NaN where a value is not finite
#pragma unroll
      for (int c = 0; c < RW / 8; ++c) {
        uint32_t o[8], q[8];
        tmem_ld8_wait(lanes + C::O_COL + row0 + 8 * c, o);
        tmem_ld8_wait(lanes + C::O_COL + N + row0 + 8 * c, q);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float x = fmaf(__uint_as_float(q[r]), low, __uint_as_float(o[r]));
          spoilt = fmaf(x, 0.f, spoilt);
          if (active && r_query[row0 + 8 * c + r] >= 0) dst[(size_t)(8 * c + r) * D] = x;
        }
      }
      if (active && spoilt != 0.f) *again = 1;
      group_sync(group);
      if (w4 == 0 && lane < RW) {
        const int r = row0 + lane;
        const float s = (r_part[r] + r_part[N + r]) + (r_part[2 * N + r] + r_part[3 * N + r]);
        if (active && r_query[r] >= 0) p.part_ml[slot * N + r] = make_float2(r_max[r] - bias, s);
      }
      tc_fence_before();
      group_sync(group);                                 // the row words may be overwritten
    }
  }
  if (p.chain == EX_ENTRIES) griddep_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == C::WORKERS + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::COLS) : "memory");
  }
  if (*again && !*abort) exm_again(p, warp, C::WORKERS + 2, reinterpret_cast<float*>(sV));
}

template <int N, int CT, int KC, int VC>
static cudaError_t launch(const ExtendParams& p, cudaStream_t s) {
  const auto kernel = extend_mma_kernel<N, CT, KC, VC>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, EXM_SMEM_MAX);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.n_ctas);
  cfg.blockDim = dim3(Shape<N, CT>::THREADS);
  cfg.dynamicSmemBytes = (size_t)Shape<N, CT>::OFF_RAW + (size_t)p.n_raw * 2 * p.page_stage;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t l = cudaLaunchKernelEx(&cfg, kernel, p);
  note_launches(1);
  return l;
}
// Layers whose heads all hold 4-bit values of one codec, with keys in the same codec or (q4_0) in
// q8_0, have kernels of their own, and so have projection plans; everything else takes the kernel
// that reads the codecs per head.  A kernel of its own has no dispatch in its loops and saves 10
// to 17 % (32 query heads over 8; 64 sequences of 1000 to 8000 x 4 drafts: q4_0 / q4_0 205 us,
// 246 with the common kernel; q8_0 / q4_0 212, 254; q4_1 / q4_1 221, 258; 16 of them x 16:
// 130, 148; 131, 152; 144, 168), and costs three instantiations, so the pairs that caches are
// most often held in have one.  The common kernel on others, the same 64 sequences: q4_0 / q4_1
// 245, q8_0 / q8_0 274, q6_0 / q6_0 375.
// One CTA of 16 rows an SM (CT = 1) is taken only where two CTAs' stages of page-heads do not fit,
// which those of these pairs do.
template <int N, int CT>
static cudaError_t launch_codecs(const ExtendParams& p, cudaStream_t s) {
  if (p.rot == KVQ_ROT_PROJECTION) return launch<N, CT, KVQ_RANK, KVQ_RANK>(p, s);
  if constexpr (N > 16 || CT == 2) {
    int kc = p.heads[0].kcodec, vc = p.heads[0].vcodec;
    for (int h = 1; h < p.Hkv; ++h)
      if (p.heads[h].kcodec != kc || p.heads[h].vcodec != vc) kc = -1;
    if (kc == KVQ_Q4_0 && vc == KVQ_Q4_0) return launch<N, CT, KVQ_Q4_0, KVQ_Q4_0>(p, s);
    if (kc == KVQ_Q8_0 && vc == KVQ_Q4_0) return launch<N, CT, KVQ_Q8_0, KVQ_Q4_0>(p, s);
    if (kc == KVQ_Q4_1 && vc == KVQ_Q4_1) return launch<N, CT, KVQ_Q4_1, KVQ_Q4_1>(p, s);
  }
  return launch<N, CT, -1, -1>(p, s);
}

template <int N, int CT>
static int stages(int page_stage) {
  // two CTAs share an SM's 228 KiB (1 KiB of each is reserved)
  const int n = (std::min(EXM_SMEM_MAX, 228 * 1024 / CT - 1024) - Shape<N, CT>::OFF_RAW) / (2 * page_stage);
  return n < EXM_MIN_STAGES ? 0 : std::min(n, 8);
}
ExtendShape extend_mma_shape(int N, int page_stage) {
  if (N == 64) return ExtendShape{1, stages<64, 1>(page_stage)};
  if (N == 32) return ExtendShape{1, stages<32, 1>(page_stage)};
  if (const int two = stages<16, 2>(page_stage)) return ExtendShape{2, two};
  return ExtendShape{1, stages<16, 1>(page_stage)};      // large page-heads: one CTA with the whole SM's ring
}

cudaError_t launch_extend_mma(const ExtendParams& p, cudaStream_t s) {
  if (p.N == 64) return launch_codecs<64, 1>(p, s);
  if (p.N == 32) return launch_codecs<32, 1>(p, s);
  return p.ctas_per_sm == 2 ? launch_codecs<16, 2>(p, s) : launch_codecs<16, 1>(p, s);
}

}  // namespace kvq
