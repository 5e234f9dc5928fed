// Attention of the last n_q tokens of several sequences (kvq_extend_attention): the work
// list of a launch (a call has one or two, see EX_ALONE), the kernel that walks it and the
// merge of the partial results.
//
// Three kinds of token ranges are walked in tiles of 128 positions: the pages that a
// group of sequences shares (every query of the group sees all of them), a sequence's
// own pages behind those, and its raw tail.  A unit is one range, one kv head and one
// block of `QB` queries (QB * G rows of at most `N`).  All tiles of all units form one
// axis, units in order, a tile as long as it is costly (`page_cost`, or `tail_cost` for a
// raw tail tile, a unit's first tile `unit_cost` more); CTA c takes the tiles that start in
// [c per, (c + 1) per), so every CTA has about the same work whatever the lengths.  Where a CTA's run and a unit meet it
// writes one partial result (running maximum, sum, unnormalised output); walking the
// axis, either the CTA or the unit steps on from one partial to the next, so partial
// (c, u) has slot c + u to itself and no counter is needed.  `per` is no shorter than any
// tile, so a unit has a partial in every CTA from its first to its last.
#pragma once

#include "kvq_internal.h"

namespace kvq {

constexpr int EX_TILE = 128;
constexpr int EX_MAX_ROWS = 64;
constexpr int EX_SHARED = 0, EX_OWN = 1, EX_TAIL = 2;
// Launches of a call: one of all units, or one of the groups' and one of the entries' own,
// which have fewer rows.  The second starts when the first has begun (and so everything
// before it is complete) and ends after it.
constexpr int EX_ALONE = 0, EX_GROUPS = 1, EX_ENTRIES = 2;

struct ExtendParams {
  const uint8_t* pool;           // the layer's page pool
  uint32_t page_bytes;
  const int* table;              // block table [max_seqs][mpps]
  int mpps;
  const uint8_t* tail;
  int T, L, layer, Hkv, Hq, G;
  int rot;
  int bf16;
  const __half* q;               // [total_q][Hq][128] raw 16-bit
  __half* out;                   // [total_q][Hq][128] raw 16-bit
  const unsigned long long* mask;   // [total_q] or null (causal)
  const float* s_k;              // [Hkv][128] or null
  const float* s_v;
  const float* M;
  float qscale;                  // softmax scale * log2(e)
  int* err;
  unsigned long long wait_ns;
  int drop_last_tile;            // test-only fault injection: producers skip their last tile of pages
  float* part_o;                 // [slots][N][128]
  float2* part_ml;               // [slots][N]: what the weights are taken against (log2 units), their sum
  int N, QB;                     // rows of a unit, queries of a block
  int n_entries, n_groups, total_q;
  int page_cost, tail_cost, unit_cost;
  int total, per, n_ctas;        // the axis: length, length per CTA, CTAs
  int page_stage, n_raw;         // bytes of a page in a stage, stages of two pages,
  int ctas_per_sm;               // CTAs an SM
  int chain;                     // EX_ALONE, or one of two launches of a call
  HeadInfo heads[MAX_HKV];
  // entries, in call order
  int seq[MAX_BATCH], len[MAX_BATCH], nq[MAX_BATCH];
  int q0[MAX_BATCH + 1];         // first query row
  int own0[MAX_BATCH];           // positions below this are the group's
  int member0[MAX_BATCH];        // first query among the group's queries
  int16_t group[MAX_BATCH];      // -1: none
  // groups
  int g_tok[MAX_BATCH / 2];      // shared positions
  int g_nq[MAX_BATCH / 2];       // queries of all members
  int g_first[MAX_BATCH / 2 + 1];   // first member in `order`
  uint8_t order[MAX_BATCH];      // entries by group
  // prefix sums along the axis and of the units: the groups, then the entries
  int s_at[MAX_BATCH / 2 + 1], s_unit[MAX_BATCH / 2 + 1];
  int e_at[MAX_BATCH + 1], e_unit[MAX_BATCH + 1];
};

__host__ __device__ inline int ex_tiles(int tokens) { return (tokens + EX_TILE - 1) / EX_TILE; }
__host__ __device__ inline int ex_paged(const ExtendParams& p, int e) { return p.len[e] > p.T ? p.len[e] - p.T : 0; }

// A unit and its place on the axis.
struct ExtendUnit {
  int kind, index, head, block;  // index: the group (EX_SHARED) or the entry
  int unit;                      // ordinal of the unit
  int at, tiles, cost;           // where its first tile starts, its tiles, the length of the others
};
__host__ __device__ inline int ex_length(const ExtendParams& p, int kind, int tiles) {   // of a unit
  return tiles ? p.unit_cost + tiles * (kind == EX_TAIL ? p.tail_cost : p.page_cost) : 0;
}
__host__ __device__ inline int ex_start(const ExtendParams& p, const ExtendUnit& u, int k) {   // of tile k
  return u.at + (k ? p.unit_cost + k * u.cost : 0);
}
__host__ __device__ inline int ex_unit_tiles(const ExtendParams& p, int kind, int index) {
  return kind == EX_SHARED ? ex_tiles(p.g_tok[index])
         : kind == EX_OWN  ? ex_tiles(ex_paged(p, index) - p.own0[index])
                           : ex_tiles(p.len[index] - ex_paged(p, index));
}
__host__ __device__ inline int ex_blocks(const ExtendParams& p, int queries) { return (queries + p.QB - 1) / p.QB; }
// An entry's part of the axis is, kv head by kv head, its own pages' units and then its
// tail's, so that tails are spread over the CTAs.
__host__ __device__ inline ExtendUnit ex_unit(const ExtendParams& p, int kind, int index, int head, int block) {
  ExtendUnit u;
  u.kind = kind;
  u.index = index;
  u.head = head;
  u.block = block;
  u.tiles = ex_unit_tiles(p, kind, index);
  u.cost = kind == EX_TAIL ? p.tail_cost : p.page_cost;
  if (kind == EX_SHARED) {
    const int k = head * ex_blocks(p, p.g_nq[index]) + block;
    u.unit = p.s_unit[index] + k;
    u.at = p.s_at[index] + k * ex_length(p, kind, u.tiles);
    return u;
  }
  const int nb = ex_blocks(p, p.nq[index]);
  const int to = kind == EX_OWN ? u.tiles : ex_unit_tiles(p, EX_OWN, index);
  const int tt = kind == EX_TAIL ? u.tiles : ex_unit_tiles(p, EX_TAIL, index);
  const int lo = ex_length(p, EX_OWN, to), lt = ex_length(p, EX_TAIL, tt);
  u.unit = p.e_unit[index] + nb * head * ((to > 0) + (tt > 0)) + block;
  u.at = p.e_at[index] + nb * head * (lo + lt);
  if (kind == EX_OWN) {
    u.at += block * lo;
  } else {
    u.unit += nb * (to > 0);
    u.at += nb * lo + block * lt;
  }
  return u;
}
// The unit that covers place x of the axis.
__host__ __device__ inline ExtendUnit ex_find(const ExtendParams& p, int x) {
  if (x < p.e_at[0]) {
    const int g = prefix_find(p.s_at, p.n_groups, x), nb = ex_blocks(p, p.g_nq[g]);
    const int k = (x - p.s_at[g]) / ex_length(p, EX_SHARED, ex_unit_tiles(p, EX_SHARED, g));
    return ex_unit(p, EX_SHARED, g, k / nb, k % nb);
  }
  const int e = prefix_find(p.e_at, p.n_entries, x), nb = ex_blocks(p, p.nq[e]);
  const int lo = ex_length(p, EX_OWN, ex_unit_tiles(p, EX_OWN, e)), lt = ex_length(p, EX_TAIL, ex_unit_tiles(p, EX_TAIL, e));
  const int head = (x - p.e_at[e]) / (nb * (lo + lt)), rest = (x - p.e_at[e]) % (nb * (lo + lt));
  if (rest < nb * lo) return ex_unit(p, EX_OWN, e, head, rest / lo);
  return ex_unit(p, EX_TAIL, e, head, (rest - nb * lo) / lt);
}
// A CTA's walk over its part of the axis: the next unit of which it has tiles, [k0, k1).
struct ExtendWalk { int x, end; };
__host__ __device__ inline ExtendWalk ex_walk(const ExtendParams& p, int cta) {
  const int x = cta * p.per;
  return ExtendWalk{x, x + p.per < p.total ? x + p.per : p.total};
}
__host__ __device__ inline bool ex_next(const ExtendParams& p, ExtendWalk& w, ExtendUnit& u, int& k0, int& k1) {
  while (w.x < w.end) {
    u = ex_find(p, w.x);
    // the first tile that starts at or behind a place
    const int a = w.x - u.at, b = w.end - u.at;
    const int ka = a <= p.unit_cost + u.cost ? 1 : (a - p.unit_cost + u.cost - 1) / u.cost;
    const int kb = b <= p.unit_cost + u.cost ? 1 : (b - p.unit_cost + u.cost - 1) / u.cost;
    k0 = a <= 0 ? 0 : ka;
    k1 = kb < u.tiles ? kb : u.tiles;
    w.x = u.at + ex_length(p, u.kind, u.tiles);
    if (k0 < k1) return true;
  }
  return false;
}
// Row r of a unit: entry, query of the entry and query head; entry < 0 for padding.
struct ExtendRow { int entry, query, head; };
__host__ __device__ inline ExtendRow ex_row(const ExtendParams& p, const ExtendUnit& u, int r) {
  ExtendRow x;
  const int j = u.block * p.QB + r / p.G;
  x.head = u.head * p.G + r % p.G;
  x.entry = -1;
  x.query = 0;
  if (r / p.G >= p.QB) return x;
  if (u.kind != EX_SHARED) {
    if (j < p.nq[u.index]) { x.entry = u.index; x.query = j; }
    return x;
  }
  if (j >= p.g_nq[u.index]) return x;
  int lo = p.g_first[u.index], hi = p.g_first[u.index + 1] - 1;   // the last member whose queries start at or before j
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.member0[p.order[mid]] <= j) lo = mid; else hi = mid - 1;
  }
  x.entry = p.order[lo];
  x.query = j - p.member0[x.entry];
  return x;
}
// Whether the unit's keys (values) are raw rows in the original basis.
__host__ __device__ inline bool ex_raw_k(const ExtendParams& p, const ExtendUnit& u) {
  return u.kind == EX_TAIL || p.heads[u.head].kcodec == KVQ_F16;
}
__host__ __device__ inline bool ex_raw_v(const ExtendParams& p, const ExtendUnit& u) {
  return u.kind == EX_TAIL || p.heads[u.head].vcodec == KVQ_F16;
}

// Position range of a unit: [begin, end).
__host__ __device__ inline void ex_range(const ExtendParams& p, const ExtendUnit& u, int* begin, int* end) {
  if (u.kind == EX_SHARED) { *begin = 0; *end = p.g_tok[u.index]; }
  else if (u.kind == EX_OWN) { *begin = p.own0[u.index]; *end = ex_paged(p, u.index); }
  else { *begin = ex_paged(p, u.index); *end = p.len[u.index]; }
}

// The axis of the launch x.chain for N rows a unit and these costs; false if it does not
// fit 31 bits.
inline bool ex_lay_out(ExtendParams& x, int N, int page_cost, int tail_cost, int unit_cost) {
  x.N = N;
  x.QB = N / x.G;
  x.page_cost = page_cost;
  x.tail_cost = tail_cost;
  x.unit_cost = unit_cost;
  int64_t at = 0, unit = 0;
  for (int g = 0; g < x.n_groups && at < INT32_MAX; ++g) {
    const int64_t units = x.chain == EX_ENTRIES ? 0 : (int64_t)x.Hkv * ex_blocks(x, x.g_nq[g]);
    x.s_at[g] = (int)at;
    x.s_unit[g] = (int)unit;
    at += units * ex_length(x, EX_SHARED, ex_unit_tiles(x, EX_SHARED, g));
    unit += units;
  }
  for (int e = 0; e < x.n_entries && at < INT32_MAX; ++e) {
    const int64_t units = x.chain == EX_GROUPS ? 0 : (int64_t)x.Hkv * ex_blocks(x, x.nq[e]);
    const int to = ex_unit_tiles(x, EX_OWN, e), tt = ex_unit_tiles(x, EX_TAIL, e);
    x.e_at[e] = (int)at;
    x.e_unit[e] = (int)unit;
    at += units * (ex_length(x, EX_OWN, to) + ex_length(x, EX_TAIL, tt));
    unit += units * ((to > 0) + (tt > 0));
  }
  x.s_at[x.n_groups] = x.e_at[0];
  x.e_at[x.n_entries] = (int)at;
  x.e_unit[x.n_entries] = (int)unit;
  x.total = (int)at;
  return at < INT32_MAX && unit < INT32_MAX;
}
// Cut the axis for `ctas` CTAs.  A tile per CTA while there are CTAs for all; else by cost:
// in page tiles (2.4 us with one of two CTAs an SM), a raw tail tile takes 2 and a unit's
// start and end 3 more: queries, the wait for the first tile, the partial result.  Without
// them the CTAs whose share is many short tails end last (64 sequences x 4 drafts: 356 us
// with tails at 1.5 and starts at 1.5, 325 us so; 16 x 8 drafts: 171, 142; tails of 1024
// tokens instead of 256: 443, 369).
inline bool ex_cut(ExtendParams& x, int N, int ctas) {
  if (!ex_lay_out(x, N, 1, 1, 0)) return false;
  if (x.total > ctas && !ex_lay_out(x, N, 1, 2, 3)) return false;
  x.per = std::max(std::max(x.page_cost, x.tail_cost) + x.unit_cost, (x.total + ctas - 1) / ctas);
  x.n_ctas = (x.total + x.per - 1) / x.per;
  return true;
}

inline size_t extend_slot_bytes(int N) { return (size_t)N * (D * sizeof(float) + sizeof(float2)); }

// CTAs per SM and stages of the attention kernel for page-heads of page_stage bytes;
// n_raw = 0: too few stages fit beside the operand images of N rows.
struct ExtendShape { int ctas_per_sm, n_raw; };
ExtendShape extend_mma_shape(int N, int page_stage);
cudaError_t launch_extend_mma(const ExtendParams& p, cudaStream_t s);
// groups: the parameters of the groups' launch, or null if there was one launch.
cudaError_t launch_extend_merge(const ExtendParams& p, const ExtendParams* groups, cudaStream_t s);

}  // namespace kvq
