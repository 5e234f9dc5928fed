// Attention of the last n_q tokens of several sequences in one launch
// (kvq_extend_attention): the work list, its kernels and the merge of their partial
// results.
//
// Three kinds of token ranges are walked in tiles of 128 positions: the pages that a
// group of sequences shares (every query of the group sees all of them), a sequence's
// own pages behind those, and its raw tail.  A unit is one range, one kv head and one
// block of `QB` queries (QB * G rows of at most `N`).  All tiles of all units form one
// axis, units in order; CTA c takes the tiles [c per, (c + 1) per), so every CTA has
// the same number of tiles whatever the lengths.  Where a CTA's run and a unit meet it
// writes one partial result (running maximum, sum, unnormalised output); walking the
// axis, either the CTA or the unit steps on from one partial to the next, so partial
// (c, u) has slot c + u to itself and no counter is needed.
#pragma once

#include "kvq_internal.h"

namespace kvq {

constexpr int EX_TILE = 128;
constexpr int EX_MAX_ROWS = 64;
constexpr int EX_SHARED = 0, EX_OWN = 1, EX_TAIL = 2;

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
  float* part_o;                 // [slots][N][128]
  float2* part_ml;               // [slots][N]: running maximum (log2 units), sum
  int N, QB;                     // rows of a unit, queries of a block
  int n_entries, n_groups, total_q;
  int total_tiles, per, n_ctas;
  int stage_bytes, n_raw;        // tensor-core kernel: page stages
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
  // prefix sums along the tile axis and of the units, shared | own | tail
  int s_tile[MAX_BATCH / 2 + 1], s_unit[MAX_BATCH / 2 + 1];
  int o_tile[MAX_BATCH + 1], o_unit[MAX_BATCH + 1];
  int t_tile[MAX_BATCH + 1], t_unit[MAX_BATCH + 1];
};

__host__ __device__ inline int ex_tiles(int tokens) { return (tokens + EX_TILE - 1) / EX_TILE; }
__host__ __device__ inline int ex_paged(const ExtendParams& p, int e) { return p.len[e] > p.T ? p.len[e] - p.T : 0; }

// A unit and the tiles of it.
struct ExtendUnit {
  int kind, index, head, block;  // index: the group (EX_SHARED) or the entry
  int unit;                      // ordinal of the unit on the axis
  int first, tiles;              // its tiles on the axis
};
__host__ __device__ inline ExtendUnit ex_unit(const ExtendParams& p, int kind, int index, int head, int block) {
  ExtendUnit u;
  u.kind = kind;
  u.index = index;
  u.head = head;
  u.block = block;
  int nb, tile0, unit0;
  if (kind == EX_SHARED) {
    nb = (p.g_nq[index] + p.QB - 1) / p.QB;
    u.tiles = ex_tiles(p.g_tok[index]);
    tile0 = p.s_tile[index];
    unit0 = p.s_unit[index];
  } else {
    nb = (p.nq[index] + p.QB - 1) / p.QB;
    u.tiles = kind == EX_OWN ? ex_tiles(ex_paged(p, index) - p.own0[index]) : ex_tiles(p.len[index] - ex_paged(p, index));
    tile0 = kind == EX_OWN ? p.o_tile[index] : p.t_tile[index];
    unit0 = kind == EX_OWN ? p.o_unit[index] : p.t_unit[index];
  }
  u.unit = unit0 + head * nb + block;
  u.first = tile0 + (head * nb + block) * u.tiles;
  return u;
}
// The unit that tile t of the axis belongs to.
__host__ __device__ inline ExtendUnit ex_find(const ExtendParams& p, int t) {
  int kind, index, tile0, nb, tiles;
  if (t < p.o_tile[0]) {
    kind = EX_SHARED;
    index = prefix_find(p.s_tile, p.n_groups, t);
    tile0 = p.s_tile[index];
    tiles = ex_tiles(p.g_tok[index]);
    nb = (p.g_nq[index] + p.QB - 1) / p.QB;
  } else {
    kind = t < p.t_tile[0] ? EX_OWN : EX_TAIL;
    const int* pre = kind == EX_OWN ? p.o_tile : p.t_tile;
    index = prefix_find(pre, p.n_entries, t);
    tile0 = pre[index];
    tiles = kind == EX_OWN ? ex_tiles(ex_paged(p, index) - p.own0[index]) : ex_tiles(p.len[index] - ex_paged(p, index));
    nb = (p.nq[index] + p.QB - 1) / p.QB;
  }
  const int k = (t - tile0) / tiles;
  return ex_unit(p, kind, index, k / nb, k % nb);
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

inline size_t extend_slot_bytes(int N) { return (size_t)N * (D * sizeof(float) + sizeof(float2)); }

// CTAs per SM and page stages of the tensor-core kernel for page-heads of stage_bytes;
// n_raw < 2: it cannot take them.
struct ExtendShape { int ctas_per_sm, n_raw; };
ExtendShape extend_mma_shape(int N, int stage_bytes);
cudaError_t launch_extend_mma(const ExtendParams& p, cudaStream_t s);
cudaError_t launch_extend_simple(const ExtendParams& p, cudaStream_t s);
cudaError_t launch_extend_merge(const ExtendParams& p, cudaStream_t s);

}  // namespace kvq
