// Host side of kvq_extend_attention: validation, which sequences share pages, and the
// work lists of the launches.
#include <exception>
#include <utility>

#include "extend.h"
#include "plan.h"

using namespace kvq;

namespace {

constexpr int CTAS_PER_SM = 2;
// Positions a group must share before its pages are walked once for the group.  A unit of
// all members' queries is wider, and in one launch so are then the members' own (16 forks of
// 1344 shared positions: 63 us apart, 71 together; of 2304: 75, 73; of 7936: 107, 76; 64
// forks of 768: 147, 166; of 1344: 168, 147).
constexpr int MIN_SHARED = 12 * EX_TILE;

size_t extend_workspace(const kvq_plan* p, int n, int64_t total_q) {
  // one launch of every unit, or two: the groups' with the widest units and the entries'
  size_t most = 0, groups = 0;
  for (int N = 16; N <= EX_MAX_ROWS; N *= 2) {
    const int64_t qb = N / p->G, blocks = total_q / qb, ctas = (int64_t)p->num_sms * CTAS_PER_SM;
    const int64_t own = p->Hkv * 2 * (n + blocks), shared = p->Hkv * (n / 2 + blocks);
    most = std::max(most, (size_t)(own + ctas) * extend_slot_bytes(N));
    groups = std::max(groups, (size_t)(shared + ctas) * extend_slot_bytes(N));
  }
  return most + groups;
}

// Rows of a unit, at most 64.  A unit costs the same page loads and unpacking whatever its
// rows, so the fewest that hold every group's and every sequence's queries are best where
// CTAs have many tiles (16 sequences x 16 drafts x 4 heads: 64 rows 190 us, 32: 245, 16: 322; x 8 drafts: 32 rows 144 us, 16: 179).  A tile
// and a unit's start take longer with more rows, so fewer are taken where every CTA then has
// one tile at most (one sequence of 1024 tokens x 16 drafts: 19 us with 16, 22 with 64) and
// 32 instead of 64 where a CTA has less than 4 tiles (4096 tokens: 27 us, 35; 16384: 46, 42).
int rows_for(const kvq_plan* p, int widest, int stage) {
  int most = widest <= 16 / p->G ? 16 : widest <= 32 / p->G ? 32 : 64;
  while (most > 16 && extend_mma_shape(most, stage).n_raw == 0) most /= 2;   // F16 page-heads (32 KiB) leave no room for 64
  return most;
}
int unit_rows(const kvq_plan* p, ExtendParams& x, int widest) {
  const int stage = x.page_stage, most = rows_for(p, widest, stage);
  for (int N = 16; N < most; N *= 2)
    if (ex_lay_out(x, N, 1, 1, 0) && x.total <= p->num_sms * extend_mma_shape(N, stage).ctas_per_sm) return N;
  if (most == 64 && ex_lay_out(x, 64, 1, 1, 0) && x.total > p->num_sms && x.total < 4 * p->num_sms) return 32;
  return most;
}

// The work list of one launch, its partial results behind *used bytes of the workspace.
kvq_status place(const kvq_plan* p, ExtendParams& x, int widest, void* workspace, size_t* used) {
  const int N = unit_rows(p, x, widest);
  const ExtendShape shape = extend_mma_shape(N, x.page_stage);
  if (shape.n_raw == 0) return fail(KVQ_ERR_UNSUPPORTED, "page-heads of %d bytes do not fit the kernel's stages", x.page_stage);
  x.n_raw = shape.n_raw;
  x.ctas_per_sm = shape.ctas_per_sm;
  if (!ex_cut(x, N, p->num_sms * shape.ctas_per_sm)) return fail(KVQ_ERR_UNSUPPORTED, "the call has more than 2^31 tiles of work");
  const size_t slots = (size_t)x.n_ctas + x.e_unit[x.n_entries];
  x.part_o = (float*)((uint8_t*)workspace + *used);
  x.part_ml = (float2*)(x.part_o + slots * N * D);
  *used += slots * extend_slot_bytes(N);
  return KVQ_OK;
}

// Groups of entries whose sequences begin with the same pages, and how many positions
// they share: whole pages, all of them before every member's last n_q tokens.
void find_groups(const kvq_plan* p, ExtendParams& x) {
  x.n_groups = 0;
  x.g_first[0] = 0;
  std::vector<std::pair<int, int>> first;               // (first page, entry)
  for (int e = 0; e < x.n_entries; ++e) {
    x.own0[e] = 0;
    x.member0[e] = 0;
    x.group[e] = -1;
    const int whole = std::min(ex_paged(x, e), x.len[e] - x.nq[e]) / PAGE;
    if (x.nq[e] > 0 && whole * PAGE >= MIN_SHARED)
      first.emplace_back(p->bt[(size_t)x.seq[e] * p->mpps], e);
  }
  std::sort(first.begin(), first.end());
  int n_order = 0;
  for (size_t a = 0; a < first.size();) {
    size_t b = a + 1;
    while (b < first.size() && first[b].first == first[a].first) ++b;
    if (b - a > 1) {
      const int* lead = p->bt.data() + (size_t)x.seq[first[a].second] * p->mpps;
      int same = INT32_MAX;
      for (size_t k = a; k < b; ++k) {
        const int e = first[k].second;
        const int* mine = p->bt.data() + (size_t)x.seq[e] * p->mpps;
        const int whole = std::min(same, std::min(ex_paged(x, e), x.len[e] - x.nq[e]) / PAGE);
        same = (int)(std::mismatch(mine, mine + whole, lead).first - mine);
      }
      if (same * PAGE >= MIN_SHARED) {
        const int g = x.n_groups++;
        x.g_tok[g] = same * PAGE;
        x.g_nq[g] = 0;
        for (size_t k = a; k < b; ++k) {
          const int e = first[k].second;
          x.group[e] = (int16_t)g;
          x.own0[e] = same * PAGE;
          x.member0[e] = x.g_nq[g];
          x.g_nq[g] += x.nq[e];
          x.order[n_order++] = (uint8_t)e;
        }
        x.g_first[g + 1] = n_order;
      }
    }
    a = b;
  }
}

kvq_status extend(kvq_plan* p, int layer, int n, const int* seq_ids, const int* n_q, const uint64_t* mask, const void* q,
                  void* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (!p) return fail(KVQ_ERR_INVALID_ARG, "null plan");
  if (const kvq_status st = require_plan_device(p); st != KVQ_OK) return st;
  if (!p->cache) return fail(KVQ_ERR_STATE, "no cache bound");
  if (layer < 0 || layer >= p->L) return fail(KVQ_ERR_INVALID_ARG, "layer %d out of range", layer);
  if (n < 0 || n > MAX_BATCH) return fail(KVQ_ERR_INVALID_ARG, "n_seqs must be in [0, %d]", MAX_BATCH);
  if (n > 0 && (!seq_ids || !n_q)) return fail(KVQ_ERR_INVALID_ARG, "null seq_ids or n_q");
  ExtendParams x;
  int64_t total = 0;
  for (int e = 0; e < n; ++e) {
    const int s = seq_ids[e];
    if (s < 0 || s >= p->max_seqs) return fail(KVQ_ERR_INVALID_ARG, "sequence id %d out of range", s);
    const int64_t len = p->length(s, layer);
    if (n_q[e] < 0 || n_q[e] > len) return fail(KVQ_ERR_INVALID_ARG, "n_q %d outside [0, %lld]", n_q[e], (long long)len);
    if (mask && n_q[e] > KVQ_MAX_MASKED)
      return fail(KVQ_ERR_UNSUPPORTED, "masks cover at most %d tokens (got %d)", KVQ_MAX_MASKED, n_q[e]);
    x.seq[e] = s;
    x.len[e] = (int)len;
    x.nq[e] = n_q[e];
    x.q0[e] = (int)total;
    total += n_q[e];
  }
  if (total == 0) return KVQ_OK;
  if (total * p->Hq > INT32_MAX) return fail(KVQ_ERR_UNSUPPORTED, "too many queries (%lld)", (long long)total);
  if (!q || !out) return fail(KVQ_ERR_INVALID_ARG, "null q or out");
  if (((uintptr_t)q % 16) || ((uintptr_t)out % 16)) return fail(KVQ_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if ((uintptr_t)mask % 8) return fail(KVQ_ERR_INVALID_ARG, "the masks must be 8-byte aligned");
  const DecodeParams d = p->base_params(layer);
  x.pool = d.pool;
  x.page_bytes = d.page_bytes;
  x.table = d.block_table;
  x.mpps = d.max_pages_per_seq;
  x.tail = d.tail;
  x.T = d.T; x.L = d.L; x.layer = layer; x.Hkv = d.Hkv; x.Hq = d.Hq; x.G = d.G;
  x.rot = d.rot;
  x.bf16 = d.bf16;
  x.q = (const __half*)q;
  x.out = (__half*)out;
  x.mask = (const unsigned long long*)mask;
  x.s_k = d.s_k;
  x.s_v = d.s_v;
  x.M = d.M;
  x.qscale = d.qscale;
  x.err = d.err;
  x.wait_ns = d.wait_ns;
  x.drop_last_tile = d.drop_last_tile;
  x.n_entries = n;
  x.q0[n] = (int)total;
  x.total_q = (int)total;
  std::copy(d.heads, d.heads + MAX_HKV, x.heads);
  find_groups(p, x);
  int stage = 0, widest = 0, widest_group = 0;
  for (int h = 0; h < p->Hkv; ++h) stage = std::max(stage, (int)x.heads[h].bytes);
  for (int e = 0; e < n; ++e) widest = std::max(widest, x.nq[e]);
  for (int g = 0; g < x.n_groups; ++g) widest_group = std::max(widest_group, x.g_nq[g]);
  stage = (stage + 127) & ~127;
  // Groups whose queries fill units of 64 rows get a launch of their own where their members'
  // own need fewer and the groups have a tile for every SM (64 forks of 1800: 122 us, 161 in
  // one launch; of 32768: 238, 272; 16 of 4096: 57, 61; of 32768: 87, 94; with fewer tiles, 16 of
  // 1800: 58, 53; with 32 rows, 8 of 8192: 50, 45).
  x.page_stage = stage;
  x.chain = EX_GROUPS;
  const bool two = rows_for(p, widest_group, stage) == 64 && rows_for(p, widest, stage) < 64 &&
                   ex_lay_out(x, 64, 1, 1, 0) && x.total >= p->num_sms;
  x.chain = EX_ALONE;
  ExtendParams groups;
  size_t used = 0;
  if (two) {
    groups = x;
    groups.chain = EX_GROUPS;
    x.chain = EX_ENTRIES;
    if (const kvq_status st = place(p, groups, widest_group, workspace, &used); st != KVQ_OK) return st;
  }
  if (const kvq_status st = place(p, x, two ? widest : std::max(widest, widest_group), workspace, &used); st != KVQ_OK) return st;
  if (!workspace || workspace_bytes < used)
    return fail(KVQ_ERR_INVALID_ARG, "workspace of %zu bytes needed (got %zu)", used, workspace_bytes);
  if ((uintptr_t)workspace % 16) return fail(KVQ_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  cudaError_t e = two ? launch_extend_mma(groups, (cudaStream_t)stream) : cudaSuccess;
  if (e == cudaSuccess) e = launch_extend_mma(x, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "extend launch");
  e = launch_extend_merge(x, two ? &groups : nullptr, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "extend merge launch");
  return KVQ_OK;
}

}  // namespace

extern "C" {

kvq_status kvq_plan_extend_workspace_bytes(const kvq_plan* p, int n_seqs, int64_t total_q, size_t* bytes) {
  if (!p || !bytes) return fail(KVQ_ERR_INVALID_ARG, "null argument");
  if (n_seqs < 0 || n_seqs > MAX_BATCH) return fail(KVQ_ERR_INVALID_ARG, "n_seqs must be in [0, %d]", MAX_BATCH);
  if (total_q < 0 || total_q > INT32_MAX / p->Hq) return fail(KVQ_ERR_INVALID_ARG, "total_q out of range");
  *bytes = extend_workspace(p, n_seqs, total_q);
  return KVQ_OK;
}

kvq_status kvq_extend_attention(kvq_plan* p, int layer, int n_seqs, const int* seq_ids, const int* n_q,
                                const uint64_t* tree_mask, const void* q, void* out, void* workspace,
                                size_t workspace_bytes, void* stream) try {
  return extend(p, layer, n_seqs, seq_ids, n_q, tree_mask, q, out, workspace, workspace_bytes, stream);
} catch (const std::exception&) {
  return fail(KVQ_ERR_OOM, "host allocation failed");
}

}  // extern "C"
