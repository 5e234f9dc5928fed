// Host side of the sequence operations: fork, compact and truncate.  A page is held
// by one or more sequences (kvq_plan::refs); a sequence that writes into a page
// others hold gets its own copy first (kvq_append_quantize), and a compaction only
// ever writes fresh pages.
#include <exception>
#include <unordered_map>

#include "plan.h"

using namespace kvq;

namespace {

// every-layer launches use one grid row per (layer, kv head, K|V)
bool grid_fits(const kvq_plan* p) { return (int64_t)p->L * p->Hkv * 2 <= 65535; }

kvq_status check_sequences(const kvq_plan* p, int n, const int* ids) {
  if (n < 0 || n > MAX_BATCH) return fail(KVQ_ERR_INVALID_ARG, "the number of sequences must be in [0, %d]", MAX_BATCH);
  if (n > 0 && !ids) return fail(KVQ_ERR_INVALID_ARG, "null sequence ids");
  for (int i = 0; i < n; ++i) {
    if (ids[i] < 0 || ids[i] >= p->max_seqs) return fail(KVQ_ERR_INVALID_ARG, "sequence id %d out of range", ids[i]);
    for (int j = 0; j < i; ++j)
      if (ids[j] == ids[i]) return fail(KVQ_ERR_INVALID_ARG, "sequence id %d repeated", ids[i]);
  }
  return KVQ_OK;
}

// One page index of a compaction that needs a fresh page.
struct Task { int entry, index; };

}  // namespace

extern "C" {

kvq_status kvq_seq_fork(kvq_plan* p, int src, int n_dst, const int* dst_ids, void* stream) {
  if (!p) return fail(KVQ_ERR_INVALID_ARG, "null plan");
  if (const kvq_status st = require_plan_device(p); st != KVQ_OK) return st;
  if (!p->cache) return fail(KVQ_ERR_STATE, "no cache bound");
  if (!grid_fits(p)) return fail(KVQ_ERR_UNSUPPORTED, "more than 65535 (layer, kv head, K|V) rows");
  if (src < 0 || src >= p->max_seqs) return fail(KVQ_ERR_INVALID_ARG, "sequence id %d out of range", src);
  if (const kvq_status st = check_sequences(p, n_dst, dst_ids); st != KVQ_OK) return st;
  for (int i = 0; i < n_dst; ++i) {
    if (dst_ids[i] == src) return fail(KVQ_ERR_INVALID_ARG, "a sequence cannot be forked into itself");
    if (p->longest(dst_ids[i]) > 0 || p->npages[dst_ids[i]] > 0)
      return fail(KVQ_ERR_STATE, "sequence %d holds tokens: reset it before forking into it", dst_ids[i]);
  }
  if (n_dst == 0) return KVQ_OK;
  const int np = p->npages[src];
  const int ring = (int)std::min<int64_t>(p->T, p->longest(src));
  const cudaError_t e = launch_fork(p->page_params(), src, n_dst, dst_ids, np, ring, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "fork launch");
  const int* from = p->bt.data() + (size_t)src * p->mpps;
  for (int i = 0; i < n_dst; ++i) {
    const int d = dst_ids[i];
    std::copy(from, from + np, p->bt.begin() + (size_t)d * p->mpps);
    for (int j = 0; j < np; ++j) ++p->refs[from[j]];
    p->npages[d] = np;
    std::copy_n(p->len.begin() + (size_t)src * p->L, p->L, p->len.begin() + (size_t)d * p->L);
  }
  return KVQ_OK;
}

// Shared by compact (n_keep, keep) and truncate (n_keep null: no row behind `start`).
static kvq_status compact(kvq_plan* p, int n, const int* ids, const int64_t* start, const int* n_keep, const int* keep,
                          void* stream) {
  if (!p) return fail(KVQ_ERR_INVALID_ARG, "null plan");
  if (const kvq_status st = require_plan_device(p); st != KVQ_OK) return st;
  if (!p->cache) return fail(KVQ_ERR_STATE, "no cache bound");
  if (!grid_fits(p)) return fail(KVQ_ERR_UNSUPPORTED, "more than 65535 (layer, kv head, K|V) rows");
  if (const kvq_status st = check_sequences(p, n, ids); st != KVQ_OK) return st;
  if (n == 0) return KVQ_OK;
  if (!start) return fail(KVQ_ERR_INVALID_ARG, "null lengths");
  if (p->T > compact_max_tail())
    return fail(KVQ_ERR_UNSUPPORTED, "tails above %d tokens cannot be moved", compact_max_tail());
  std::vector<CompactSeq> q(n);
  std::vector<Task> tasks;
  int64_t kept = 0;
  for (int i = 0; i < n; ++i) {
    const int64_t len = p->length(ids[i], 0);
    for (int l = 1; l < p->L; ++l)
      if (p->length(ids[i], l) != len)
        return fail(KVQ_ERR_STATE, "sequence %d has %lld tokens in layer 0 and %lld in layer %d", ids[i],
                    (long long)len, (long long)p->length(ids[i], l), l);
    const int k = n_keep ? n_keep[i] : 0;
    if (start[i] < 0 || k < 0 || start[i] > len || k > len - start[i])
      return fail(KVQ_ERR_INVALID_ARG, "sequence %d: %lld + %d tokens of %lld cannot be kept", ids[i],
                  (long long)start[i], k, (long long)len);
    q[i] = CompactSeq{ids[i], (int)len, (int)start[i], k, kept};
    kept += k;
    if (k > 0 && p->quantized_rows(start[i] + k) > start[i])   // pages that hold a row at or behind `start`
      for (int j = (int)(start[i] / PAGE); j < p->pages_for(start[i] + k); ++j) tasks.push_back(Task{i, j});
  }
  if (kept > 0 && !keep) return fail(KVQ_ERR_INVALID_ARG, "null keep list");
  if ((uintptr_t)keep % 4) return fail(KVQ_ERR_INVALID_ARG, "the keep list must be 4-byte aligned");
  // The fresh pages: a launch takes as many as are free, and the pages it replaced
  // (those no other sequence holds) serve the next one.
  if ((int64_t)p->free_pages.size() < (int64_t)tasks.size()) {
    int64_t have = (int64_t)p->free_pages.size(), back = 0;
    std::unordered_map<int, int> left;
    for (const Task& t : tasks) {
      if (have == 0) { have = back; back = 0; }
      if (have == 0) return fail(KVQ_ERR_CAPACITY, "no free page to compact into");
      --have;
      const int pid = p->bt[(size_t)q[t.entry].seq * p->mpps + t.index];
      if (p->refs[pid] == ++left[pid]) ++back;
    }
  }
  const cudaStream_t st = (cudaStream_t)stream;
  const PageParams g = p->page_params();
  for (int i0 = 0; i0 < n; i0 += MAX_COMPACT_SEQS) {
    CompactSeqs cs;
    cs.keep = keep;
    cs.n = std::min(MAX_COMPACT_SEQS, n - i0);
    std::copy(q.begin() + i0, q.begin() + i0 + cs.n, cs.s);
    cudaError_t e = launch_compact_tail(g, cs, st);
    if (e != cudaSuccess) return cuda_fail(e, "tail launch");
    size_t t0 = 0;
    while (t0 < tasks.size() && tasks[t0].entry < i0) ++t0;
    while (t0 < tasks.size() && tasks[t0].entry < i0 + cs.n) {
      CompactPages d;
      d.n = 0;
      size_t t = t0;
      while (t < tasks.size() && tasks[t].entry < i0 + cs.n && d.n < MAX_COMPACT_PAGES && !p->free_pages.empty()) {
        d.entry[d.n] = (uint8_t)(tasks[t].entry - i0);
        d.index[d.n] = tasks[t].index;
        d.page[d.n] = p->take_page();
        ++d.n;
        ++t;
      }
      if (d.n == 0) return fail(KVQ_ERR_CAPACITY, "no free page to compact into");
      e = launch_compact_pages(g, cs, d, st);
      if (e != cudaSuccess) return cuda_fail(e, "page gather launch");
      for (int k = 0; k < d.n; ++k) {
        int& slot = p->bt[(size_t)cs.s[d.entry[k]].seq * p->mpps + d.index[k]];
        p->drop_page(slot);
        slot = d.page[k];
      }
      t0 = t;
    }
  }
  for (const CompactSeq& s : q) {
    const int64_t m = (int64_t)s.start + s.n_keep;
    const int pages = p->pages_for(m);
    while (p->npages[s.seq] > pages) {
      int& slot = p->bt[(size_t)s.seq * p->mpps + --p->npages[s.seq]];
      p->drop_page(slot);
      slot = -1;
    }
    for (int l = 0; l < p->L; ++l) p->len[(size_t)s.seq * p->L + l] = m;
  }
  return KVQ_OK;
}

kvq_status kvq_seq_load(kvq_plan* p, int layer, int seq_id, int64_t n_rows, const void* k_codes, const void* k_scales,
                        const void* v_codes, const void* v_scales, int64_t n_tail, const void* k_tail,
                        const void* v_tail, void* stream) try {
  if (!p) return fail(KVQ_ERR_INVALID_ARG, "null plan");
  if (const kvq_status st = require_plan_device(p); st != KVQ_OK) return st;
  if (!p->cache) return fail(KVQ_ERR_STATE, "no cache bound");
  if (layer < 0 || layer >= p->L) return fail(KVQ_ERR_INVALID_ARG, "layer %d out of range", layer);
  if (seq_id < 0 || seq_id >= p->max_seqs) return fail(KVQ_ERR_INVALID_ARG, "sequence id %d out of range", seq_id);
  if (p->length(seq_id, layer) != 0)
    return fail(KVQ_ERR_STATE, "sequence %d holds tokens in layer %d: reset it before loading", seq_id, layer);
  if (n_rows < 0 || n_tail < 0 || n_tail > p->T || (n_rows > 0 && n_tail != p->T))
    return fail(KVQ_ERR_INVALID_ARG, "%lld packed and %lld tail rows: with a tail of %d the tail must be full before "
                "rows are packed", (long long)n_rows, (long long)n_tail, p->T);
  if (n_rows > p->max_tokens - n_tail) return fail(KVQ_ERR_CAPACITY, "sequence %d would exceed max_tokens_per_seq", seq_id);
  bool scales = false;                                   // F16 rows have none
  for (int h = 0; h < p->Hkv; ++h) scales |= p->head(layer, h).sbK || p->head(layer, h).sbV;
  if (n_rows > 0 && (!k_codes || !v_codes || (scales && (!k_scales || !v_scales))))
    return fail(KVQ_ERR_INVALID_ARG, "null codes or scales");
  if (n_tail > 0 && (!k_tail || !v_tail)) return fail(KVQ_ERR_INVALID_ARG, "null tail rows");
  for (const void* a : {k_codes, k_scales, v_codes, v_scales, k_tail, v_tail})
    if ((uintptr_t)a % 16) return fail(KVQ_ERR_INVALID_ARG, "the rows must be 16-byte aligned");
  const int n = (int)(n_rows + n_tail);
  if (n == 0) return KVQ_OK;
  if (const kvq_status st = prepare_pages(p, layer, 1, &seq_id, &n, stream); st != KVQ_OK) return st;
  LoadParams q;
  q.g = p->page_params();
  q.layer = layer;
  q.seq = seq_id;
  q.n_rows = (int)n_rows;
  q.n_tail = (int)n_tail;
  q.codes[0] = (const uint8_t*)k_codes;
  q.codes[1] = (const uint8_t*)v_codes;
  q.scales[0] = (const uint8_t*)k_scales;
  q.scales[1] = (const uint8_t*)v_scales;
  q.tail[0] = (const uint8_t*)k_tail;
  q.tail[1] = (const uint8_t*)v_tail;
  const cudaError_t e = launch_load(q, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "load launch");
  p->len[(size_t)seq_id * p->L + layer] = n;
  return KVQ_OK;
} catch (const std::exception&) {
  return fail(KVQ_ERR_OOM, "host allocation failed");
}

kvq_status kvq_seq_compact(kvq_plan* p, int n_seqs, const int* seq_ids, const int64_t* start, const int* n_keep,
                           const int* keep, void* stream) try {
  if (n_seqs > 0 && !n_keep) return fail(KVQ_ERR_INVALID_ARG, "null n_keep");
  return compact(p, n_seqs, seq_ids, start, n_keep, keep, stream);
} catch (const std::exception&) {
  return fail(KVQ_ERR_OOM, "host allocation failed");
}

kvq_status kvq_seq_truncate(kvq_plan* p, int n_seqs, const int* seq_ids, const int64_t* new_len, void* stream) try {
  return compact(p, n_seqs, seq_ids, new_len, nullptr, nullptr, stream);
} catch (const std::exception&) {
  return fail(KVQ_ERR_OOM, "host allocation failed");
}

}  // extern "C"
