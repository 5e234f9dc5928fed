// Page operations over every layer of a plan's cache (pages.cu): copying pages
// before a shared one is written, forking a sequence, and compacting one to a
// list of kept positions.
#pragma once

#include "kvq_internal.h"

namespace kvq {

struct LayerInfo {               // one layer's page pool
  uint64_t off;                  // bytes from the cache's start
  uint32_t page_bytes;
  uint32_t pad;
};

struct PageParams {
  uint8_t* cache;
  const LayerInfo* layers;       // device [L]
  const HeadInfo* heads;         // device [L][Hkv]
  int* table;                    // block table [max_seqs][mpps]
  uint8_t* tail;                 // tail rings of every sequence and layer
  int mpps;
  int T, L, Hkv;
  int rot;
  int bf16;
  const float* s_k;              // [L][Hkv][128] or null
  const float* s_v;
  const float* M;
  int* err;
};

// One sequence of a compaction: positions below `start` stay where they are, then
// come the positions keep[keep0 .. keep0 + n_keep), ascending, each below `len`.
struct CompactSeq {
  int seq;
  int len;                       // tokens before the call
  int start;
  int n_keep;
  int64_t keep0;
};
constexpr int MAX_COMPACT_SEQS = 64;
constexpr int MAX_COMPACT_PAGES = 2048;   // destination pages per launch
struct CompactSeqs {
  const int* keep;
  int n;
  CompactSeq s[MAX_COMPACT_SEQS];
};
struct CompactPages {
  int n;
  uint8_t entry[MAX_COMPACT_PAGES];       // the page's sequence (index into CompactSeqs)
  int index[MAX_COMPACT_PAGES];           // its page index in the sequence
  int page[MAX_COMPACT_PAGES];            // the free page that takes the rows
};

// Copy n pages (src[i] -> dst[i]) in every layer.
cudaError_t launch_copy_pages(const PageParams& g, int n, const int* src, const int* dst, cudaStream_t s);
// The descriptors of one layer after a regrade.
cudaError_t launch_layer_tables(HeadInfo* heads, LayerInfo* layer, const HeadInfo* h, int n_heads, LayerInfo li,
                                cudaStream_t s);
// Sequences dst[0..n) get src's first n_pages block-table entries and the used part
// of its tail rings (ring_tokens of every ring).
cudaError_t launch_fork(const PageParams& g, int src, int n, const int* dst, int n_pages, int ring_tokens,
                        cudaStream_t s);
// Bring the tail rings of the sequences to their new lengths: ring rows that are
// kept move to their new slots (only where some sequence keeps rows behind its
// start), then rows that were below the tail come back from their pages.
cudaError_t launch_compact_tail(const PageParams& g, const CompactSeqs& q, cudaStream_t s);
// Gather kept rows into the fresh pages of `d`, then enter those in the block table.
cudaError_t launch_compact_pages(const PageParams& g, const CompactSeqs& q, const CompactPages& d, cudaStream_t s);
// Canonical packed rows and raw tail rows of one (sequence, layer) into its pages and
// ring; the sequence's pages are in the block table.
struct LoadParams {
  PageParams g;
  int layer, seq;
  int n_rows, n_tail;
  const uint8_t* codes[2];       // K, V: head after head, rows of the head's code bytes
  const uint8_t* scales[2];
  const uint8_t* tail[2];        // [n_tail][Hkv][128] raw 16-bit
};
cudaError_t launch_load(const LoadParams& p, cudaStream_t s);
// Longest tail (tokens) launch_compact_tail can take.
int compact_max_tail();

}  // namespace kvq
