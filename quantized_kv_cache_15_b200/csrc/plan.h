// The plan and the host helpers that the entry points share (not part of the
// public ABI).
#pragma once

#include <algorithm>
#include <cstring>
#include <vector>

#include "kvq_internal.h"
#include "pages.h"

namespace kvq {
// Record a failure for kvq_last_error() and return its status.
kvq_status fail(kvq_status st, const char* fmt, ...);
kvq_status cuda_fail(cudaError_t e, const char* what);
// Kernels are launched on the current device and read the plan's memory, so a call
// that enqueues work needs the plan's device current: on another device (through
// the legacy stream, say) they would reach that memory only by peer access, which
// this library never enables.  Checked before anything is enqueued.
kvq_status require_plan_device(const kvq_plan* p);
// Give every sequence the pages that n_new[i] more tokens of one layer need: new ones,
// and its own copy of a page it writes into that another sequence holds too.
// KVQ_ERR_CAPACITY before anything changes if the pool has too few.
kvq_status prepare_pages(kvq_plan* p, int layer, int n_seqs, const int* seq_ids, const int* n_new, void* stream);
}  // namespace kvq

using namespace kvq;

struct kvq_plan {
  int device = 0;
  int num_sms = 148;
  int L = 0, Hq = 0, Hkv = 0, G = 0, T = 0, max_seqs = 0;
  int64_t max_tokens = 0;
  int mpps = 0;            // max pages per sequence
  int64_t n_pages = 0;
  int rot = 0;
  bool bf16 = false;             // raw rows are bf16
  float scale = 0.f;
  std::vector<HeadInfo> heads;        // [L][Hkv]
  std::vector<uint64_t> layer_off;    // [L]
  std::vector<uint32_t> page_bytes;   // [L]
  std::vector<int> stage_bytes;       // [L] max region (and tail page) bytes
  uint64_t tail_off = 0, cache_bytes = 0;
  uint8_t* cache = nullptr;
  float* d_inv = nullptr;   // [L][Hkv][2][128] inverse RMS (append)
  float* d_sk = nullptr;    // [L][Hkv][128] 1/inv_rms of K (decode, dequantize)
  float* d_sv = nullptr;    // [L][Hkv][128] 1/inv_rms of V
  float* d_M = nullptr;     // fused projections M_h, fp32 [r][128] per head
  double* d_MT = nullptr;   // their transposes, widened to double [128][r] per head (append projection)
  int* d_bt = nullptr;      // block table [max_seqs][mpps]
  HeadInfo* d_heads = nullptr;        // [L][Hkv], the device copy of `heads` (every-layer kernels)
  LayerInfo* d_layers = nullptr;      // [L] pool offsets and page sizes
  int* d_err = nullptr;
  std::vector<int64_t> len;           // [max_seqs][L]
  std::vector<int> bt;                // host mirror of the block table
  std::vector<int> npages;            // pages held per sequence
  std::vector<int> free_pages;        // stack of free page ids
  std::vector<int> refs;              // [n_pages] sequences that hold the page (0: free)
  // test-only settings (kvq_debug_set_decode_split, kvq_debug_fault_injection)
  int debug_pps = 0;                          // fixed pages per split, 0 = chosen per call
  unsigned long long wait_ns = 2000000000ull; // give-up time of the kernels' bounded waits
  int drop_last_tile = 0;                     // decode producers skip their last tile
  int prefill_path = 0;                       // 0: tensor cores where the layer allows, 1: decode kernel

  ~kvq_plan() {
    int prev = 0;
    cudaGetDevice(&prev);
    cudaSetDevice(device);
    cudaFree(d_inv); cudaFree(d_sk); cudaFree(d_sv); cudaFree(d_M); cudaFree(d_MT); cudaFree(d_bt); cudaFree(d_err);
    cudaFree(d_heads); cudaFree(d_layers);
    cudaSetDevice(prev);
  }

  const HeadInfo& head(int l, int h) const { return heads[(size_t)l * Hkv + h]; }

  void reset_all() {
    std::fill(len.begin(), len.end(), 0);
    std::fill(bt.begin(), bt.end(), -1);
    std::fill(npages.begin(), npages.end(), 0);
    free_pages.clear();
    refs.assign((size_t)n_pages, 0);
    for (int64_t i = n_pages - 1; i >= 0; --i) free_pages.push_back((int)i);
  }

  // Pages.  take_page needs a free page; drop_page gives one holder's claim back
  // and returns the page to the pool when nobody holds it any more.
  int take_page() {
    const int pid = free_pages.back();
    free_pages.pop_back();
    refs[pid] = 1;
    return pid;
  }
  void drop_page(int pid) {
    if (--refs[pid] == 0) free_pages.push_back(pid);
  }
  int64_t length(int seq, int layer) const { return len[(size_t)seq * L + layer]; }
  int64_t longest(int seq) const {
    int64_t n = 0;
    for (int l = 0; l < L; ++l) n = std::max(n, length(seq, l));
    return n;
  }
  // rows of a sequence of n tokens that sit in pages, and the pages they take
  int64_t quantized_rows(int64_t n) const { return n > T ? n - T : 0; }
  int pages_for(int64_t n) const { return (int)((quantized_rows(n) + PAGE - 1) / PAGE); }
  PageParams page_params() const {
    PageParams g;
    g.cache = cache;
    g.layers = d_layers;
    g.heads = d_heads;
    g.table = d_bt;
    g.tail = cache + tail_off;
    g.mpps = mpps;
    g.T = T; g.L = L; g.Hkv = Hkv;
    g.rot = rot;
    g.bf16 = bf16;
    g.s_k = rot == KVQ_ROT_VARNORM_HADAMARD ? d_sk : nullptr;
    g.s_v = rot == KVQ_ROT_VARNORM_HADAMARD ? d_sv : nullptr;
    g.M = d_M;
    g.err = d_err;
    return g;
  }

  DecodeParams base_params(int layer) const {
    DecodeParams p;
    std::memset(&p, 0, sizeof(p));
    p.pool = cache + layer_off[layer];
    p.page_bytes = page_bytes[layer];
    p.block_table = d_bt;
    p.max_pages_per_seq = mpps;
    p.tail = cache + tail_off;
    p.T = T; p.L = L; p.layer = layer; p.Hkv = Hkv; p.Hq = Hq; p.G = G;
    p.rot = rot;
    p.bf16 = bf16;
    p.s_k = (rot == KVQ_ROT_VARNORM_HADAMARD) ? d_sk + (size_t)layer * Hkv * D : nullptr;
    p.s_v = (rot == KVQ_ROT_VARNORM_HADAMARD) ? d_sv + (size_t)layer * Hkv * D : nullptr;
    p.M = d_M;
    p.qscale = scale * 1.4426950408889634f;
    p.err = d_err;
    p.wait_ns = wait_ns;
    p.drop_last_tile = drop_last_tile;
    for (int h = 0; h < Hkv; ++h) p.heads[h] = head(layer, h);
    return p;
  }
};

