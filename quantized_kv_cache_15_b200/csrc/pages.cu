// Page operations: copy-on-write page copies, fork, compaction of a sequence to the
// positions it keeps (these in every layer), and loading saved rows.  Nothing is
// requantized, so a row that stays in the pages keeps its bytes.
//
// Compaction of one sequence (kvq_seq_compact): with old length n, tail T and kept
// positions p_0 < p_1 < ... < p_{m-1} (the first `start` of them are 0 .. start-1),
// row j of the result is old row p_j >= j.  Old rows below n - T sit in pages, the
// others raw in the tail ring; new rows below m - T belong in pages, the others in
// the ring.  A kept ring row has at most T - 1 kept rows behind it, so it stays in
// the ring; a kept page row stays in the pages or comes back to the ring, as its
// dequantized value in the original basis, rounded once to the raw type.
//   1. ring rows to their new slots (j mod T): a slot's old row can be needed by a
//      later one, so a CTA reads all T slots of some 16-byte columns into shared
//      memory before it writes any;
//   2. page rows that come back to the ring, one warp each;
//   3. page rows that stay, gathered into fresh pages: the old page at an index is
//      not read by rows of later pages (p_j >= j), so the host hands it out again
//      after the launch that replaced it.
// Every step is bound by memory: a moved row is read once and written once.
#include "pages.h"

#include "dequant_row.cuh"

namespace kvq {

namespace {

constexpr int COPY_MAX = 512;
struct PagePairs {
  int n;
  int src[COPY_MAX], dst[COPY_MAX];
};

// grid (pairs, layers): one page of one layer
__global__ void __launch_bounds__(256) copy_pages_kernel(const __grid_constant__ PageParams g,
                                                         const __grid_constant__ PagePairs q) {
  const LayerInfo li = g.layers[blockIdx.y];
  const uint4* src = reinterpret_cast<const uint4*>(g.cache + li.off + (size_t)q.src[blockIdx.x] * li.page_bytes);
  uint4* dst = reinterpret_cast<uint4*>(g.cache + li.off + (size_t)q.dst[blockIdx.x] * li.page_bytes);
  const int n = (int)(li.page_bytes / 16);             // page-head regions are multiples of 128 bytes
  for (int i0 = threadIdx.x; i0 < n; i0 += 4 * 256) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + 256 * k < n) v[k] = src[i0 + 256 * k];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + 256 * k < n) dst[i0 + 256 * k] = v[k];
  }
}

struct LayerTables {
  HeadInfo* heads;
  LayerInfo* layer;
  int n_heads;
  LayerInfo li;
  HeadInfo h[MAX_HKV];
};
__global__ void layer_tables_kernel(const __grid_constant__ LayerTables t) {
  if ((int)threadIdx.x < t.n_heads) t.heads[threadIdx.x] = t.h[threadIdx.x];
  if (threadIdx.x == 0) *t.layer = t.li;
}

struct ForkDst {
  int src, n, n_pages;
  int ring_vecs;                 // used 16-byte vectors of one (layer, head) ring
  int dst[MAX_BATCH];
};
// blockIdx.y = 0: the block-table entries; blockIdx.y - 1 < L * Hkv: that ring's used
// part, each vector read once and written n times.
__global__ void __launch_bounds__(256) fork_kernel(const __grid_constant__ PageParams g,
                                                   const __grid_constant__ ForkDst f) {
  const int step = gridDim.x * blockDim.x, i0 = blockIdx.x * blockDim.x + threadIdx.x;
  if (blockIdx.y == 0) {
    for (int j = i0; j < f.n_pages; j += step) {
      const int pid = g.table[(size_t)f.src * g.mpps + j];
      for (int k = 0; k < f.n; ++k) g.table[(size_t)f.dst[k] * g.mpps + j] = pid;
    }
    return;
  }
  const size_t ring = (size_t)g.T * (D * 2 * 2), lh = blockIdx.y - 1;
  const uint4* src = reinterpret_cast<const uint4*>(g.tail + ((size_t)f.src * g.L * g.Hkv + lh) * ring);
  for (int i = i0; i < f.ring_vecs; i += step) {
    const uint4 v = src[i];
    for (int k = 0; k < f.n; ++k)
      reinterpret_cast<uint4*>(g.tail + ((size_t)f.dst[k] * g.L * g.Hkv + lh) * ring)[i] = v;
  }
}

// Old position of new row j, below `limit`: the old length, or for a row of the pages the
// old rows that pages hold (the block table may name pages behind them, from the id's
// earlier use, that other sequences own by now).  A list that is not ascending or passes the
// limit latches an error, and the row's own position is taken in its place (always below
// the limit: new length <= old length, with and without the tails).
__device__ __forceinline__ int kept_position(const CompactSeqs& q, const CompactSeq& s, int j, int limit, int* err) {
  if (j < s.start) return j;
  const int* k = q.keep + s.keep0 + (j - s.start);
  const int p = *k;
  const int before = j == s.start ? s.start - 1 : k[-1];
  if (p < j || p >= limit || p <= before) {
    atomicOr(err, ERR_BAD_ARG);
    return j;
  }
  return p;
}

__device__ __forceinline__ uint8_t* ring_chunk(uint8_t* ring, int slot, int kv, int c8) {
  uint8_t* tp = ring + (size_t)(slot / TAIL_TOK) * TAIL_PAGE_BYTES;
  const int r = slot % TAIL_TOK;
  return kv == 0 ? tp + (c8 * TAIL_TOK + r) * 16 : tp + TAIL_TOK * D * 2 + r * (D * 2) + c8 * 16;
}

// grid (slices of `cols` 16-byte columns, layer x head x K|V, sequence)
__global__ void __launch_bounds__(256) ring_move_kernel(const __grid_constant__ PageParams g,
                                                        const __grid_constant__ CompactSeqs q, int cols) {
  extern __shared__ uint4 held[];                        // [new tail rows][cols]
  const CompactSeq s = q.s[blockIdx.z];
  if (s.n_keep == 0) return;                             // nothing behind `start`: no ring row moves
  const int lhk = blockIdx.y, kv = lhk & 1;
  const int m = s.start + s.n_keep, nq_old = max(0, s.len - g.T);
  const int j0 = max(0, m - g.T), n = (m - j0) * cols, c0 = blockIdx.x * cols;
  uint8_t* ring = g.tail + ((size_t)s.seq * g.L * g.Hkv + (lhk >> 1)) * (size_t)g.T * (D * 2 * 2);
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int p = kept_position(q, s, j0 + i / cols, s.len, g.err);
    if (p >= nq_old) held[i] = *reinterpret_cast<const uint4*>(ring_chunk(ring, p % g.T, kv, c0 + i % cols));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int j = j0 + i / cols, p = kept_position(q, s, j, s.len, g.err);
    if (p >= nq_old && p != j) *reinterpret_cast<uint4*>(ring_chunk(ring, j % g.T, kv, c0 + i % cols)) = held[i];
  }
}

// grid (blocks of 8 ring rows, layer x head x K|V, sequence), a warp per row
__global__ void __launch_bounds__(256) ring_restore_kernel(const __grid_constant__ PageParams g,
                                                           const __grid_constant__ CompactSeqs q) {
  __shared__ __align__(16) float zs[8][D];
  const CompactSeq s = q.s[blockIdx.z];
  const int lane = threadIdx.x & 31, wib = threadIdx.x >> 5;
  const int lh = blockIdx.y >> 1, kv = blockIdx.y & 1;
  const int m = s.start + s.n_keep, nq_old = max(0, s.len - g.T);
  const int j = max(0, m - g.T) + (int)blockIdx.x * 8 + wib;
  if (j >= m) return;
  const int p = kept_position(q, s, j, s.len, g.err);
  if (p >= nq_old) return;
  const int pid = g.table[(size_t)s.seq * g.mpps + p / PAGE];
  if (pid < 0) { if (lane == 0) atomicOr(g.err, ERR_NO_PAGE); return; }
  const LayerInfo li = g.layers[lh / g.Hkv];
  const HeadInfo h = g.heads[lh];
  const float* mul = kv ? g.s_v : g.s_k;
  float x[4];
  page_row_original(g.cache + li.off + (size_t)pid * li.page_bytes + h.off, h, kv, p % PAGE, g.rot, g.bf16,
                    mul ? mul + (size_t)lh * D : nullptr, g.M, zs[wib], x);
  uint8_t* ring = g.tail + ((size_t)s.seq * g.L * g.Hkv + lh) * (size_t)g.T * (D * 2 * 2);
  *reinterpret_cast<uint2*>(ring_chunk(ring, j % g.T, kv, lane >> 1) + 8 * (lane & 1)) =
      make_uint2(float2_to_raw2(x[0], x[1], g.bf16), float2_to_raw2(x[2], x[3], g.bf16));
}

// The W-byte pieces of one plane: dst piece (i, t) <- src piece (i, its row's).  K code
// planes keep piece i of all 64 rows together, the others a row's pieces.
template <typename V>
__device__ __forceinline__ void gather_plane(uint8_t* dst, size_t plane, int row_bytes, bool kplane, int n_rows,
                                             const uint8_t* const* page, const uint8_t* row, uint32_t head_off) {
  const int pieces = row_bytes / (int)sizeof(V);
  for (int k = threadIdx.x; k < pieces * PAGE; k += blockDim.x) {
    const int t = kplane ? k % PAGE : k / pieces, i = kplane ? k / PAGE : k % pieces;
    if (t >= n_rows || !page[t]) continue;
    const int ts = row[t];
    const uint8_t* src = page[t] + head_off + plane;
    const int so = kplane ? i * PAGE + ts : ts * pieces + i, d = kplane ? i * PAGE + t : t * pieces + i;
    reinterpret_cast<V*>(dst + plane)[d] = reinterpret_cast<const V*>(src)[so];
  }
}
__device__ __forceinline__ void gather_rows(uint8_t* dst, size_t plane, int row_bytes, bool kplane, int n_rows,
                                            const uint8_t* const* page, const uint8_t* row, uint32_t head_off) {
  switch (interleave_w(row_bytes)) {
    case 16: gather_plane<uint4>(dst, plane, row_bytes, kplane, n_rows, page, row, head_off); break;
    case 8: gather_plane<uint2>(dst, plane, row_bytes, kplane, n_rows, page, row, head_off); break;
    case 4: gather_plane<uint32_t>(dst, plane, row_bytes, kplane, n_rows, page, row, head_off); break;
    default: gather_plane<uint16_t>(dst, plane, row_bytes, kplane, n_rows, page, row, head_off); break;
  }
}

// grid (destination pages, layers, kv heads): one page-head
__global__ void __launch_bounds__(128) gather_pages_kernel(const __grid_constant__ PageParams g,
                                                           const __grid_constant__ CompactSeqs q,
                                                           const __grid_constant__ CompactPages d) {
  __shared__ const uint8_t* page[PAGE];                 // source page of each row, null for none
  __shared__ uint8_t row[PAGE];
  const CompactSeq s = q.s[d.entry[blockIdx.x]];
  const int first = d.index[blockIdx.x] * PAGE;
  const int n_rows = min(PAGE, s.start + s.n_keep - g.T - first);
  const LayerInfo li = g.layers[blockIdx.y];
  if ((int)threadIdx.x < n_rows) {
    const int p = kept_position(q, s, first + threadIdx.x, max(0, s.len - g.T), g.err);
    const int pid = g.table[(size_t)s.seq * g.mpps + p / PAGE];
    if (pid < 0) atomicOr(g.err, ERR_NO_PAGE);
    page[threadIdx.x] = pid < 0 ? nullptr : g.cache + li.off + (size_t)pid * li.page_bytes;
    row[threadIdx.x] = (uint8_t)(p % PAGE);
  }
  __syncthreads();
  const HeadInfo h = g.heads[blockIdx.y * g.Hkv + blockIdx.z];
  uint8_t* dst = g.cache + li.off + (size_t)d.page[blockIdx.x] * li.page_bytes + h.off;
  size_t plane = 0;
  gather_rows(dst, plane, h.cbK, true, n_rows, page, row, h.off);
  plane += (size_t)PAGE * h.cbK;
  if (h.sbK) gather_rows(dst, plane, h.sbK, false, n_rows, page, row, h.off);
  plane += (size_t)PAGE * h.sbK;
  gather_rows(dst, plane, h.cbV, false, n_rows, page, row, h.off);
  plane += (size_t)PAGE * h.cbV;
  if (h.sbV) gather_rows(dst, plane, h.sbV, false, n_rows, page, row, h.off);
}

__global__ void __launch_bounds__(256) enter_pages_kernel(const __grid_constant__ PageParams g,
                                                          const __grid_constant__ CompactSeqs q,
                                                          const __grid_constant__ CompactPages d) {
  for (int i = threadIdx.x; i < d.n; i += blockDim.x)
    g.table[(size_t)q.s[d.entry[i]].seq * g.mpps + d.index[i]] = d.page[i];
}

// One plane of a page from canonical rows, in units of V.  A K code plane keeps the
// w-byte pieces of all 64 rows together (w as in kplane_off); the other planes, and the
// canonical rows, are row-major.
template <typename V>
__device__ __forceinline__ void scatter_plane(uint8_t* dst, const uint8_t* src, int row_bytes, bool kplane, int n_rows) {
  const int units = row_bytes / (int)sizeof(V);
  for (int k = threadIdx.x; k < units * PAGE; k += blockDim.x) {
    const int t = k / units, i = (k % units) * (int)sizeof(V);
    if (t < n_rows)
      *reinterpret_cast<V*>(dst + (kplane ? kplane_off(row_bytes, t, i) : t * row_bytes + i)) =
          *reinterpret_cast<const V*>(src + (size_t)t * row_bytes + i);
  }
}
// A head's canonical rows start behind those of the heads before it, so `src` need only
// be a multiple of 2: the unit is the widest that divides it and the row.
__device__ __forceinline__ void scatter_rows(uint8_t* dst, const uint8_t* src, int row_bytes, bool kplane, int n_rows) {
  const int w = min(interleave_w(row_bytes), interleave_w((int)((uintptr_t)src & 15) | 16));
  switch (w) {
    case 16: scatter_plane<uint4>(dst, src, row_bytes, kplane, n_rows); break;
    case 8: scatter_plane<uint2>(dst, src, row_bytes, kplane, n_rows); break;
    case 4: scatter_plane<uint32_t>(dst, src, row_bytes, kplane, n_rows); break;
    default: scatter_plane<uint16_t>(dst, src, row_bytes, kplane, n_rows); break;
  }
}

// grid (pages of the sequence, kv heads, K|V)
__global__ void __launch_bounds__(128) load_pages_kernel(const __grid_constant__ LoadParams p) {
  const int first = blockIdx.x * PAGE, kv = blockIdx.z;
  const int n = min(PAGE, p.n_rows - first);
  const PageParams& g = p.g;
  const int pid = g.table[(size_t)p.seq * g.mpps + blockIdx.x];
  if (pid < 0) { if (threadIdx.x == 0) atomicOr(g.err, ERR_NO_PAGE); return; }
  const LayerInfo li = g.layers[p.layer];
  const HeadInfo* heads = g.heads + (size_t)p.layer * g.Hkv;
  const HeadInfo h = heads[blockIdx.y];
  const int cb = kv ? h.cbV : h.cbK, sb = kv ? h.sbV : h.sbK;
  size_t c0 = 0, s0 = 0;                                 // bytes of a row over the heads before this one
  for (int k = 0; k < (int)blockIdx.y; ++k) {
    c0 += kv ? heads[k].cbV : heads[k].cbK;
    s0 += kv ? heads[k].sbV : heads[k].sbK;
  }
  uint8_t* region = g.cache + li.off + (size_t)pid * li.page_bytes + h.off;
  uint8_t* codes = kv ? region + PAGE * (h.cbK + h.sbK) : region;
  scatter_rows(codes, p.codes[kv] + c0 * p.n_rows + (size_t)first * cb, cb, kv == 0, n);
  if (sb) scatter_rows(codes + (size_t)PAGE * cb, p.scales[kv] + s0 * p.n_rows + (size_t)first * sb, sb, false, n);
}

// grid (blocks of 16 ring rows, kv heads, K|V): thread = (row, 16-byte chunk)
__global__ void __launch_bounds__(256) load_tail_kernel(const __grid_constant__ LoadParams p) {
  const int i = blockIdx.x * 16 + (threadIdx.x >> 4), c8 = threadIdx.x & 15, kv = blockIdx.z;
  if (i >= p.n_tail) return;
  const PageParams& g = p.g;
  uint8_t* ring = g.tail + (((size_t)p.seq * g.L + p.layer) * g.Hkv + blockIdx.y) * (size_t)g.T * (D * 2 * 2);
  *reinterpret_cast<uint4*>(ring_chunk(ring, (p.n_rows + i) % g.T, kv, c8)) =
      *reinterpret_cast<const uint4*>(p.tail[kv] + ((size_t)i * g.Hkv + blockIdx.y) * (D * 2) + c8 * 16);
}

constexpr int RING_SMEM = 200 * 1024;

}  // namespace

int compact_max_tail() { return RING_SMEM / 16; }

cudaError_t launch_copy_pages(const PageParams& g, int n, const int* src, const int* dst, cudaStream_t s) {
  for (int k = 0; k < n; k += COPY_MAX) {
    PagePairs q;
    q.n = std::min(COPY_MAX, n - k);
    std::copy(src + k, src + k + q.n, q.src);
    std::copy(dst + k, dst + k + q.n, q.dst);
    copy_pages_kernel<<<dim3(q.n, g.L), 256, 0, s>>>(g, q);
    note_launches(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_layer_tables(HeadInfo* heads, LayerInfo* layer, const HeadInfo* h, int n_heads, LayerInfo li,
                                cudaStream_t s) {
  LayerTables t;
  t.heads = heads;
  t.layer = layer;
  t.n_heads = n_heads;
  t.li = li;
  std::copy(h, h + n_heads, t.h);
  layer_tables_kernel<<<1, 32, 0, s>>>(t);
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_fork(const PageParams& g, int src, int n, const int* dst, int n_pages, int ring_tokens,
                        cudaStream_t s) {
  ForkDst f;
  f.src = src;
  f.n = n;
  f.n_pages = n_pages;
  f.ring_vecs = (ring_tokens + TAIL_TOK - 1) / TAIL_TOK * (TAIL_PAGE_BYTES / 16);
  std::copy(dst, dst + n, f.dst);
  const int work = std::max(f.ring_vecs, n_pages);
  if (work == 0) return cudaSuccess;
  const int bx = std::max(1, std::min(64, (work + 511) / 512));
  fork_kernel<<<dim3(bx, f.ring_vecs ? g.L * g.Hkv + 1 : 1), 256, 0, s>>>(g, f);
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_compact_tail(const PageParams& g, const CompactSeqs& q, cudaStream_t s) {
  if (g.T == 0 || q.n == 0) return cudaSuccess;
  int rows = 0;
  bool moves = false, back = false;
  for (int i = 0; i < q.n; ++i) {
    const int m = q.s[i].start + q.s[i].n_keep;
    rows = std::max(rows, std::min(m, g.T));
    moves |= q.s[i].n_keep > 0;
    back |= q.s[i].len > g.T && m > 0;                   // rows below the tail exist and may come back
  }
  if (moves && rows > 0) {
    // 16-byte columns of a CTA: about 8 KiB of held rows (a 256-token tail of 2 x 8 heads:
    // 14 us with 32 KiB and a quarter of the CTAs, 7 us so)
    int cols = 16;
    while (cols > 1 && (size_t)rows * 16 * cols > 8 * 1024) cols >>= 1;
    const size_t smem = (size_t)rows * 16 * cols;
    const cudaError_t a = cudaFuncSetAttribute(ring_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_SMEM);
    if (a != cudaSuccess) return a;
    ring_move_kernel<<<dim3(16 / cols, g.L * g.Hkv * 2, q.n), 256, smem, s>>>(g, q, cols);
    note_launches(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (back && rows > 0) {
    ring_restore_kernel<<<dim3((rows + 7) / 8, g.L * g.Hkv * 2, q.n), 256, 0, s>>>(g, q);
    note_launches(1);
    return cudaGetLastError();
  }
  return cudaSuccess;
}

cudaError_t launch_compact_pages(const PageParams& g, const CompactSeqs& q, const CompactPages& d, cudaStream_t s) {
  if (d.n == 0) return cudaSuccess;
  gather_pages_kernel<<<dim3(d.n, g.L, g.Hkv), 128, 0, s>>>(g, q, d);
  note_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  enter_pages_kernel<<<1, 256, 0, s>>>(g, q, d);
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_load(const LoadParams& p, cudaStream_t s) {
  if (p.n_rows > 0) {
    load_pages_kernel<<<dim3((p.n_rows + PAGE - 1) / PAGE, p.g.Hkv, 2), 128, 0, s>>>(p);
    note_launches(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (p.n_tail > 0) {
    load_tail_kernel<<<dim3((p.n_tail + 15) / 16, p.g.Hkv, 2), 256, 0, s>>>(p);
    note_launches(1);
    return cudaGetLastError();
  }
  return cudaSuccess;
}

}  // namespace kvq
