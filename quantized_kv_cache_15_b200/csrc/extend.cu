// Attention of several new tokens per sequence: the CUDA-core kernel (layers with the
// rank codec) and the merge of the partial results of either kernel.
//
//   s_t = q . k_t * scale,  p_t = 2^(s_t - m),  out = sum_t p_t v_t / sum_t p_t
//
// over the positions a query sees: all before the sequence's last n_q tokens, and of
// those the ones its mask bits name (without a mask: up to its own).
#include "extend.h"

#include "dequant_row.cuh"
#include "ptx.cuh"

namespace kvq {

namespace {

constexpr int SIMPLE_ROWS = 16;
constexpr int SIMPLE_WARPS = 4;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// One row's query in the basis of the unit's keys, times the softmax scale (log2 units).
__device__ void load_query(const ExtendParams& p, const ExtendUnit& u, const ExtendRow& w, float* zs, float x[4]) {
  const int lane = threadIdx.x & 31;
  load_row_raw(p.q + ((size_t)(p.q0[w.entry] + w.query) * p.Hq + w.head) * D, x, p.bf16);
  if (!ex_raw_k(p, u)) {
    const HeadInfo& h = p.heads[u.head];
    if (h.kcodec == KVQ_RANK) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) zs[4 * lane + i] = x[i];
      __syncwarp();
      float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * lane + i < h.r) {
          const float* M = p.M + h.m_off + (size_t)(4 * lane + i) * D;
          for (int c = 0; c < D; ++c) y[i] = fmaf(M[c], zs[c], y[i]);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = y[i];
    } else if (p.rot != KVQ_ROT_NONE) {
      if (p.s_k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] *= p.s_k[(size_t)u.head * D + 4 * lane + i];
      }
      fwht_row(x);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] *= p.qscale;
}

}  // namespace

// CUDA-core form: a warp takes every fourth token of a tile, a lane four channels of
// it; each (row, token) product is a warp sum.  Bound by instructions (about 15 a row
// and token); it serves the rank codec, whose rows have no 32-value blocks for the
// tensor-core kernel's operand images.
__global__ void __launch_bounds__(32 * SIMPLE_WARPS) extend_simple_kernel(const __grid_constant__ ExtendParams p) {
  __shared__ __align__(16) float qs[SIMPLE_ROWS][D];
  __shared__ __align__(16) float os[SIMPLE_WARPS][SIMPLE_ROWS][D];
  __shared__ float ms[SIMPLE_WARPS][SIMPLE_ROWS], ls[SIMPLE_WARPS][SIMPLE_ROWS];
  __shared__ __align__(16) float zs[SIMPLE_WARPS][D];
  __shared__ int base[SIMPLE_ROWS];                      // first of the entry's last n_q positions; > every position: all seen
  __shared__ unsigned long long bits[SIMPLE_ROWS];       // which of them the row sees, or (causal) its own query index
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ExtendWalk walk = ex_walk(p, blockIdx.x);
  ExtendUnit u;
  int k0, k1;
  while (ex_next(p, walk, u, k0, k1)) {
    for (int r = warp; r < SIMPLE_ROWS; r += SIMPLE_WARPS) {
      const ExtendRow w = ex_row(p, u, r);
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (w.entry >= 0) load_query(p, u, w, zs[warp], x);
      *reinterpret_cast<float4*>(&qs[r][4 * lane]) = make_float4(x[0], x[1], x[2], x[3]);
      if (lane == 0) {
        base[r] = w.entry < 0 ? -1 : u.kind == EX_SHARED ? 0x7fffffff : p.len[w.entry] - p.nq[w.entry];
        bits[r] = w.entry < 0 ? 0ull : p.mask ? p.mask[p.q0[w.entry] + w.query] : (unsigned long long)w.query;
      }
    }
    __syncthreads();
    const HeadInfo& h = p.heads[u.head];
    const int seq = u.kind == EX_SHARED ? p.seq[p.order[p.g_first[u.index]]] : p.seq[u.index];
    int lo, hi;
    ex_range(p, u, &lo, &hi);
    float m[SIMPLE_ROWS], l[SIMPLE_ROWS], acc[SIMPLE_ROWS][4];
#pragma unroll
    for (int r = 0; r < SIMPLE_ROWS; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
      acc[r][0] = acc[r][1] = acc[r][2] = acc[r][3] = 0.f;
    }
    const int p0 = lo + k0 * EX_TILE, p1 = min(hi, lo + k1 * EX_TILE);
    for (int pos = p0 + warp; pos < p1; pos += SIMPLE_WARPS) {
      float k[4], v[4];
      if (u.kind == EX_TAIL) {
        const int slot = pos % p.T;
        const uint8_t* tp = p.tail + (((size_t)seq * p.L + p.layer) * p.Hkv + u.head) * (size_t)p.T * (D * 2 * 2) +
                            (size_t)(slot / TAIL_TOK) * TAIL_PAGE_BYTES;
        const int r16 = slot % TAIL_TOK;
        const uint2 a = *reinterpret_cast<const uint2*>(tp + ((lane >> 1) * TAIL_TOK + r16) * 16 + (lane & 1) * 8);
        const uint2 b = *reinterpret_cast<const uint2*>(tp + TAIL_TOK * D * 2 + r16 * (D * 2) + 8 * lane);
        const float2 a0 = raw2_to_float2(a.x, p.bf16), a1 = raw2_to_float2(a.y, p.bf16);
        const float2 b0 = raw2_to_float2(b.x, p.bf16), b1 = raw2_to_float2(b.y, p.bf16);
        k[0] = a0.x; k[1] = a0.y; k[2] = a1.x; k[3] = a1.y;
        v[0] = b0.x; v[1] = b0.y; v[2] = b1.x; v[3] = b1.y;
      } else {
        const int pid = p.table[(size_t)seq * p.mpps + pos / PAGE];
        if (pid < 0) { if (lane == 0) atomicOr(p.err, ERR_NO_PAGE); continue; }
        const uint8_t* region = p.pool + (size_t)pid * p.page_bytes + h.off;
        page_row_stored(region, h, 0, pos % PAGE, p.bf16, k);
        page_row_stored(region, h, 1, pos % PAGE, p.bf16, v);
      }
#pragma unroll
      for (int r = 0; r < SIMPLE_ROWS; ++r) {
        if (base[r] < 0) continue;
        if (pos >= base[r]) {
          const int j = pos - base[r];
          if (p.mask ? !((bits[r] >> j) & 1ull) : j > (int)bits[r]) continue;
        }
        const float4 q = *reinterpret_cast<const float4*>(&qs[r][4 * lane]);
        const float s = warp_sum(fmaf(q.x, k[0], fmaf(q.y, k[1], fmaf(q.z, k[2], q.w * k[3]))));
        float w = 1.f;
        if (s > m[r]) {
          const float a = ex2(m[r] - s);
          l[r] *= a;
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][i] *= a;
          m[r] = s;
        } else {
          w = ex2(s - m[r]);
        }
        l[r] += w;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][i] = fmaf(w, v[i], acc[r][i]);
      }
    }
#pragma unroll
    for (int r = 0; r < SIMPLE_ROWS; ++r) {
      *reinterpret_cast<float4*>(&os[warp][r][4 * lane]) = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
      if (lane == 0) { ms[warp][r] = m[r]; ls[warp][r] = l[r]; }
    }
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x + u.unit;
    for (int r = warp; r < SIMPLE_ROWS; r += SIMPLE_WARPS) {
      if (base[r] < 0) continue;
      float M = ms[0][r];
      for (int w = 1; w < SIMPLE_WARPS; ++w) M = fmaxf(M, ms[w][r]);
      float L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
      for (int w = 0; w < SIMPLE_WARPS; ++w) {
        const float f = ls[w][r] == 0.f ? 0.f : ls[w][r] != ls[w][r] ? ls[w][r] : ex2(ms[w][r] - M);
        if (f == 0.f) continue;
        L = fmaf(f, ls[w][r], L);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = fmaf(f, os[w][r][4 * lane + i], o[i]);
      }
      *reinterpret_cast<float4*>(p.part_o + (slot * p.N + r) * D + 4 * lane) = make_float4(o[0], o[1], o[2], o[3]);
      if (lane == 0) p.part_ml[slot * p.N + r] = make_float2(M, L);
    }
    __syncthreads();
  }
}

// W warps per (query, query head): its units' partials (at most one shared, one own and
// one tail unit) are weighed by 2^(m - max) in slot order, so the result does not depend on
// which CTA finished first; pages' partials go back to the original basis (staged Hadamard
// and variance multipliers, or M_h^T), the tail's already are.  Bound by reading the
// partials, (128 + 2) floats each.
template <int W>
__global__ void __launch_bounds__(128) extend_merge_kernel(const __grid_constant__ ExtendParams p) {
  griddep_launch_dependents();
  constexpr int ROWS = 4 / W;                            // rows of a CTA
  __shared__ __align__(16) float os[ROWS][2][W][D];
  __shared__ float lsum[ROWS][W];
  __shared__ __align__(16) float zs[ROWS][D];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % W, mine = (threadIdx.x >> 5) / W;
  const int at_row = blockIdx.x * ROWS + mine;
  if (at_row >= p.total_q * p.Hq) return;                // whole rows (W = 4: the whole CTA)
  const int qi = at_row / p.Hq, hq = at_row % p.Hq;
  const int e = prefix_find(p.q0, p.n_entries, qi);
  const int j = qi - p.q0[e], head = hq / p.G, g = hq % p.G;
  // the slots of this row's partials: up to three runs
  int first[3], count[3], row[3];
  int n = 0;
#pragma unroll
  for (int kind = 0; kind < 3; ++kind) {
    first[kind] = count[kind] = row[kind] = 0;
    const int at = kind == EX_SHARED ? p.member0[e] + j : j;
    if (kind == EX_SHARED && p.group[e] < 0) continue;
    const ExtendUnit u = ex_unit(p, kind, kind == EX_SHARED ? p.group[e] : e, head, at / p.QB);
    if (u.tiles == 0) continue;
    const int c0 = u.at / p.per, c1 = ex_start(p, u, u.tiles - 1) / p.per;
    first[kind] = c0 + u.unit;
    count[kind] = c1 - c0 + 1;
    row[kind] = (at % p.QB) * p.G + g;
    n += count[kind];
  }
  auto place = [&](int i) -> size_t {                    // partial i of the row
    const int k = i < count[0] ? 0 : i < count[0] + count[1] ? 1 : 2;
    const int in = k == 0 ? i : k == 1 ? i - count[0] : i - count[0] - count[1];
    return (size_t)(first[k] + in) * p.N + row[k];
  };
  griddep_wait();
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, p.part_ml[place(i)].x);
#pragma unroll
  for (int m = 16; m; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
  const int n_paged = count[0] + count[1];
  float l = 0.f, a[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    const int i0 = part == 0 ? 0 : n_paged, i1 = part == 0 ? n_paged : n;
#pragma unroll 4
    for (int i = i0 + warp; i < i1; i += W) {
      const size_t at = place(i);
      const float2 ml = p.part_ml[at];
      const float4 o = *reinterpret_cast<const float4*>(p.part_o + at * D + 4 * lane);
      const float f = ml.y == 0.f ? 0.f : ml.y != ml.y ? ml.y : ex2(ml.x - M);
      if (f != 0.f) {                                     // also NaN
        l = fmaf(f, ml.y, l);
        a[part][0] = fmaf(f, o.x, a[part][0]);
        a[part][1] = fmaf(f, o.y, a[part][1]);
        a[part][2] = fmaf(f, o.z, a[part][2]);
        a[part][3] = fmaf(f, o.w, a[part][3]);
      }
    }
  }
  if (W > 1) {
#pragma unroll
    for (int part = 0; part < 2; ++part)
      *reinterpret_cast<float4*>(&os[mine][part][warp][4 * lane]) = make_float4(a[part][0], a[part][1], a[part][2], a[part][3]);
    if (lane == 0) lsum[mine][warp] = l;
    __syncthreads();
    if (warp) return;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) l += lsum[mine][w];
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[part][i] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) a[part][i] += os[mine][part][w][4 * lane + i];
      }
  }
  const HeadInfo& h = p.heads[head];
  if (n_paged) row_to_original(h.vcodec, h, p.rot, p.s_v ? p.s_v + (size_t)head * D : nullptr, p.M, zs[mine], a[0]);
  const float inv = l == 0.f ? 0.f : 1.f / l;            // a row that sees nothing is zero
  const uint2 w = make_uint2(float2_to_raw2((a[0][0] + a[1][0]) * inv, (a[0][1] + a[1][1]) * inv, p.bf16),
                             float2_to_raw2((a[0][2] + a[1][2]) * inv, (a[0][3] + a[1][3]) * inv, p.bf16));
  *reinterpret_cast<uint2*>(p.out + ((size_t)qi * p.Hq + hq) * D + 4 * lane) = w;
}

cudaError_t launch_extend_simple(const ExtendParams& p, cudaStream_t s) {
  extend_simple_kernel<<<p.n_ctas, 32 * SIMPLE_WARPS, 0, s>>>(p);
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_extend_merge(const ExtendParams& p, cudaStream_t s) {
  // Four warps share a row's partials where rows are few and long; else a warp takes a row
  // (2048 rows of 3 partials: 15 us with four warps a row, 6 us with one).
  const int rows = p.total_q * p.Hq;
  const int W = rows <= 1024 ? 4 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + 4 / W - 1) / (4 / W)));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, W == 4 ? extend_merge_kernel<4> : extend_merge_kernel<1>, p);
  note_launches(1);
  return e;
}

}  // namespace kvq
