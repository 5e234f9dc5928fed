// Merge of the multi-token attention's partial results.
#include "extend.h"

#include "dequant_row.cuh"
#include "ptx.cuh"

namespace kvq {

namespace {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
}  // namespace

// W warps per (query, query head): its units' partials (at most one shared, one own and
// one tail unit) are weighed by 2^(m - max) in slot order, so the result does not depend on
// which CTA finished first; pages' partials go back to the original basis (staged Hadamard
// and variance multipliers, or M_h^T), the tail's already are.  Bound by reading the
// partials, (128 + 2) floats each.
// Of two launches p is the entries' and s the groups'.
template <int W, bool TWO>
__device__ __forceinline__ void merge_rows(const ExtendParams& p, const ExtendParams& s) {
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
    const ExtendParams& c = TWO && kind == EX_SHARED ? s : p;
    const ExtendUnit u = ex_unit(c, kind, kind == EX_SHARED ? p.group[e] : e, head, at / c.QB);
    if (u.tiles == 0) continue;
    const int c0 = u.at / c.per, c1 = ex_start(c, u, u.tiles - 1) / c.per;
    first[kind] = c0 + u.unit;
    count[kind] = c1 - c0 + 1;
    row[kind] = (at % c.QB) * p.G + g;
    n += count[kind];
  }
  auto place = [&](int i) -> size_t {                    // partial i of the row
    const int k = i < count[0] ? 0 : i < count[0] + count[1] ? 1 : 2;
    const int in = k == 0 ? i : k == 1 ? i - count[0] : i - count[0] - count[1];
    return (size_t)(first[k] + in) * (TWO && k == 0 ? s.N : p.N) + row[k];
  };
  griddep_wait();
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, (TWO && i < count[0] ? s : p).part_ml[place(i)].x);
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
      const ExtendParams& c = TWO && i < count[0] ? s : p;
      const float2 ml = c.part_ml[at];
      const float4 o = *reinterpret_cast<const float4*>(c.part_o + at * D + 4 * lane);
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

template <int W>
__global__ void __launch_bounds__(128) extend_merge_kernel(const __grid_constant__ ExtendParams p) {
  merge_rows<W, false>(p, p);
}
template <int W>
__global__ void __launch_bounds__(128) extend_merge_two_kernel(const __grid_constant__ ExtendParams p,
                                                               const __grid_constant__ ExtendParams s) {
  merge_rows<W, true>(p, s);
}
static_assert(2 * sizeof(ExtendParams) <= 32764, "kernel parameters");

cudaError_t launch_extend_merge(const ExtendParams& p, const ExtendParams* groups, cudaStream_t s) {
  // Four warps share a row's partials where rows are few and long; else a warp takes a row
  // (the whole call with four and with one: 256 rows of some 20 partials 111 us and 117;
  // 512 rows 47, 50; 1024 rows 291, 293; 2048 rows 99, 96; 4096 rows of 3 to 9 partials 66, 60).
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
  const cudaError_t e = groups ? cudaLaunchKernelEx(&cfg, W == 4 ? extend_merge_two_kernel<4> : extend_merge_two_kernel<1>, p, *groups)
                               : cudaLaunchKernelEx(&cfg, W == 4 ? extend_merge_kernel<4> : extend_merge_kernel<1>, p);
  note_launches(1);
  return e;
}

}  // namespace kvq
