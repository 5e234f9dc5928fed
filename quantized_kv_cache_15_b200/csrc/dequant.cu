// Reading the cache back: rows in the original basis (kvq_dequantize) and the
// canonical packed rows (kvq_read_rows).
#include "dequant_row.cuh"

namespace kvq {

// A warp a row: plans with a projection.
__global__ void __launch_bounds__(256) dequant_kernel(const __grid_constant__ DecodeParams p, int seq, int len,
                                                      long t0, long n_rows, float* k_out, float* v_out) {
  __shared__ __align__(16) float zs[8][D];
  const int lane = threadIdx.x & 31, wib = threadIdx.x >> 5;
  const long gw = (long)blockIdx.x * 8 + wib;
  const long row = gw / (p.Hkv * 2);
  if (row >= n_rows) return;
  const int rem = (int)(gw % (p.Hkv * 2));
  const int head = rem >> 1, kv = rem & 1;
  float* out = kv ? v_out : k_out;
  if (!out) return;
  const long pos = t0 + row;
  const int T = p.T;
  const long nq = len > T ? len - T : 0;
  const HeadInfo& h = p.heads[head];
  float x[4];
  if (pos >= nq) {
    // tail ring, raw fp16
    const uint8_t* ring = p.tail + (((size_t)seq * p.L + p.layer) * p.Hkv + head) * (size_t)T * (D * 2 * 2);
    const int slot = (int)(pos % T);
    const uint8_t* tp = ring + (size_t)(slot / TAIL_TOK) * TAIL_PAGE_BYTES;
    const int r = slot % TAIL_TOK;
    const uint8_t* src = kv == 0 ? tp + ((lane >> 1) * TAIL_TOK + r) * 16 + (lane & 1) * 8
                                 : tp + TAIL_TOK * D * 2 + r * (D * 2) + 8 * lane;
    const uint2 w = *reinterpret_cast<const uint2*>(src);
    const float2 a = raw2_to_float2(w.x, p.bf16), b = raw2_to_float2(w.y, p.bf16);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  } else {
    const int pid = p.block_table[(size_t)seq * p.max_pages_per_seq + pos / PAGE];
    if (pid < 0) { if (lane == 0) atomicOr(p.err, ERR_NO_PAGE); return; }
    const float* mul = kv ? p.s_v : p.s_k;
    page_row_original(p.pool + (size_t)pid * p.page_bytes + h.off, h, kv, (int)(pos % PAGE), p.rot, p.bf16,
                      mul ? mul + (size_t)head * D : nullptr, p.M, zs[wib], x);
  }
  float4 o = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(out + ((size_t)row * p.Hkv + head) * D + 4 * lane) = o;
}

// 32 bytes to global memory in one store (a whole sector; two 16-byte stores of a lane whose
// neighbours write elsewhere cost two partial ones).
__device__ __forceinline__ void store8(float* dst, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
               "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// The same rows with four threads a row, a 32-value block each, for the plans without a
// projection: the Hadamard stages inside a block need no communication and a block's codes
// come in a few wide loads.  For the stages across blocks the values then turn in shared
// memory, so that a thread has channels 8 q .. 8 q + 7 of every block; a quad's stores then
// fill 128-byte lines.  What bounds it is the number of passes that loads, stores and
// exchanges take through the L1 data pipe (8192 rows of 8 heads, K and V: shuffles and
// stores block by block 31 us, so 19 us; a warp a row 60 us; filling the output with a
// constant takes 12).  Neighbouring quads take neighbouring rows of one
// (head, K|V).  Every value goes through the same correctly rounded operations as above.
__global__ void __launch_bounds__(128) dequant_quad_kernel(const __grid_constant__ DecodeParams p, int seq, int len,
                                                           long t0, int n_rows, float* k_out, float* v_out) {
  // neighbouring CTAs take the heads of the same 32 rows, which lie next to each other
  const int rows = blockIdx.x / (p.Hkv * 2), of = blockIdx.x % (p.Hkv * 2);
  const int row = rows * 32 + ((int)threadIdx.x >> 2), q = threadIdx.x & 3;
  const int head = of % p.Hkv, kv = of / p.Hkv;
  float* out = kv ? v_out : k_out;
  if (!out) return;
  __shared__ float4 turn[32][32];                        // [row of the CTA][16-byte chunk of the row, swizzled]
  bool ok = row < n_rows, rotated = false;
  const long pos = t0 + row;
  const int T = p.T;
  const int nq = len > T ? len - T : 0;
  const HeadInfo& h = p.heads[head];
  float v[32];
  if (!ok) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.f;
  } else if (pos >= nq) {
    const uint8_t* ring = p.tail + (((size_t)seq * p.L + p.layer) * p.Hkv + head) * (size_t)T * (D * 2 * 2);
    const int slot = (int)(pos % T), r = slot % TAIL_TOK;
    const uint8_t* tp = ring + (size_t)(slot / TAIL_TOK) * TAIL_PAGE_BYTES;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int c8 = 4 * q + c;
      const uint8_t* src = kv == 0 ? tp + (c8 * TAIL_TOK + r) * 16 : tp + TAIL_TOK * D * 2 + r * (D * 2) + 16 * c8;
      chunk_to_float(*reinterpret_cast<const uint4*>(src), v + 8 * c, p.bf16);
    }
  } else {
    const int codec = kv ? h.vcodec : h.kcodec;
    const int cb = kv ? h.cbV : h.cbK, sb = kv ? h.sbV : h.sbK;
    const int pid = p.block_table[(size_t)seq * p.max_pages_per_seq + pos / PAGE];
    if (pid < 0) { if (q == 0) atomicOr(p.err, ERR_NO_PAGE); ok = false; }
    const uint8_t* region = p.pool + (size_t)max(pid, 0) * p.page_bytes + h.off;
    const uint8_t* codes = kv ? region + PAGE * (h.cbK + h.sbK) : region;
    const uint8_t* scales = codes + PAGE * cb;
    const int t = (int)(pos % PAGE);
    const bool kplane = kv == 0;
    switch (codec) {
      case KVQ_F16:
#pragma unroll
        for (int c = 0; c < 4; ++c)
          chunk_to_float(*reinterpret_cast<const uint4*>(row_word_ptr(codes, kplane, cb, t, 16 * q + 4 * c)), v + 8 * c,
                         p.bf16);
        break;
      case KVQ_Q8_0: dequantize_block_quad<0, 8>(codes, scales, t, kplane, cb, sb, v); break;
      case KVQ_Q6_0: dequantize_block_quad<0, 6>(codes, scales, t, kplane, cb, sb, v); break;
      case KVQ_Q5_0: dequantize_block_quad<0, 5>(codes, scales, t, kplane, cb, sb, v); break;
      case KVQ_Q4_0: dequantize_block_quad<0, 4>(codes, scales, t, kplane, cb, sb, v); break;
      case KVQ_Q3_0: dequantize_block_quad<0, 3>(codes, scales, t, kplane, cb, sb, v); break;
      case KVQ_Q2_0: dequantize_block_quad<0, 2>(codes, scales, t, kplane, cb, sb, v); break;
      case KVQ_Q8_1: dequantize_block_quad<1, 8>(codes, scales, t, kplane, cb, sb, v); break;
      case KVQ_Q6_1: dequantize_block_quad<1, 6>(codes, scales, t, kplane, cb, sb, v); break;
      case KVQ_Q5_1: dequantize_block_quad<1, 5>(codes, scales, t, kplane, cb, sb, v); break;
      case KVQ_Q4_1: dequantize_block_quad<1, 4>(codes, scales, t, kplane, cb, sb, v); break;
      case KVQ_Q3_1: dequantize_block_quad<1, 3>(codes, scales, t, kplane, cb, sb, v); break;
      case KVQ_Q2_1: dequantize_block_quad<1, 2>(codes, scales, t, kplane, cb, sb, v); break;
      default: ok = false; break;
    }
    rotated = codec != KVQ_F16 && p.rot != KVQ_ROT_NONE;
  }
  if (rotated) {                                         // the Hadamard stages h = 1 .. 16
#pragma unroll
    for (int s = 1; s < 32; s <<= 1)
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if ((i & s) == 0) {
          const float a = v[i], b = v[i + s];
          v[i] = __fadd_rn(a, b);
          v[i + s] = __fsub_rn(a, b);
        }
  }
  // Chunk k of block b of a row lies at 8 b + (k ^ (b + 4 (row mod 2))); odd rows take their
  // two chunks of a block in the other order: a phase of eight lanes meets all banks, both ways.
  const int r = (int)threadIdx.x >> 2, odd = r & 1;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    turn[r][8 * q + (k ^ (q + 4 * odd))] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  __syncwarp();                                          // a row is one quad's
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const float4 x = turn[r][8 * b + ((2 * q + odd) ^ (b + 4 * odd))], y = turn[r][8 * b + ((2 * q + 1 - odd) ^ (b + 4 * odd))];
    const float4 lo = odd ? y : x, hi = odd ? x : y;
    v[8 * b] = lo.x; v[8 * b + 1] = lo.y; v[8 * b + 2] = lo.z; v[8 * b + 3] = lo.w;
    v[8 * b + 4] = hi.x; v[8 * b + 5] = hi.y; v[8 * b + 6] = hi.z; v[8 * b + 7] = hi.w;
  }
  if (!ok) return;
  const float* mul = kv ? p.s_v : p.s_k;
  if (rotated) {
#pragma unroll
    for (int s = 8; s < 32; s <<= 1)                     // h = 32, 64, then the factors
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if ((i & s) == 0) {
          const float a = v[i], b = v[i + s];
          v[i] = __fadd_rn(a, b);
          v[i + s] = __fsub_rn(a, b);
        }
    const float c = hadamard_c();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __fmul_rn(v[i], c);
    if (mul) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float4* m4 = reinterpret_cast<const float4*>(mul + (size_t)head * D + 32 * b + 8 * q);
        const float4 m = m4[0], n = m4[1];
        v[8 * b] *= m.x; v[8 * b + 1] *= m.y; v[8 * b + 2] *= m.z; v[8 * b + 3] *= m.w;
        v[8 * b + 4] *= n.x; v[8 * b + 5] *= n.y; v[8 * b + 6] *= n.z; v[8 * b + 7] *= n.w;
      }
    }
  }
  float* dst = out + ((size_t)row * p.Hkv + head) * D + 8 * q;
  if ((uintptr_t)out % 32 == 0) {
#pragma unroll
    for (int b = 0; b < 4; ++b) store8(dst + 32 * b, v + 8 * b);
  } else {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      *reinterpret_cast<float4*>(dst + 32 * b) = make_float4(v[8 * b], v[8 * b + 1], v[8 * b + 2], v[8 * b + 3]);
      *reinterpret_cast<float4*>(dst + 32 * b + 4) = make_float4(v[8 * b + 4], v[8 * b + 5], v[8 * b + 6], v[8 * b + 7]);
    }
  }
}

cudaError_t launch_dequantize(const DecodeParams& p, int seq, int64_t t0, int64_t t1, float* k_out, float* v_out,
                              cudaStream_t s) {
  const long n_rows = (long)(t1 - t0);
  if (n_rows <= 0) return cudaSuccess;
  if (p.rot != KVQ_ROT_PROJECTION) {
    dequant_quad_kernel<<<(unsigned)((n_rows + 31) / 32 * p.Hkv * 2), 128, 0, s>>>(p, seq, p.len[0], (long)t0, (int)n_rows,
                                                                                   k_out, v_out);
    note_launches(1);
    return cudaGetLastError();
  }
  const long warps = n_rows * p.Hkv * 2;
  dequant_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, s>>>(p, seq, p.len[0], (long)t0, n_rows, k_out, v_out);
  note_launches(1);
  return cudaGetLastError();
}

__global__ void read_rows_kernel(const __grid_constant__ DecodeParams p, int seq, long t0, long n_rows, int kv,
                                 uint8_t* codes_out, uint8_t* scales_out) {
  const int lane = threadIdx.x & 31, wib = threadIdx.x >> 5;
  const long gw = (long)blockIdx.x * 8 + wib;
  const long row = gw / p.Hkv;
  if (row >= n_rows) return;
  const int head = (int)(gw % p.Hkv);
  size_t coff = 0, soff = 0;
  for (int hh = 0; hh < head; ++hh) {
    coff += (size_t)n_rows * (kv ? p.heads[hh].cbV : p.heads[hh].cbK);
    soff += (size_t)n_rows * (kv ? p.heads[hh].sbV : p.heads[hh].sbK);
  }
  const HeadInfo& h = p.heads[head];
  const int cb = kv ? h.cbV : h.cbK, sb = kv ? h.sbV : h.sbK;
  const long pos = t0 + row;
  const int pid = p.block_table[(size_t)seq * p.max_pages_per_seq + pos / PAGE];
  if (pid < 0) { if (lane == 0) atomicOr(p.err, ERR_NO_PAGE); return; }
  const uint8_t* region = p.pool + (size_t)pid * p.page_bytes + h.off;
  const uint8_t* codes = kv ? region + PAGE * (h.cbK + h.sbK) : region;
  const uint8_t* scales = codes + PAGE * cb;
  const int t = (int)(pos % PAGE);
  for (int i = lane; i < cb; i += 32)
    codes_out[coff + (size_t)row * cb + i] = codes[kv == 0 ? kplane_off(cb, t, i) : t * cb + i];
  for (int i = lane; i < sb; i += 32) scales_out[soff + (size_t)row * sb + i] = scales[t * sb + i];
}

cudaError_t launch_read_rows(const DecodeParams& p, int seq, int64_t t0, int64_t t1, int kv, uint8_t* codes,
                             uint8_t* scales, cudaStream_t s) {
  const long n_rows = (long)(t1 - t0);
  if (n_rows <= 0) return cudaSuccess;
  const long warps = n_rows * p.Hkv;
  read_rows_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, s>>>(p, seq, (long)t0, n_rows, kv, codes, scales);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace kvq
