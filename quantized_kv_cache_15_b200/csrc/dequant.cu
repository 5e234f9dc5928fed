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
// projection: the Hadamard stages inside a block need no shuffles and a block's codes come
// in a few wide loads (8192 rows of 8 heads, K and V: 60 us with a warp a row, 15 us so;
// the reads and writes alone take 12 at the measured copy rate).  Neighbouring quads take
// neighbouring rows of one (head, K|V).  Every value goes through the same correctly
// rounded operations as above.
__global__ void __launch_bounds__(256) dequant_quad_kernel(const __grid_constant__ DecodeParams p, int seq, int len,
                                                           long t0, int n_rows, float* k_out, float* v_out) {
  const int row = (blockIdx.x * 256 + threadIdx.x) >> 2, q = threadIdx.x & 3;
  const int head = blockIdx.y >> 1, kv = blockIdx.y & 1;
  float* out = kv ? v_out : k_out;
  if (row >= n_rows || !out) return;                     // whole quads
  const long pos = t0 + row;
  const int T = p.T;
  const int nq = len > T ? len - T : 0;
  const HeadInfo& h = p.heads[head];
  float v[32];
  if (pos >= nq) {
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
    if (pid < 0) { if (q == 0) atomicOr(p.err, ERR_NO_PAGE); return; }
    const uint8_t* region = p.pool + (size_t)pid * p.page_bytes + h.off;
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
      default: return;
    }
    if (codec != KVQ_F16 && p.rot != KVQ_ROT_NONE) {
      fwht_quad(v);
      if (const float* s = kv ? p.s_v : p.s_k) {
        const float4* s4 = reinterpret_cast<const float4*>(s + (size_t)head * D) + 8 * q;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float4 m = s4[c];
          v[4 * c] *= m.x; v[4 * c + 1] *= m.y; v[4 * c + 2] *= m.z; v[4 * c + 3] *= m.w;
        }
      }
    }
  }
  float* dst = out + ((size_t)row * p.Hkv + head) * D + 32 * q;
  if ((uintptr_t)out % 32 == 0) {
#pragma unroll
    for (int c = 0; c < 4; ++c) store8(dst + 8 * c, v + 8 * c);
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) *reinterpret_cast<float4*>(dst + 4 * c) = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  }
}

cudaError_t launch_dequantize(const DecodeParams& p, int seq, int64_t t0, int64_t t1, float* k_out, float* v_out,
                              cudaStream_t s) {
  const long n_rows = (long)(t1 - t0);
  if (n_rows <= 0) return cudaSuccess;
  if (p.rot != KVQ_ROT_PROJECTION) {
    dequant_quad_kernel<<<dim3((unsigned)((n_rows + 63) / 64), p.Hkv * 2), 256, 0, s>>>(p, seq, p.len[0], (long)t0,
                                                                                      (int)n_rows, k_out, v_out);
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
