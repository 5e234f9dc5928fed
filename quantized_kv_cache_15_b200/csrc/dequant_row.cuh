// One cached page row in the original basis, by one warp.
//
// Dequantization in the stored basis is exact (each value is one correctly
// rounded operation): _0 code*d, _1 u*d + m, rank (2u - (2^b-1)) * d/2, all of
// which are what fmaf(u, d, off) returns because u*d and off are exact.  The
// inverse transform then applies the staged Hadamard transform (times the
// per-channel variance multiplier) or M_h^T for the projection path.
#pragma once

#include "kvq_internal.h"
#include "quant.cuh"

namespace kvq {

// Row t of a page-head region (K: kv = 0, V: kv = 1) in the stored basis -> values
// 4 lane .. 4 lane + 3 (zeros behind a rank row's r values).
__device__ __forceinline__ void page_row_stored(const uint8_t* region, const HeadInfo& h, int kv, int t, bool bf16,
                                                float x[4]) {
  const int lane = threadIdx.x & 31;
  const int codec = kv ? h.vcodec : h.kcodec;
  const int bits = kv ? h.vbits : h.kbits;
  const int cb = kv ? h.cbV : h.cbK, sb = kv ? h.sbV : h.sbK;
  const uint8_t* codes = kv ? region + PAGE * (h.cbK + h.sbK) : region;
  const uint8_t* scales = codes + PAGE * cb;
  const int n = codec == KVQ_RANK ? h.r : D;
  if (codec == KVQ_F16) {
    const int o = 8 * lane;
    const uint8_t* src = codes + (kv == 0 ? kplane_off(cb, t, o) : t * cb + o);
    const uint2 w = *reinterpret_cast<const uint2*>(src);
    const float2 a = raw2_to_float2(w.x, bf16), b = raw2_to_float2(w.y, bf16);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    return;
  }
  uint32_t u[4];
  if (4 * lane < n) lane_codes(codes, cb, t, kv == 0, bits, n, lane, u);
  else u[0] = u[1] = u[2] = u[3] = 0;
  const int blk = n < 32 ? n : 32;
  const int b = (4 * lane < n) ? (4 * lane) / blk : 0;
  float d, m = 0.f;
  if (codec_is_asym(codec)) {
    __half2 dm = *reinterpret_cast<const __half2*>(scales + t * sb + 4 * b);
    d = __low2float(dm); m = __high2float(dm);
  } else {
    d = __half2float(*reinterpret_cast<const __half*>(scales + t * sb + 2 * b));
  }
  float off;
  if (codec == KVQ_RANK) off = -0.5f * (float)((1 << bits) - 1) * d;
  else if (codec_is_asym(codec)) off = m;
  else off = -(float)(1 << (bits - 1)) * d;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = (4 * lane + i < n) ? fmaf((float)u[i], d, off) : 0.f;
}

// Stored basis -> original basis, the warp's row in place (values 4 lane ..).
// mul: the head's 128 variance multipliers, or null; zs: 128 floats of the warp's
// shared memory (projection path).
__device__ __forceinline__ void row_to_original(int codec, const HeadInfo& h, int rot, const float* mul,
                                                const float* Mtab, float* zs, float x[4]) {
  const int lane = threadIdx.x & 31;
  if (codec == KVQ_F16) return;
  if (codec == KVQ_RANK) {
    if (rot == KVQ_ROT_PROJECTION) {
      __syncwarp();                                   // the warp's previous row has been read
#pragma unroll
      for (int i = 0; i < 4; ++i) zs[4 * lane + i] = x[i];
      __syncwarp();
      const float* M = Mtab + h.m_off;
      float y[4] = {0.f, 0.f, 0.f, 0.f};
      for (int i = 0; i < h.r; ++i) {
        const float z = zs[i];
        float4 mr = *reinterpret_cast<const float4*>(M + (size_t)i * D + 4 * lane);
        y[0] = fmaf(mr.x, z, y[0]); y[1] = fmaf(mr.y, z, y[1]);
        y[2] = fmaf(mr.z, z, y[2]); y[3] = fmaf(mr.w, z, y[3]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = y[i];
    }
  } else if (rot != KVQ_ROT_NONE) {
    fwht_row(x);
    if (mul) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] *= mul[4 * lane + i];
    }
  }
}

__device__ __forceinline__ void page_row_original(const uint8_t* region, const HeadInfo& h, int kv, int t, int rot,
                                                  bool bf16, const float* mul, const float* Mtab, float* zs,
                                                  float x[4]) {
  page_row_stored(region, h, kv, t, bf16, x);
  row_to_original(kv ? h.vcodec : h.kcodec, h, rot, mul, Mtab, zs, x);
}

}  // namespace kvq
