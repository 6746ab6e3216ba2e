// fos_kv.cuh -- device code that the attention kernels over the key/value
// cache share.
#pragma once

#include "fos_device.cuh"
#include "fos_kv.h"

namespace fos {

// Weights are 2^(x - m + kLift) with m a row's running maximum, raised when a
// score passes it by kSlack: at most 2^14, and rounded to f16 (2^-11
// relative down to 2^-20 of the largest, 2^-31 of it absolute below).
constexpr float kLift = 6.0f, kSlack = 8.0f;   // log2

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The 8 codes of a word -> four f16x2 (value 2j in the low half of h[j]).
// The word is split in one move and its bytes converted as they are: 72 codes a
// cycle and SM, 47 with a byte permute for each (e2m1x8_to_h2).  That one keeps
// bytes zero-extended because split ones were once measured wrong; these are
// compared for every word (tests/test_gpu_exhaustive.py) and, in the kernels,
// for every byte in every place (tests/test_gpu_kv.py).
__device__ __forceinline__ void codes_h2x4(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// two E4M3 bytes -> f16x2
__device__ __forceinline__ uint32_t scales_h2(uint32_t w16) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)w16));
  return h;
}

__device__ __forceinline__ int query_hi(const KvAttnArgs& a, int n, int len, int i) {
  return a.causal ? max(0, len - n + i + 1) : len;
}

__device__ __forceinline__ int query_lo(const KvAttnArgs& a, int hi) {
  return a.window && hi > a.window ? (int)(hi - a.window) : 0;
}

// Queries and keys of sequence b, clamped to what the arguments allow (`bad`
// if they had to be).  False if its offsets descend or leave the queries: it
// has none then.
__device__ __forceinline__ bool lengths_of(const KvAttnArgs& a, int b, int& q0, int& n, int& len, bool& bad) {
  const int x = a.cu_q[b], y = a.cu_q[b + 1];
  const long long cap = a.max_pages << a.p.page_shift;
  const int m = a.kv_len[b];
  const bool ordered = x >= 0 && y >= x && y <= a.total_q;
  bad = !ordered || m < 0 || m > cap;
  q0 = x;
  n = ordered ? y - x : 0;
  len = max(0, (int)min((long long)m, cap));
  return ordered;
}

// Whether the sequences of a batch have more queries together than there are:
// then none is answered, for all that counts rows and items over them (in 32
// bits, for grids and loops) relies on total_q.  Only offsets that descend
// somewhere can do it, so the block asks only if a sequence is not in order.
// `mine`: this thread's sequences; sums: a place for each warp.
__device__ __forceinline__ bool too_many(const KvAttnArgs& a, long long mine, long long* sums) {
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(~0u, mine, o);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = mine;
  __syncthreads();
  long long all = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) all += sums[w];
  return all > a.total_q;
}

// The scaling of a query row to below 2^15 by a power of two, for its f16
// operand: exact for values down to 2^-31 of the row's largest, smaller ones
// off by 2^-39 of it at most (half of f16's last subnormal bit).  up1 * up2
// scales the values, down1 * down2 the scores (two factors, so that none
// leaves the normal range); a row with NaN or Inf is not finite.
struct RowScale {
  float up1, up2, down1, down2;
  bool finite;
};

__device__ __forceinline__ RowScale row_scale(uint32_t top) {   // bits of the largest |value|
  RowScale s;
  s.finite = top < 0x7f800000u;
  const int e = top == 0 || !s.finite ? 14 : max((int)(top >> 23), 1) - 127;
  const int up = 14 - e, u1 = up / 2, u2 = up - u1;
  s.up1 = __uint_as_float((uint32_t)(127 + u1) << 23);
  s.up2 = __uint_as_float((uint32_t)(127 + u2) << 23);
  s.down1 = __uint_as_float((uint32_t)(127 - u1) << 23);
  s.down2 = __uint_as_float((uint32_t)(127 - u2) << 23);
  return s;
}

}  // namespace fos
