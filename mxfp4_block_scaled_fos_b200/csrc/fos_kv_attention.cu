// fos_kv_attention.cu -- softmax attention over the key/value cache
// (semantics: include/fos.h).
#include <math_constants.h>

#include "fos_device.cuh"
#include "fos_kv.h"

namespace fos {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float block_reduce(float v, float* buf, bool is_max) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float w = __shfl_xor_sync(~0u, v, o);
    v = is_max ? fmaxf(v, w) : v + w;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = buf[0];
  for (int i = 1; i < kThreads / 32; ++i) v = is_max ? fmaxf(v, buf[i]) : v + buf[i];
  return v;
}

// The plain kernel: one CTA for a query and a head, one key for each thread
// at a time, one output value for each of the first dim threads.
__global__ void __launch_bounds__(kThreads) k_kv_attention(const KvAttnArgs a) {
  __shared__ float sq[128], sp[kThreads], buf[kThreads / 32];
  __shared__ long long srow[kThreads];
  __shared__ int sseq;
  const int t = blockIdx.x, hq = blockIdx.y, h = hq / a.group, dim = a.p.dim, tid = threadIdx.x;
  if (tid == 0) {
    int lo = -1, bad = 0;
    for (int b = 0; b < a.batch; ++b) {
      const int x = a.cu_q[b], y = a.cu_q[b + 1];
      if (x < 0 || y < x || y > a.total_q) { bad = 1; continue; }
      if (t >= x && t < y) { lo = b; break; }
    }
    if (bad && a.status) atomicOr(a.status, FOS_STATUS_INDEX);
    sseq = lo;
  }
  __syncthreads();
  const int b = sseq;
  if (b < 0) return;
  const int q0 = a.cu_q[b], n = a.cu_q[b + 1] - q0;
  const long long cap = a.max_pages << a.p.page_shift;
  long long len = a.kv_len[b];
  if (len < 0 || len > cap) {
    len = len < 0 ? 0 : cap;
    if (tid == 0 && a.status) atomicOr(a.status, FOS_STATUS_INDEX);
  }
  long long hi = len, lo = 0;
  if (a.causal) {
    hi = len - n + (t - q0) + 1;
    if (a.window && hi - a.window > 0) lo = hi - a.window;
  }
  if (tid < dim) sq[tid] = __uint_as_float((uint32_t)a.q[(long long)t * a.q_ld + (long long)hq * dim + tid] << 16);
  __syncthreads();
  const float scale = a.scale_log2 * a.p.kst[h];
  float m = -CUDART_INF_F, l = 0.0f, o = 0.0f;
  for (long long j0 = lo; j0 < hi; j0 += kThreads) {
    const long long j = j0 + tid;
    float x = -CUDART_INF_F;
    long long row = -1;
    if (j < hi) {
      const long long page = a.pages[b * a.max_pages + (j >> a.p.page_shift)];
      if (page < 0 || page >= a.p.num_pages) {
        if (a.status) atomicOr(a.status, FOS_STATUS_INDEX);
      } else {
        const long long r = ((long long)h << a.p.page_shift) + (j & ((1 << a.p.page_shift) - 1));
        const uint8_t* c = a.p.kc + page * a.p.codes_stride + r * (dim / 2);
        const uint8_t* s = a.p.ks + page * a.p.scales_stride + r * (dim / 16);
        float dot = 0.0f;
        for (int k = 0; k < dim / 8; ++k) {
          uint32_t w[4];
          e2m1x8_to_h2(reinterpret_cast<const uint32_t*>(c)[k], w);
          float part = 0.0f;
          for (int i = 0; i < 4; ++i)
            part = __fmaf_rn(h_hi(w[i]), sq[8 * k + 2 * i + 1], __fmaf_rn(h_lo(w[i]), sq[8 * k + 2 * i], part));
          dot = __fmaf_rn(part, e4m3_to_f32(s[k >> 1]), dot);
        }
        x = dot * scale;
        row = page;
      }
    }
    const float top = fmaxf(m, block_reduce(x, buf, true));
    const float ref = top == -CUDART_INF_F ? 0.0f : top;
    const float p = row < 0 ? 0.0f : exp2f(x - ref), keep = exp2f(m - ref);
    sp[tid] = p;
    srow[tid] = row;
    l = l * keep + block_reduce(p, buf, false);
    m = top;
    o *= keep;
    if (tid < dim)
      for (int i = 0; i < kThreads && j0 + i < hi; ++i) {
        if (srow[i] < 0) continue;
        const long long r = ((long long)h << a.p.page_shift) + ((j0 + i) & ((1 << a.p.page_shift) - 1));
        const uint8_t c = (a.p.vc + srow[i] * a.p.codes_stride + r * (dim / 2))[tid >> 1];
        const float s = e4m3_to_f32((a.p.vs + srow[i] * a.p.scales_stride + r * (dim / 16))[tid >> 4]);
        o = __fmaf_rn(sp[i], h_lo(e2m1x2_to_h2((tid & 1) ? c >> 4 : c & 15)) * s, o);
      }
  }
  if (tid < dim) {
    const float y = l == 0.0f ? 0.0f : o / l * a.p.vst[h];
    a.out[(long long)t * a.out_ld + (long long)hq * dim + tid] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
  }
  if (tid == 0 && a.lse)
    a.lse[(long long)t * a.q_heads + hq] = l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_kv_attention(const KvAttnArgs& a, cudaStream_t st) {
  k_kv_attention<<<dim3(a.total_q, a.q_heads), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace fos
