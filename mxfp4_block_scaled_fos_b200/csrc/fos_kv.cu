// fos_kv.cu -- filling and reading the key/value cache (semantics:
// include/fos.h): the position rotation and the 4/6 quantizer of new keys
// and values in one pass, and the cache's dequantizer.
#include "fos_core.cuh"
#include "fos_kv.h"

namespace fos {
namespace {

constexpr int kThreads = 128;

// One 16-value block (8 bf16x2 words) -> codes and scale byte by the
// quantizer's rule with S_t = ts.St.  Pools have one S_t for each head, so
// the two scales that a block tries are formed here instead of being looked
// up in a table of all 128.  Returns false for NaN/Inf.
template <bool F46>
__device__ __forceinline__ bool quantize_block(const uint4 (&w)[2], const TScale& ts, float nz, uint32_t (&codes)[2],
                                               uint32_t& sc) {
  const uint32_t m = amax_bits_bf16(w);
  const uint32_t W[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
  float2 P[8];
  unpack_split(W, P);
  uint32_t s6, s4;
  cand_scales<F46>(__uint_as_float(m), ts, s6, s4);
  const float E6 = __fmul_rn(e4m3_to_f32(s6), ts.St);
  const float i6 = (E6 == 0.0f) ? 0.0f : fminf(__frcp_rn(E6), kFltMax);
  const Cand1 c6 = candidate1<F46>(P, i6, -E6, nz);
  codes[0] = c6.c[0];
  codes[1] = c6.c[1];
  sc = s6;
  if (F46) {
    const float E4 = __fmul_rn(e4m3_to_f32(s4), ts.St);
    const float i4 = (E4 == 0.0f) ? 0.0f : fminf(__frcp_rn(E4), kFltMax);
    const Cand1 c4 = candidate1<true>(P, i4, -E4, nz);
    if (c4.err < c6.err) { codes[0] = c4.c[0]; codes[1] = c4.c[1]; sc = s4; }
  }
  return m < 0x7f800000u;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// x c + y s with both products rounded before the sum (s carries the sign).
__device__ __forceinline__ float turn(float x, float c, float y, float s) {
  return __fadd_rn(__fmul_rn(x, c), __fmul_rn(y, s));
}

__device__ __forceinline__ void load8(const float* p, float* r) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
  r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
}

// Append.  A token's rows are its query heads, key heads and value heads; a
// group of dim/16 neighbouring lanes takes one row, a 16-value block each,
// and steps through rows of the same token, so that the angles of a block's
// positions (the same for all heads) stay in registers.  With halves as
// pairs the other value of each pair is in the block rot/2 further on, which
// another lane of the group holds too: it is loaded again, from L1.  One
// CTA takes one token and gridDim.y splits its rows when tokens are few.
// Memory-bound for long prompts, latency for a decoding step.
template <bool F46, bool INTER>
__global__ void __launch_bounds__(kThreads) k_kv_append(const KvAppendArgs a) {
  const int nb = a.p.dim >> 4;
  const int bi = threadIdx.x & (nb - 1), rl = threadIdx.x / nb, rstep = (kThreads / nb) * gridDim.y;
  const int t = blockIdx.x;
  const int rows = a.q_heads + 2 * a.p.heads;
  const long long slot = a.slots[t];
  const long long page = slot >> a.p.page_shift;
  bool write = slot >= 0, turn_q = true;
  if (write && page >= a.p.num_pages) {
    write = false;
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, FOS_STATUS_INDEX);
  }
  // the block's angles: INTER has a pair in (2i, 2i + 1), 8 pairs a block;
  // otherwise value d is turned by pair d mod rot/2, with the partner rot/2
  // away, the same way for 8 values at a time (rot/2 is a multiple of 8)
  float c[INTER ? 8 : 16], s[INTER ? 8 : 16];
  int part[2] = {0, 0};                    // distance of each half block's partners; 0: not turned
  const int d0 = bi * 16, half = a.rot >> 1;
  if (a.table) {
    const int pos = a.positions[t];
    if (pos < 0 || pos >= a.max_positions) {
      if (threadIdx.x == 0 && a.status) atomicOr(a.status, FOS_STATUS_INDEX);
      write = turn_q = false;
    } else {
      const float* row = a.table + (long long)pos * a.rot;
      if (INTER) {
        if (d0 < a.rot) {
          part[0] = part[1] = 1;
          load8(row + (d0 >> 1), c);
          load8(row + half + (d0 >> 1), s);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int d = d0 + 8 * h;
          if (d >= a.rot) continue;
          const bool first = d < half;
          const int i = first ? d : d - half;
          part[h] = first ? half : -half;
          load8(row + i, c + (INTER ? 0 : 8 * h));
          load8(row + half + i, s + (INTER ? 0 : 8 * h));
          if (first)
#pragma unroll
            for (int k = 0; k < 8; ++k) s[(INTER ? 0 : 8 * h) + k] = -s[(INTER ? 0 : 8 * h) + k];
        }
      }
    }
  }
  const long long code_at = page * a.p.codes_stride, scale_at = page * a.p.scales_stride;
  const int off = (int)(slot & ((1 << a.p.page_shift) - 1));
  bool bad = false;
  // every lane of a warp runs the same number of steps: q_out may be q, so
  // the stores of a row wait for the loads of its partners
  for (int r0 = (rl & ~(32 / nb - 1)) + (kThreads / nb) * blockIdx.y; r0 < rows; r0 += rstep) {
    const int r = r0 + (rl & (32 / nb - 1));
    const int kind = r < a.q_heads ? 0 : r < a.q_heads + a.p.heads ? 1 : 2;
    const int h = kind == 0 ? r : kind == 1 ? r - a.q_heads : r - a.q_heads - a.p.heads;
    const bool live = r < rows && (kind == 0 ? turn_q : write);
    uint4 w[2];
    if (live) {
      const uint16_t* src = kind == 0 ? a.q + (long long)t * a.q_ld
                                      : kind == 1 ? a.k + (long long)t * a.k_ld : a.v + (long long)t * a.v_ld;
      src += (long long)h * a.p.dim + d0;
      w[0] = *reinterpret_cast<const uint4*>(src);
      w[1] = *reinterpret_cast<const uint4*>(src + 8);
      if (kind < 2 && (part[0] || part[1])) {
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
          if (!part[hb]) continue;
          uint32_t x[4] = {w[hb].x, w[hb].y, w[hb].z, w[hb].w};
          if (INTER) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float u = bf_lo(x[k]), v = bf_hi(x[k]);
              x[k] = pack_bf16(turn(u, c[4 * hb + k], v, -s[4 * hb + k]), turn(v, c[4 * hb + k], u, s[4 * hb + k]));
            }
          } else {
            const uint4 p = *reinterpret_cast<const uint4*>(src + 8 * hb + part[hb]);
            const uint32_t y[4] = {p.x, p.y, p.z, p.w};
            const float *ch = c + (INTER ? 0 : 8 * hb), *sh = s + (INTER ? 0 : 8 * hb);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[k] = pack_bf16(turn(bf_lo(x[k]), ch[2 * k], bf_lo(y[k]), sh[2 * k]),
                               turn(bf_hi(x[k]), ch[2 * k + 1], bf_hi(y[k]), sh[2 * k + 1]));
          }
          w[hb] = make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
    }
    __syncwarp();
    if (!live) continue;
    if (kind == 0) {
      uint16_t* dst = a.q_out + (long long)t * a.q_out_ld + (long long)h * a.p.dim + d0;
      *reinterpret_cast<uint4*>(dst) = w[0];
      *reinterpret_cast<uint4*>(dst + 8) = w[1];
    } else {
      const TScale ts = make_tscale(__ldg((kind == 1 ? a.p.kst : a.p.vst) + h));
      uint32_t codes[2], sc;
      bad |= !quantize_block<F46>(w, ts, a.neg_zero, codes, sc);
      const long long row = ((long long)h << a.p.page_shift) + off;
      *reinterpret_cast<uint2*>((kind == 1 ? a.p.kc : a.p.vc) + code_at + row * (a.p.dim >> 1) + 8 * bi) =
          make_uint2(codes[0], codes[1]);
      ((kind == 1 ? a.p.ks : a.p.vs) + scale_at)[row * nb + bi] = (uint8_t)sc;
    }
  }
  if (bad && a.status) atomicOr(a.status, FOS_STATUS_NONFINITE);
}

// 16 values of a pool -> bf16, two 16-byte stores.
__device__ __forceinline__ void read_block(const uint8_t* codes, const uint8_t* scale, float St, bool live,
                                           uint16_t* y) {
  uint32_t o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
  if (live) {
    const uint2 cw = __ldg(reinterpret_cast<const uint2*>(codes));
    const float s = e4m3_to_f32(__ldg(scale));
    uint32_t h[8];
    e2m1x8_to_h2(cw.x, h);
    e2m1x8_to_h2(cw.y, h + 4);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 q = mul2(mul2(make_float2(h_lo(h[k]), h_hi(h[k])), make_float2(s, s)), make_float2(St, St));
      o[k] = pack_bf16(q.x, q.y);
    }
  }
  __stcs(reinterpret_cast<uint4*>(y), make_uint4(o[0], o[1], o[2], o[3]));
  __stcs(reinterpret_cast<uint4*>(y) + 1, make_uint4(o[4], o[5], o[6], o[7]));
}

// Read.  One thread for a block of a token's head, keys and values both;
// neighbouring threads read neighbouring codes and write whole lines.
// Memory-bound: 2.56 bytes a value.
__global__ void __launch_bounds__(256) k_kv_read(const KvReadArgs a, int row_blocks, long long n) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const long long t = i / row_blocks;
  const int r = (int)(i - t * row_blocks), nb = a.p.dim >> 4;
  const int h = r / nb, bi = r & (nb - 1);
  const long long slot = __ldg(reinterpret_cast<const long long*>(a.slots) + t);
  const long long page = slot >> a.p.page_shift;
  const bool live = slot >= 0 && page < a.p.num_pages;
  if (slot >= 0 && !live && r == 0 && a.status) atomicOr(a.status, FOS_STATUS_INDEX);
  const long long row = ((long long)h << a.p.page_shift) + (slot & ((1 << a.p.page_shift) - 1));
  const long long c = page * a.p.codes_stride + row * (a.p.dim >> 1) + 8 * bi;
  const long long s = page * a.p.scales_stride + row * nb + bi;
  read_block(a.p.kc + c, a.p.ks + s, live ? __ldg(a.p.kst + h) : 0.0f, live, a.k + i * 16);
  read_block(a.p.vc + c, a.p.vs + s, live ? __ldg(a.p.vst + h) : 0.0f, live, a.v + i * 16);
}

template <bool F46, bool INTER>
cudaError_t append(const KvAppendArgs& a, cudaStream_t st) {
  const int lanes = kThreads / (a.p.dim / 16), rows = a.q_heads + 2 * a.p.heads;
  // one step for each lane while that leaves SMs without work
  const int steps = (rows + lanes - 1) / lanes;
  const int split = a.tokens >= 148 * 8 ? 1 : steps;
  k_kv_append<F46, INTER><<<dim3(a.tokens, split), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, int fmt, bool interleaved, cudaStream_t st) {
  if (fmt == FOS_FMT_NVFP4_46) return interleaved ? append<true, true>(a, st) : append<true, false>(a, st);
  return interleaved ? append<false, true>(a, st) : append<false, false>(a, st);
}

cudaError_t launch_kv_read(const KvReadArgs& a, cudaStream_t st) {
  const int row_blocks = a.p.heads * (a.p.dim / 16);
  const long long n = (long long)a.tokens * row_blocks, grid = (n + 255) / 256;
  if (grid > 0x7fffffffll) return cudaErrorNotSupported;
  k_kv_read<<<(unsigned)grid, 256, 0, st>>>(a, row_blocks, n);
  return cudaGetLastError();
}

}  // namespace fos
