// fos_kv.cu -- filling and reading the key/value cache (semantics:
// include/fos.h): the position rotation and the 4/6 quantizer of new keys
// and values in one pass, and the cache's dequantizer.
#include "fos_core.cuh"
#include "fos_kv.cuh"

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

// 32 bytes to global memory: one store where they are 32-byte aligned.
template <bool WIDE>
__device__ __forceinline__ void store32(uint16_t* p, const uint4 (&w)[2]) {
  if (WIDE) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(w[0].x), "r"(w[0].y), "r"(w[0].z), "r"(w[0].w), "r"(w[1].x), "r"(w[1].y),
                    "r"(w[1].z), "r"(w[1].w) : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = w[0];
    reinterpret_cast<uint4*>(p)[1] = w[1];
  }
}

template <bool WIDE>
__device__ __forceinline__ void load32(const uint16_t* p, uint4 (&w)[2]) {
  if (WIDE) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0].x), "=r"(w[0].y), "=r"(w[0].z), "=r"(w[0].w), "=r"(w[1].x), "=r"(w[1].y), "=r"(w[1].z),
                   "=r"(w[1].w) : "l"(p) : "memory");
  } else {
    w[0] = reinterpret_cast<const uint4*>(p)[0];
    w[1] = reinterpret_cast<const uint4*>(p)[1];
  }
}

// Append.  A token's rows are its query heads, key heads and value heads; a
// thread takes a 16-value block of one row, dim/16 neighbouring lanes a row.
// With halves as pairs the other value of each pair is rot/2 further on, in a
// block that another lane of the row holds too: it is loaded again, from L1,
// and so are the angles, which the rows of a token share.  (Keeping the
// angles in registers through several rows of a token cost more in occupancy
// than it saved in loads.)  Memory-bound for long prompts, where the queries
// are most of the bytes; launch and latency for a decoding step.
// WIDE: all rows 32-byte aligned, one load and one store a block.
template <bool F46, bool INTER, bool WIDE>
__global__ void __launch_bounds__(kThreads, 6) k_kv_append(const KvAppendArgs a) {
  const int nb = a.p.dim >> 4;
  const int bi = threadIdx.x & (nb - 1);
  const int r = blockIdx.y * (kThreads / nb) + threadIdx.x / nb;
  const int t = blockIdx.x;
  const int kind = r < a.q_heads ? 0 : r < a.q_heads + a.p.heads ? 1 : r < a.q_heads + 2 * a.p.heads ? 2 : 3;
  const int h = kind == 0 ? r : kind == 1 ? r - a.q_heads : r - a.q_heads - a.p.heads;
  const int d0 = bi * 16, half = a.rot >> 1;
  uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)}, y[2];
  int part[2] = {0, 0};                    // distance of each half block's partners; 0: not turned
  if (kind < 3) {
    const uint16_t* src = kind == 0 ? a.q + (long long)t * a.q_ld
                                    : kind == 1 ? a.k + (long long)t * a.k_ld : a.v + (long long)t * a.v_ld;
    src += (long long)h * a.p.dim + d0;
    load32<WIDE>(src, w);
    // value d is turned with d + rot/2 or d - rot/2, the same way for 8 values
    // at a time (rot/2 is a multiple of 8); INTER: with its neighbour
    if (a.table && kind < 2) {
#pragma unroll
      for (int hb = 0; hb < 2; ++hb) {
        const int d = d0 + 8 * hb;
        if (d >= a.rot) continue;
        part[hb] = d < half ? half : -half;
        if (!INTER) y[hb] = *reinterpret_cast<const uint4*>(src + 8 * hb + part[hb]);
      }
    }
  }
  const long long slot = a.slots[t];
  const long long page = slot >> a.p.page_shift;
  bool write = slot >= 0, turn_ok = true;
  if (write && page >= a.p.num_pages) {
    write = false;
    if (threadIdx.x == 0 && blockIdx.y == 0 && a.status) atomicOr(a.status, FOS_STATUS_INDEX);
  }
  if (a.table) {
    const int pos = a.positions[t];
    if (pos < 0 || pos >= a.max_positions) {
      if (threadIdx.x == 0 && blockIdx.y == 0 && a.status) atomicOr(a.status, FOS_STATUS_INDEX);
      write = turn_ok = false;
    } else {
      const float* row = a.table + (long long)pos * a.rot;
#pragma unroll
      for (int hb = 0; hb < 2; ++hb) {
        if (!part[hb]) continue;
        uint32_t x[4] = {w[hb].x, w[hb].y, w[hb].z, w[hb].w};
        const int d = d0 + 8 * hb;
        if (INTER) {
          const float4 c = __ldg(reinterpret_cast<const float4*>(row + (d >> 1)));
          const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + (d >> 1)));
          const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float u = bf_lo(x[k]), v = bf_hi(x[k]);
            x[k] = pack_bf16(turn(u, cc[k], v, -ss[k]), turn(v, cc[k], u, ss[k]));
          }
        } else {
          const bool first = part[hb] > 0;
          float c[8], s[8];
          load8(row + (first ? d : d - half), c);
          load8(row + half + (first ? d : d - half), s);
          const uint32_t z[4] = {y[hb].x, y[hb].y, y[hb].z, y[hb].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float s0 = first ? -s[2 * k] : s[2 * k], s1 = first ? -s[2 * k + 1] : s[2 * k + 1];
            x[k] = pack_bf16(turn(bf_lo(x[k]), c[2 * k], bf_lo(z[k]), s0),
                             turn(bf_hi(x[k]), c[2 * k + 1], bf_hi(z[k]), s1));
          }
        }
        w[hb] = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
  }
  __syncwarp();   // q_out may be q: a row is written after its lanes have read their partners in it
  if (kind == 0 && turn_ok) {
    store32<WIDE>(a.q_out + (long long)t * a.q_out_ld + (long long)h * a.p.dim + d0, w);
  } else if ((kind == 1 || kind == 2) && write) {
    const TScale ts = make_tscale(__ldg((kind == 1 ? a.p.kst : a.p.vst) + h));
    uint32_t codes[2], sc;
    if (!quantize_block<F46>(w, ts, a.neg_zero, codes, sc) && a.status) atomicOr(a.status, FOS_STATUS_NONFINITE);
    const long long row = ((long long)h << a.p.page_shift) + (slot & ((1 << a.p.page_shift) - 1));
    *reinterpret_cast<uint2*>((kind == 1 ? a.p.kc : a.p.vc) + page * a.p.codes_stride + row * (a.p.dim >> 1) +
                              8 * bi) = make_uint2(codes[0], codes[1]);
    ((kind == 1 ? a.p.ks : a.p.vs) + page * a.p.scales_stride)[row * nb + bi] = (uint8_t)sc;
  }
}

// 16 values of a pool -> bf16.
template <bool WIDE>
__device__ __forceinline__ void read_block(uint2 cw, uint32_t scale, float St, uint16_t* y) {
  const float s = e4m3_to_f32(scale);
  uint32_t o[8], h[4];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    codes_h2x4(b ? cw.y : cw.x, h);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 q = mul2(mul2(make_float2(h_lo(h[k]), h_hi(h[k])), make_float2(s, s)), make_float2(St, St));
      o[4 * b + k] = pack_bf16(q.x, q.y);
    }
  }
  const uint4 w[2] = {make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7])};
  store32<WIDE>(y, w);
}

// Read.  One thread for a block of a token's head, keys and values both;
// neighbouring threads read neighbouring codes and write whole lines.
// Memory-bound: 2.56 bytes a value.
template <bool WIDE>
__global__ void __launch_bounds__(256) k_kv_read(const KvReadArgs a, FastDiv row_blocks, uint32_t n) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= n) return;
  const uint32_t t = fdiv(i, row_blocks);
  const uint32_t r = i - t * row_blocks.d, nb = a.p.dim >> 4;
  const uint32_t h = r >> (nb == 8 ? 3 : 2), bi = r & (nb - 1);
  const long long slot = __ldg(reinterpret_cast<const long long*>(a.slots) + a.token0 + t);
  const long long page = slot >> a.p.page_shift;
  const bool live = slot >= 0 && page < a.p.num_pages;
  if (slot >= 0 && !live && r == 0 && a.status) atomicOr(a.status, FOS_STATUS_INDEX);
  const uint32_t row = (h << a.p.page_shift) + ((uint32_t)slot & ((1u << a.p.page_shift) - 1));
  uint2 kw = make_uint2(0u, 0u), vw = kw;
  uint32_t ks = 0, vs = 0;
  float kt = 0.0f, vt = 0.0f;
  if (live) {
    const long long c = page * a.p.codes_stride + row * (a.p.dim >> 1) + 8 * bi;
    const long long s = page * a.p.scales_stride + row * nb + bi;
    kw = __ldg(reinterpret_cast<const uint2*>(a.p.kc + c));
    vw = __ldg(reinterpret_cast<const uint2*>(a.p.vc + c));
    ks = __ldg(a.p.ks + s);
    vs = __ldg(a.p.vs + s);
    kt = __ldg(a.p.kst + h);
    vt = __ldg(a.p.vst + h);
  }
  const long long at = ((long long)a.token0 * row_blocks.d + i) * 16;
  read_block<WIDE>(kw, ks, kt, a.k + at);
  read_block<WIDE>(vw, vs, vt, a.v + at);
}

inline bool aligned32(const void* p, long long ld) { return (uintptr_t)p % 32 == 0 && ld % 16 == 0; }

template <bool F46, bool INTER>
cudaError_t append(const KvAppendArgs& a, cudaStream_t st) {
  const int lanes = kThreads / (a.p.dim / 16), rows = a.q_heads + 2 * a.p.heads;
  const dim3 grid(a.tokens, (rows + lanes - 1) / lanes);
  const bool wide = aligned32(a.k, a.k_ld) && aligned32(a.v, a.v_ld) &&
                    (!a.q || (aligned32(a.q, a.q_ld) && aligned32(a.q_out, a.q_out_ld)));
  if (wide) k_kv_append<F46, INTER, true><<<grid, kThreads, 0, st>>>(a);
  else      k_kv_append<F46, INTER, false><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, int fmt, bool interleaved, cudaStream_t st) {
  if (fmt == FOS_FMT_NVFP4_46) return interleaved ? append<true, true>(a, st) : append<true, false>(a, st);
  return interleaved ? append<false, true>(a, st) : append<false, false>(a, st);
}

cudaError_t launch_kv_read(const KvReadArgs& args, cudaStream_t st) {
  KvReadArgs a = args;
  const int row_blocks = a.p.heads * (a.p.dim / 16);
  const FastDiv div = make_fastdiv((uint32_t)row_blocks);
  const bool wide = aligned32(a.k, 0) && aligned32(a.v, 0);
  // 32-bit block indices below 2^31 for one launch
  const int most = 0x40000000 / row_blocks;
  for (int left = a.tokens; left > 0; left -= most) {
    const uint32_t n = (uint32_t)(left < most ? left : most) * (uint32_t)row_blocks;
    if (wide) k_kv_read<true><<<(n + 255) / 256, 256, 0, st>>>(a, div, n);
    else      k_kv_read<false><<<(n + 255) / 256, 256, 0, st>>>(a, div, n);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    a.token0 += most;
  }
  return cudaSuccess;
}

}  // namespace fos
