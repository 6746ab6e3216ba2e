// fos_kv.cu -- filling and reading the key/value cache (semantics:
// include/fos.h): the position rotation and the 4/6 quantizer of new keys
// and values in one pass, and the cache's dequantizer.
#include "fos_core.cuh"
#include "fos_kv.cuh"

namespace fos {
namespace {

constexpr int kThreads = 128;
constexpr int kAppendWarps = 24;    // of k_kv_append on an SM: 80 registers, 6 warps on each quarter

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
// thread takes two 16-value blocks of one row, with dim/32 neighbouring lanes
// a row.  With halves as pairs (rot a multiple of 32) they are a block of
// first values and the block of their partners rot/2 further on, so that
// every value is loaded and widened once and an angle serves two of them;
// otherwise they are neighbours.  Products are fma(x, c, -0) in pairs: rounded
// by themselves (see the f32x2 helpers), two to an instruction.  A CTA has the
// same rows (every gridDim.y-th) of token after token and loads the next
// token's while it works on one.
// Memory-bound for long prompts, where the queries are most of the bytes:
// 16384 tokens of 32 + 8 + 8 heads of 128 appended (363 MB) 75 us in calls that
// follow one another, 0.75 of the copy bandwidth, and 80 with nothing in L2 (86
// with interleaved pairs); 95 with a token for each CTA (8192 of 64 + 8 + 8 heads
// 73 and 77, 16384 of 8 + 8 + 8 heads of 64 46 and 42); one block a thread, whose
// partners are loaded again, took 35 more.  Launch and latency for a decoding
// step.
// WIDE: all rows 32-byte aligned, one load and one store a block.
template <bool F46, bool INTER, bool WIDE>
__global__ void __launch_bounds__(256, 3) k_kv_append(const KvAppendArgs a) {
  const int lanes = a.p.dim >> 5;
  const int r = threadIdx.x / lanes * gridDim.y + blockIdx.y, p = threadIdx.x & (lanes - 1);
  const bool teller = threadIdx.x == 0 && blockIdx.y == 0;
  const int kind = r < a.q_heads ? 0 : r < a.q_heads + a.p.heads ? 1 : r < a.q_heads + 2 * a.p.heads ? 2 : 3;
  const int h = kind == 0 ? r : kind == 1 ? r - a.q_heads : r - a.q_heads - a.p.heads;
  const int half = a.rot >> 1;
  const bool turned = a.table && kind < 2 && 32 * p < a.rot;
  const int d0 = !INTER && 32 * p < a.rot ? 16 * p : 32 * p;             // the blocks' first values
  const int d1 = !INTER && 32 * p < a.rot ? d0 + half : d0 + 16;
  const uint16_t* base = (kind == 0 ? a.q : kind == 1 ? a.k : a.v) + h * a.p.dim;
  const long long ld = kind == 0 ? a.q_ld : kind == 1 ? a.k_ld : a.v_ld;
  uint4 w[2][2], w_next[2][2];
  long long slot_next = 0;
  int pos_next = 0;
  auto fetch = [&](int t) {      // what token t brings
    if (kind < 3) {
      load32<WIDE>(base + t * ld + d0, w_next[0]);
      load32<WIDE>(base + t * ld + d1, w_next[1]);
    }
    slot_next = __ldg(reinterpret_cast<const long long*>(a.slots) + t);
    if (a.table) pos_next = __ldg(a.positions + t);
  };
  fetch(blockIdx.x);
#pragma unroll 1
  for (int t = blockIdx.x; t < a.tokens; t += gridDim.x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i >> 1][i & 1] = w_next[i >> 1][i & 1];
    const long long slot = slot_next;
    const int pos = pos_next;
    if (t + (int)gridDim.x < a.tokens) fetch(t + gridDim.x);
    const long long page = slot >> a.p.page_shift;
    bool write = slot >= 0, turn_ok = true;
    if (write && page >= a.p.num_pages) {
      write = false;
      if (teller && a.status) atomicOr(a.status, FOS_STATUS_INDEX);
    }
    if (a.table) {
      if (pos < 0 || pos >= a.max_positions) {
        if (teller && a.status) atomicOr(a.status, FOS_STATUS_INDEX);
        write = turn_ok = false;
      } else if (turned) {
        const float* row = a.table + (long long)pos * a.rot;
        const float2 nz = make_float2(a.neg_zero, a.neg_zero);
        uint32_t(&W)[2][8] = reinterpret_cast<uint32_t(&)[2][8]>(w);
#pragma unroll
        for (int q = 0; q < 4; ++q) {       // four pairs of each of two words of either block (INTER: of one word)
          const int i = INTER ? (d0 >> 1) + 4 * q : d0 + 4 * q;
          if (INTER && 2 * i >= a.rot) continue;
          const float4 c = __ldg(reinterpret_cast<const float4*>(row + i));
          const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + i));
#pragma unroll
          for (int e = 0; e < 2; ++e) {     // the angles of pairs i + 2 e, i + 2 e + 1
            const float2 c2 = e ? make_float2(c.z, c.w) : make_float2(c.x, c.y);
            const float2 s2 = e ? make_float2(s.z, s.w) : make_float2(s.x, s.y);
            // INTER: pair i is word i of the thread's 16
            uint32_t& wa = INTER ? W[q >> 1][4 * (q & 1) + 2 * e] : W[0][2 * q + e];
            uint32_t& wb = INTER ? W[q >> 1][4 * (q & 1) + 2 * e + 1] : W[1][2 * q + e];
            const float2 u = INTER ? make_float2(bf_lo(wa), bf_lo(wb)) : make_float2(bf_lo(wa), bf_hi(wa));
            const float2 v = INTER ? make_float2(bf_hi(wa), bf_hi(wb)) : make_float2(bf_lo(wb), bf_hi(wb));
            const float2 a2 = sub2(fma2(u, c2, nz), fma2(v, s2, nz));
            const float2 b2 = add2(fma2(v, c2, nz), fma2(u, s2, nz));
            wa = INTER ? pack_bf16(a2.x, b2.x) : pack_bf16(a2.x, a2.y);
            wb = INTER ? pack_bf16(a2.y, b2.y) : pack_bf16(b2.x, b2.y);
          }
        }
      }
    }
    if (kind == 0 && turn_ok) {
      uint16_t* dst = a.q_out + (long long)t * a.q_out_ld + h * a.p.dim;
      store32<WIDE>(dst + d0, w[0]);
      store32<WIDE>(dst + d1, w[1]);
    } else if ((kind == 1 || kind == 2) && write) {
      const TScale ts = make_tscale(__ldg((kind == 1 ? a.p.kst : a.p.vst) + h));
      const long long row = ((long long)h << a.p.page_shift) + (slot & ((1 << a.p.page_shift) - 1));
      uint8_t* codes = (kind == 1 ? a.p.kc : a.p.vc) + page * a.p.codes_stride + row * (a.p.dim >> 1);
      uint8_t* scales = (kind == 1 ? a.p.ks : a.p.vs) + page * a.p.scales_stride + row * (a.p.dim >> 4);
      bool good = true;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int d = b ? d1 : d0;
        uint32_t cw[2], sc;
        good &= quantize_block<F46>(w[b], ts, a.neg_zero, cw, sc);
        *reinterpret_cast<uint2*>(codes + (d >> 1)) = make_uint2(cw[0], cw[1]);
        scales[d >> 4] = (uint8_t)sc;
      }
      if (!good && a.status) atomicOr(a.status, FOS_STATUS_NONFINITE);
    }
  }
}

// The same for halves as pairs whose partners are not whole blocks apart (rot
// not a multiple of 32): a thread has one block, and the other value of each
// pair, rot/2 further on or back, is loaded again from a row that it shares
// with its lanes of the warp; 8 values at a time (rot/2 is a multiple of 8).
// A CTA for each token and no loads ahead: 16384 tokens of 32 + 8 + 8 heads of
// 128, 48 values rotated, 117 us with nothing in L2, where k_kv_append takes 86
// for the same rotation of interleaved pairs; of 8 + 8 + 8 heads of 64, 16
// rotated, 47 and 39.
template <bool F46, bool WIDE>
__global__ void __launch_bounds__(kThreads, 6) k_kv_append_odd(const KvAppendArgs a) {
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
    if (a.table && kind < 2) {
#pragma unroll
      for (int hb = 0; hb < 2; ++hb) {
        const int d = d0 + 8 * hb;
        if (d >= a.rot) continue;
        part[hb] = d < half ? half : -half;
        y[hb] = *reinterpret_cast<const uint4*>(src + 8 * hb + part[hb]);
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
// Memory-bound, 2.56 bytes a value: 131072 tokens of 8 heads of 128 (689 MB)
// 114 us, 0.94 of the copy bandwidth.
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
  const int rows = a.q_heads + 2 * a.p.heads;
  const bool wide = aligned32(a.k, a.k_ld) && aligned32(a.v, a.v_ld) &&
                    (!a.q || (aligned32(a.q, a.q_ld) && aligned32(a.q_out, a.q_out_ld)));
  if (!INTER && a.rot % 32) {
    const int lanes = kThreads / (a.p.dim / 16);
    const dim3 grid(a.tokens, (rows + lanes - 1) / lanes);
    if (wide) k_kv_append_odd<F46, true><<<grid, kThreads, 0, st>>>(a);
    else      k_kv_append_odd<F46, false><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  // a token's rows in CTAs of equal size, up to 256 threads; as many CTAs as fit
  const int all = rows * (a.p.dim / 32), ctas = (all + 255) / 256;
  const int threads = ((all + ctas - 1) / ctas + 31) / 32 * 32;
  static KvDevices devices;
  int sms = 0;
  const cudaError_t e = devices.get((const void*)k_kv_append<F46, INTER, true>, 0, &sms);
  if (e != cudaSuccess) return e;
  const int fit = sms * (kAppendWarps * 32 / threads), most = fit > ctas ? fit / ctas : 1;
  const dim3 grid(a.tokens < most ? a.tokens : most, ctas);
  if (wide) k_kv_append<F46, INTER, true><<<grid, threads, 0, st>>>(a);
  else      k_kv_append<F46, INTER, false><<<grid, threads, 0, st>>>(a);
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
