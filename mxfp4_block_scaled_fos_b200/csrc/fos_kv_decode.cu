// fos_kv_decode.cu -- attention of few queries over the key/value cache
// (semantics: include/fos.h): every byte of the visible cache is read once,
// so the kernel is built to keep HBM busy.
//
// A row is one query of one query head; the rows of a sequence that share a
// key/value head are taken 8 or 16 at a time (a row tile).  An item is (a
// sequence, a row tile, a key/value head); its visible tokens are cut into
// tiles of 128.  All tiles of all items, in order, are dealt to the CTAs in
// equal contiguous shares, whatever the lengths: a CTA finds its share from
// the lengths on the device.  An item that lies in one share is finished
// there; of the others each CTA leaves a partial result (row maxima, sums,
// unnormalised output) in the workspace and k_kv_join adds them in the order
// of the tokens.
//
// Inside a CTA each of 8 warps takes 16 tokens of a tile (a slice), which
// lie in one page, with softmax statistics and a ring of bulk copies of its
// own: no barrier until the end of an item.  The products run on m16n8k16
// with f16 operands and f32 sums:
//   S^T = K Q^T      A = 16 tokens of keys, B = 8 rows of queries
//   O^T += V^T P^T   A = 16 output values, B = the weights of 8 rows
// so that 8 rows fill an MMA and no operand goes through shared memory:
//  - An E2M1 code times its E4M3 scale has 6 significant bits between 2^-10
//    and 2688: exact in f16.  Codes are converted two at a time
//    (cvt f16x2.e2m1x2) and multiplied by their scale.
//  - The order of the head's values along the first product's reduction is
//    free: lane (g, c) takes 16 or 32 consecutive values of tokens g, g + 8.
//  - For V^T a register holds one value of two tokens: nibbles of two
//    tokens' words are zipped into bytes before the conversion.
// The running maximum of a row is raised, and its sums rescaled, only when a
// score passes it by 2^8 (fos_kv.cuh).
#include <math_constants.h>

#include "fos_kv.cuh"

namespace fos {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kSlice = 16, kTile = kSlice * kWarps;   // tokens
constexpr int kStages = 4;
constexpr int kMaxCtas = 320;                         // shares: two CTAs on each of up to 160 SMs
constexpr uint32_t kWaitLimit = 1u << 22;

template <int D, int NT>
struct Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kCodes = kSlice * D / 2, kScales = kSlice * D / 16;
  static constexpr int kStage = 2 * (kCodes + kScales);
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kLdO = D + 4;                                     // floats
  static constexpr int kMerge = kWarps * kRows * kLdO * 4;               // the warps' outputs, over the ring
  static constexpr int kBody = kRing > kMerge ? kRing : kMerge;
  static constexpr int kOffStat = kBody;                                 // m, l [warps][rows]
  static constexpr int kOffBar = kOffStat + 2 * kWarps * kRows * 4;
  static constexpr int kOffPlan = kOffBar + kWarps * kStages * 8;
  static constexpr int kSmem = kOffPlan + 64 + kWarps * 8;
  static constexpr int kPart = kRows * (D + 2);                          // floats of one partial result
};

__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
  for (uint32_t it = 0; it < kWaitLimit; ++it) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    if (done) return true;
  }
  return false;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

// The token of A row r of a slice: lane c's V tokens (rows 2c, 2c + 1,
// 2c + 8, 2c + 9) are c of each group of four, and neighbouring rows differ
// in parity, which spreads both products' shared-memory reads over the banks.
__device__ __forceinline__ int row_token(int r) {
  const int c = (r & 7) >> 1;
  return (r & 8) + ((r & 1) ? 4 + (c ^ 1) : c);
}

// The visible tokens [lo, hi) of row tile rt of a sequence with n queries
// and len keys, and its tiles (at least one: a row without keys is written too).
struct Span {
  int lo, hi, base, tiles;
};

template <int ROWS>
__device__ __forceinline__ Span span_of(const KvAttnArgs& a, int n, int len, int rt) {
  Span s;
  const int first = rt * ROWS / a.group, last = min(n * a.group - 1, rt * ROWS + ROWS - 1) / a.group;
  s.hi = query_hi(a, n, len, last);
  s.lo = query_lo(a, query_hi(a, n, len, first));
  s.base = s.lo & ~(kSlice - 1);
  s.tiles = max(1, (s.hi - s.base + kTile - 1) / kTile);
  return s;
}

template <int ROWS>
__device__ __forceinline__ long long tiles_of(const KvAttnArgs& a, int n, int len) {
  const int nrt = (n * a.group + ROWS - 1) / ROWS;
  long long t = 0;
  for (int rt = 0; rt < nrt; ++rt) t += span_of<ROWS>(a, n, len, rt).tiles;
  return t * a.p.heads;
}

// Where a share of the tiles begins.
struct Plan {
  long long total, first, at;   // all tiles, this share's first, the first of sequence b
  int b;
};

// Every thread of the block takes part.  plan.b = batch when the share is empty.
template <int ROWS>
__device__ __forceinline__ void make_plan(const KvAttnArgs& a, int share, int shares, Plan* plan, long long* warp_sum,
                                          bool tell) {
  const int tid = threadIdx.x, per = (a.batch + kThreads - 1) / kThreads;
  const int b0 = tid * per, b1 = min(a.batch, b0 + per);
  long long mine = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    int q0, n, len;
    bool wrong;
    lengths_of(a, b, q0, n, len, wrong);
    bad |= wrong;
    mine += tiles_of<ROWS>(a, n, len);
  }
  if (bad && tell && a.status) atomicOr(a.status, FOS_STATUS_INDEX);
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(~0u, upto, o);
    if ((tid & 31) >= o) upto += x;
  }
  if ((tid & 31) == 31) warp_sum[tid >> 5] = upto;
  if (tid == 0) plan->b = a.batch;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < (tid >> 5)) before += warp_sum[w];
    total += warp_sum[w];
  }
  upto += before;
  const long long first = total * share / shares;
  if (tid == 0) { plan->total = total; plan->first = first; }
  if (first >= upto - mine && first < upto) {
    long long at = upto - mine;
    for (int b = b0; b < b1; ++b) {
      int q0, n, len;
      bool wrong;
      lengths_of(a, b, q0, n, len, wrong);
      const long long t = tiles_of<ROWS>(a, n, len);
      if (first < at + t) {
        plan->b = b;
        plan->at = at;
        break;
      }
      at += t;
    }
  }
  __syncthreads();
}

// The item that holds tile `pos`, walking on from sequence b whose first
// tile is `at`.
struct Item {
  int b, rt, h, q0, n, len, nrt;
  long long at, start;          // first tile of the sequence, of the item
  Span s;
};

template <int ROWS>
__device__ __forceinline__ bool find_item(const KvAttnArgs& a, long long pos, int b, long long at, Item& it) {
  for (; b < a.batch; ++b) {
    bool wrong;
    lengths_of(a, b, it.q0, it.n, it.len, wrong);
    it.nrt = (it.n * a.group + ROWS - 1) / ROWS;
    long long x = at;
    for (int rt = 0; rt < it.nrt; ++rt) {
      const Span s = span_of<ROWS>(a, it.n, it.len, rt);
      const long long all = (long long)s.tiles * a.p.heads;
      if (pos < x + all) {
        it.b = b;
        it.rt = rt;
        it.h = (int)((pos - x) / s.tiles);
        it.at = at;
        it.start = x + (long long)it.h * s.tiles;
        it.s = s;
        return true;
      }
      x += all;
    }
    at = x;
  }
  return false;
}

// One row of a finished item: values d .. d + 3 and (lane 0 of the row) lse.
__device__ __forceinline__ void write_row(const KvAttnArgs& a, const Item& it, int r, int d, int D, float4 o, float M,
                                          float L) {
  const int i = r / a.group, hq = it.h * a.group + (r - i * a.group), t = it.q0 + i;
  const float f = L == 0.0f ? 0.0f : __fdividef(a.p.vst[it.h], L);
  const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * f, o.y * f), y = __floats2bfloat162_rn(o.z * f, o.w * f);
  uint2 w;
  w.x = *reinterpret_cast<const uint32_t*>(&x);
  w.y = *reinterpret_cast<const uint32_t*>(&y);
  *reinterpret_cast<uint2*>(a.out + (long long)t * a.out_ld + (long long)hq * D + d) = w;
  if (d == 0 && a.lse)
    a.lse[(long long)t * a.q_heads + hq] =
        L == 0.0f ? -CUDART_INF_F : (M - kLift + log2f(L)) * 0.69314718055994531f;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 2) k_kv_decode(const KvAttnArgs a, float* part) {
  using C = Cfg<D, NT>;
  constexpr int R = C::kRows, KS = D / 16, LD = D / 4;   // rows; reduction steps; values of a token in a lane
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  Plan* plan = reinterpret_cast<Plan*>(smem + C::kOffPlan);
  const uint32_t ring = smem_u32(smem) + warp * kStages * C::kStage;
  const uint8_t* ringp = smem + warp * kStages * C::kStage;
  const uint32_t bars = smem_u32(smem + C::kOffBar) + warp * kStages * 8;
  float* stat = reinterpret_cast<float*>(smem + C::kOffStat);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" :: "r"(bars + 8 * s) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  make_plan<R>(a, blockIdx.x, gridDim.x, plan, reinterpret_cast<long long*>(smem + C::kOffPlan + 64), blockIdx.x == 0);
  const long long first = plan->first, last = plan->total * (blockIdx.x + 1) / gridDim.x;
  int walk_b = plan->b;
  long long walk_at = plan->at;
  uint32_t phases = 0;          // bit s: parity of the next wait on stage s
  bool dead = false;            // a wait gave up

  for (long long pos = first; pos < last;) {
    Item it;
    if (!find_item<R>(a, pos, walk_b, walk_at, it)) break;
    walk_b = it.b;
    walk_at = it.at;
    const int ta = (int)(pos - it.start), tb = (int)min((long long)it.s.tiles, last - it.start);
    const long long seg_pos = pos;
    pos = it.start + tb;

    // ---- copies of this warp's slice of tile k: page ids 32 tiles ahead, a lane each
    const int h = it.h;
    const int32_t* row = a.pages + (long long)it.b * a.max_pages;
    int ids = -1;
    auto load_ids = [&](int k0) {
      const int tok = it.s.base + (k0 + lane) * kTile + warp * kSlice;
      ids = -1;
      if (k0 + lane < tb && tok < it.s.hi) {
        const int page = row[tok >> a.p.page_shift];
        if (page >= 0 && page < a.p.num_pages) ids = page;
        else if (a.status) atomicOr(a.status, FOS_STATUS_INDEX);
      }
    };
    int issued = ta;             // next tile to issue
    auto issue = [&]() {
      if (((issued - ta) & 31) == 0) load_ids(issued);
      const int page = __shfl_sync(~0u, ids, (issued - ta) & 31);
      if (page >= 0 && lane == 0) {
        const int st = (issued - ta) % kStages;
        const int tok = it.s.base + issued * kTile + warp * kSlice;
        const long long r = ((long long)h << a.p.page_shift) + (tok & ((1 << a.p.page_shift) - 1));
        const long long co = page * a.p.codes_stride + r * (D / 2), so = page * a.p.scales_stride + r * (D / 16);
        const uint32_t dst = ring + st * C::kStage, bar = bars + 8 * st;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(C::kStage) : "memory");
        bulk_load(dst, a.p.kc + co, C::kCodes, bar);
        bulk_load(dst + C::kCodes, a.p.vc + co, C::kCodes, bar);
        bulk_load(dst + 2 * C::kCodes, a.p.ks + so, C::kScales, bar);
        bulk_load(dst + 2 * C::kCodes + C::kScales, a.p.vs + so, C::kScales, bar);
      }
      ++issued;
      return page >= 0;
    };
    uint32_t flying = 0;         // bit s: stage s holds or awaits a slice
    auto issue_next = [&]() {
      const int st = (issued - ta) % kStages;
      if (issue()) flying |= 1u << st;
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1 && issued < tb; ++i) issue_next();

    // ---- queries: lane (g, c) holds values LD c .. LD c + LD - 1 of row g of each n-tile
    uint32_t qf[NT][KS][2];
    float rs[NT][2];             // scale of the scores of columns 2c, 2c + 1
    int hi[NT][2], lo[NT][2];
    int min_hi = 0x7fffffff, max_lo = 0;
    const float base_scale = a.scale_log2 * a.p.kst[h];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = it.rt * R + 8 * nt + g;
      float v[LD];
#pragma unroll
      for (int k = 0; k < LD; ++k) v[k] = 0.0f;
      if (r < it.n * a.group) {
        const int i = r / a.group;
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (long long)(it.q0 + i) * a.q_ld +
                                                          (long long)(h * a.group + (r - i * a.group)) * D + LD * c);
#pragma unroll
        for (int k = 0; k < LD / 8; ++k) {
          const uint4 w = __ldg(src + k);
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[8 * k + 2 * e] = bf_lo(x[e]);
            v[8 * k + 2 * e + 1] = bf_hi(x[e]);
          }
        }
      }
      uint32_t top = 0;          // |values| as bits: ordered like the values, NaN and Inf above all
#pragma unroll
      for (int k = 0; k < LD; ++k) top = max(top, __float_as_uint(v[k]) & 0x7fffffffu);
      top = max(top, __shfl_xor_sync(~0u, top, 1));
      top = max(top, __shfl_xor_sync(~0u, top, 2));
      const RowScale sc = row_scale(top);
      const float mine = sc.finite ? base_scale * sc.down1 * sc.down2 : CUDART_NAN_F;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2)
          qf[nt][k][e2] = sc.finite ? pack_h2(v[4 * k + 2 * e2] * sc.up1 * sc.up2, v[4 * k + 2 * e2 + 1] * sc.up1 * sc.up2)
                                    : 0u;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        rs[nt][k] = __shfl_sync(~0u, mine, (2 * c + k) * 4);
        const int rr = it.rt * R + 8 * nt + 2 * c + k;
        hi[nt][k] = lo[nt][k] = 0;
        if (rr < it.n * a.group) {
          hi[nt][k] = query_hi(a, it.n, it.len, rr / a.group);
          lo[nt][k] = query_lo(a, hi[nt][k]);
          min_hi = min(min_hi, hi[nt][k]);
          max_lo = max(max_lo, lo[nt][k]);
        }
      }
    }
    // rows 2c, 2c + 1 over c cover all rows of the tile
    min_hi = min(min_hi, __shfl_xor_sync(~0u, min_hi, 1));
    min_hi = min(min_hi, __shfl_xor_sync(~0u, min_hi, 2));
    max_lo = max(max_lo, __shfl_xor_sync(~0u, max_lo, 1));
    max_lo = max(max_lo, __shfl_xor_sync(~0u, max_lo, 2));

    float m[NT][2], l[NT][2], acc[KS][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -CUDART_INF_F;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[k][nt][e] = 0.0f;
    }

#pragma unroll 1
    for (int k = ta; k < tb; ++k) {
      if (issued < tb && !dead) issue_next();
      const int st = (k - ta) % kStages;
      if (!(flying & (1u << st))) continue;
      flying &= ~(1u << st);
      const uint32_t bar = bars + 8 * st, parity = (phases >> st) & 1;
      if (!__all_sync(~0u, mbar_wait(bar, parity))) {
        dead = true;             // give up, but let the copy land if it does
        mbar_wait(bar, parity);
      }
      phases ^= 1u << st;
      if (dead) continue;
      const uint8_t* base = ringp + st * C::kStage;
      const int tok0 = it.s.base + k * kTile + warp * kSlice;
      const bool edge = tok0 + kSlice > min_hi || tok0 < max_lo;

      // ---- scores
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
      {
        const int t0 = row_token(g), t1 = row_token(g + 8);
        const uint8_t* ks = base + 2 * C::kCodes;
        uint32_t w0[LD / 8], w1[LD / 8], s0[LD / 16], s1[LD / 16];
        if (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(base + t0 * (D / 2) + 16 * c);
          const uint4 y = *reinterpret_cast<const uint4*>(base + t1 * (D / 2) + 16 * c);
          w0[0] = x.x; w0[1] = x.y; w0[LD / 8 - 2] = x.z; w0[LD / 8 - 1] = x.w;
          w1[0] = y.x; w1[1] = y.y; w1[LD / 8 - 2] = y.z; w1[LD / 8 - 1] = y.w;
          const uint32_t p = scales_h2(*reinterpret_cast<const uint16_t*>(ks + t0 * (D / 16) + 2 * c));
          const uint32_t q = scales_h2(*reinterpret_cast<const uint16_t*>(ks + t1 * (D / 16) + 2 * c));
          s0[0] = __byte_perm(p, 0u, 0x1010u); s0[LD / 16 - 1] = __byte_perm(p, 0u, 0x3232u);
          s1[0] = __byte_perm(q, 0u, 0x1010u); s1[LD / 16 - 1] = __byte_perm(q, 0u, 0x3232u);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(base + t0 * (D / 2) + 8 * c);
          const uint2 y = *reinterpret_cast<const uint2*>(base + t1 * (D / 2) + 8 * c);
          w0[0] = x.x; w0[1] = x.y;
          w1[0] = y.x; w1[1] = y.y;
          const uint32_t p = scales_h2(ks[t0 * (D / 16) + c] | (uint32_t)ks[t1 * (D / 16) + c] << 8);
          s0[0] = __byte_perm(p, 0u, 0x1010u);
          s1[0] = __byte_perm(p, 0u, 0x3232u);
        }
#pragma unroll
        for (int w = 0; w < LD / 8; ++w) {
          const uint32_t a0 = hmul2(codes_h2<0>(w0[w]), s0[w >> 1]), a1 = hmul2(codes_h2<0>(w1[w]), s1[w >> 1]);
          const uint32_t a2 = hmul2(codes_h2<1>(w0[w]), s0[w >> 1]), a3 = hmul2(codes_h2<1>(w1[w]), s1[w >> 1]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma(s[nt], a0, a1, a2, a3, qf[nt][2 * w][0], qf[nt][2 * w][1]);
          const uint32_t b0 = hmul2(codes_h2<2>(w0[w]), s0[w >> 1]), b1 = hmul2(codes_h2<2>(w1[w]), s1[w >> 1]);
          const uint32_t b2 = hmul2(codes_h2<3>(w0[w]), s0[w >> 1]), b3 = hmul2(codes_h2<3>(w1[w]), s1[w >> 1]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma(s[nt], b0, b1, b2, b3, qf[nt][2 * w + 1][0], qf[nt][2 * w + 1][1]);
        }
      }
      // ---- softmax: entry e of s is token row g + 8 (e >> 1), column 2c + (e & 1)
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[nt][e] *= rs[nt][e & 1];
          if (edge) {
            const int tok = tok0 + row_token(g + 8 * (e >> 1));
            if (tok >= hi[nt][e & 1] || tok < lo[nt][e & 1]) s[nt][e] = -CUDART_INF_F;
          }
          raise |= s[nt][e] > m[nt][e & 1] + kSlack;
        }
      if (__any_sync(~0u, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2) {
            float t = fmaxf(s[nt][k2], s[nt][k2 + 2]);
            t = fmaxf(t, __shfl_xor_sync(~0u, t, 4));
            t = fmaxf(t, __shfl_xor_sync(~0u, t, 8));
            t = fmaxf(t, __shfl_xor_sync(~0u, t, 16));
            t = fmaxf(t, m[nt][k2]);
            const float keep = t == m[nt][k2] ? 1.0f : ex2(m[nt][k2] - t);
            m[nt][k2] = t;
            l[nt][k2] *= keep;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              acc[i][nt][k2] *= keep;
              acc[i][nt][k2 + 2] *= keep;
            }
          }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float r0 = m[nt][0] == -CUDART_INF_F ? 0.0f : m[nt][0] - kLift;
        const float r1 = m[nt][1] == -CUDART_INF_F ? 0.0f : m[nt][1] - kLift;
        const float p0 = ex2(s[nt][0] - r0), p1 = ex2(s[nt][1] - r1), p2 = ex2(s[nt][2] - r0), p3 = ex2(s[nt][3] - r1);
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        pf[nt][0] = transpose8x8(pack_h2(p0, p1));
        pf[nt][1] = transpose8x8(pack_h2(p2, p3));
      }
      // ---- output
      {
        constexpr int VW = D / 64;             // words of a token in a lane: 8 VW values from 8 VW g on
        const uint8_t *vc = base + C::kCodes, *vs = base + 2 * C::kCodes + C::kScales;
        const int vb = (8 * VW * g) >> 4;      // their block
        uint32_t w[4][VW], sc[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int tok = row_token(2 * c + (t & 1) + 8 * (t >> 1));
          if (VW == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(vc + tok * (D / 2) + 8 * g);
            w[t][0] = x.x;
            w[t][VW - 1] = x.y;
          } else {
            w[t][0] = *reinterpret_cast<const uint32_t*>(vc + tok * (D / 2) + 4 * g);
          }
          sc[t] = vs[tok * (D / 16) + vb];
          // what lies outside the rows' tokens may be anything, NaN too
          if (edge && (tok0 + tok >= it.s.hi || tok0 + tok < it.s.lo)) sc[t] = 0;
        }
        const uint32_t s01 = scales_h2(sc[0] | sc[1] << 8), s23 = scales_h2(sc[2] | sc[3] << 8);
#pragma unroll
        for (int v = 0; v < VW; ++v) {
          const uint32_t e01 = (w[0][v] & 0x0f0f0f0fu) | ((w[1][v] << 4) & 0xf0f0f0f0u);
          const uint32_t o01 = ((w[0][v] >> 4) & 0x0f0f0f0fu) | (w[1][v] & 0xf0f0f0f0u);
          const uint32_t e23 = (w[2][v] & 0x0f0f0f0fu) | ((w[3][v] << 4) & 0xf0f0f0f0u);
          const uint32_t o23 = ((w[2][v] >> 4) & 0x0f0f0f0fu) | (w[3][v] & 0xf0f0f0f0u);
#define FOS_KV_PV(J)                                                                                              \
  {                                                                                                               \
    const uint32_t a0 = hmul2(codes_h2<J>(e01), s01), a1 = hmul2(codes_h2<J>(o01), s01);                          \
    const uint32_t a2 = hmul2(codes_h2<J>(e23), s23), a3 = hmul2(codes_h2<J>(o23), s23);                          \
    _Pragma("unroll") for (int nt = 0; nt < NT; ++nt) mma(acc[4 * v + J][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]); \
  }
          FOS_KV_PV(0)
          FOS_KV_PV(1)
          FOS_KV_PV(2)
          FOS_KV_PV(3)
#undef FOS_KV_PV
        }
      }
      __syncwarp();              // all lanes are done with the stage before it is filled again
    }

    // ---- join the warps' results through shared memory (over the ring: its copies have all landed)
    __syncthreads();
    float* om = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        float t = l[nt][k2];
        t += __shfl_xor_sync(~0u, t, 4);
        t += __shfl_xor_sync(~0u, t, 8);
        t += __shfl_xor_sync(~0u, t, 16);
        const int r = 8 * nt + 2 * c + k2;
        if (g == 0) {
          stat[warp * R + r] = m[nt][k2];
          stat[(kWarps + warp) * R + r] = t;
        }
        float* dst = om + (warp * R + r) * C::kLdO + (D / 8) * g;
#pragma unroll
        for (int i = 0; i < KS; ++i)
          *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(acc[i][nt][k2], acc[i][nt][k2 + 2]);
      }
    __syncthreads();
    const bool whole = ta == 0 && tb == it.s.tiles;
    for (int x = tid; x < R * (D / 4); x += kThreads) {
      const int r = x / (D / 4), d = (x - r * (D / 4)) * 4;
      float M = stat[r];
      for (int w = 1; w < kWarps; ++w) M = fmaxf(M, stat[w * R + r]);
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float L = 0.0f;
      for (int w = 0; w < kWarps; ++w) {
        const float mw = stat[w * R + r], f = mw == M ? 1.0f : ex2(mw - M);
        const float4 v = *reinterpret_cast<const float4*>(om + (w * R + r) * C::kLdO + d);
        L += f * stat[(kWarps + w) * R + r];
        o.x += f * v.x; o.y += f * v.y; o.z += f * v.z; o.w += f * v.w;
      }
      if (whole) {
        if (it.rt * R + r < it.n * a.group) write_row(a, it, it.rt * R + r, d, D, o, M, L);
      } else {
        float* p = part + (long long)(2 * blockIdx.x + (seg_pos == first ? 0 : 1)) * C::kPart;
        *reinterpret_cast<float4*>(p + r * D + d) = o;
        if (d == 0) {
          p[R * D + r] = M;
          p[R * D + R + r] = L;
        }
      }
    }
    __syncthreads();
    // the ring was written by ordinary stores: order them before the next copies
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (dead && a.status) atomicOr(a.status, FOS_STATUS_TIMEOUT);
}

// Joins an item that several shares hold: the CTA of the share in which the
// item ends adds the partial results in the order of the tokens.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads) k_kv_join(const KvAttnArgs a, const float* part) {
  using C = Cfg<D, NT>;
  constexpr int R = C::kRows;
  __shared__ Plan plan;
  __shared__ long long sums[kWarps];
  make_plan<R>(a, blockIdx.x, gridDim.x, &plan, sums, false);
  const long long total = plan.total, first = plan.first, last = total * (blockIdx.x + 1) / gridDim.x;
  Item it;
  const bool mine = first < last && find_item<R>(a, first, plan.b, plan.at, it) && first > it.start &&
                    it.start + it.s.tiles <= last;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!mine) return;
  // the share that holds the item's first tile: the last one that begins at or before it
  int c0 = (int)(it.start * gridDim.x / total);
  while (c0 + 1 < (int)gridDim.x && total * (c0 + 1) / gridDim.x <= it.start) ++c0;
  while (c0 > 0 && total * c0 / gridDim.x > it.start) --c0;
  for (int x = threadIdx.x; x < R * (D / 4); x += kThreads) {
    const int r = x / (D / 4), d = (x - r * (D / 4)) * 4;
    if (it.rt * R + r >= it.n * a.group) continue;
    float M = -CUDART_INF_F, L = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = c0; s <= (int)blockIdx.x; ++s) {
      // a share that holds nothing is passed over; the item is the first segment
      // of every share but the one that it begins inside
      const long long f0 = total * s / gridDim.x, f1 = total * (s + 1) / gridDim.x;
      if (f0 == f1) continue;
      const float* p = part + (long long)(2 * s + (s == c0 && f0 < it.start ? 1 : 0)) * C::kPart;
      const float4 v = *reinterpret_cast<const float4*>(p + r * D + d);
      const float pm = p[R * D + r], top = fmaxf(M, pm);
      const float f = M == top ? 1.0f : ex2(M - top), k = pm == top ? 1.0f : ex2(pm - top);
      L = L * f + p[R * D + R + r] * k;
      o.x = o.x * f + v.x * k; o.y = o.y * f + v.y * k; o.z = o.z * f + v.z * k; o.w = o.w * f + v.w * k;
      M = top;
    }
    write_row(a, it, it.rt * R + r, d, D, o, M, L);
  }
}

template <int D, int NT>
cudaError_t launch(const KvAttnArgs& a, float* part, cudaStream_t st) {
  using C = Cfg<D, NT>;
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(k_kv_decode<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) !=
          cudaSuccess)
    return e;
  const int ctas = 2 * sms < kMaxCtas ? 2 * sms : kMaxCtas;
  k_kv_decode<D, NT><<<ctas, kThreads, C::kSmem, st>>>(a, part);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // a table of one tile at most: no item is ever shared
  if ((a.max_pages << a.p.page_shift) <= kTile) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_kv_join<D, NT>, a, (const float*)part);
}

}  // namespace

size_t kv_decode_workspace_bytes(int dim, int rows) {
  return (size_t)2 * kMaxCtas * (rows <= 8 ? 8 : 16) * (dim + 2) * 4;
}

cudaError_t launch_kv_decode(const KvAttnArgs& a, int rows, float* part, cudaStream_t st) {
  if (a.p.dim == 128) return rows <= 8 ? launch<128, 1>(a, part, st) : launch<128, 2>(a, part, st);
  return rows <= 8 ? launch<64, 1>(a, part, st) : launch<64, 2>(a, part, st);
}

}  // namespace fos
