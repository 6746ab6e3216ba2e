// fos_kv_prompt.cu -- attention of many queries over the key/value cache
// (semantics: include/fos.h), on the tcgen05 tensor cores.
//
// A row is one query of one query head.  A CTA takes 256 rows of a sequence
// that share a key/value head, as two tiles of 128, and walks their visible
// tokens 128 at a time:
//   S = Q K^T    128 x 128, Q and K in shared memory, S in tensor memory
//   O += P V     P in tensor memory (over S), V in shared memory as it is
//                held, [token][value] (an MN-major operand)
// in f16 with f32 sums.  Warps:
//   0-3, 4-7   softmax of tile 0 and 1, a row for each thread: scores out of
//              tensor memory, weights back into it.  The output is rescaled
//              in tensor memory by these warps, and only when a row's maximum
//              was passed by 2^8 (fos_kv.cuh).
//   8-11       keys and values of the next tokens from the cache: a thread
//              converts one token's codes (cvt f16x2.e2m1x2, times the E4M3
//              scale: exact in f16) into the operands' 128-byte swizzle
//   12         issues the MMAs: while one tile's softmax runs, the tensor
//              core has the other tile's products.
// Every commit covers all MMAs issued before it, so a tile's new scores also
// say that its earlier output products are done: the order PV(j), S(j + 1)
// needs no barrier of its own and S may overwrite P.
// With few rows and many tokens gridDim.y CTAs share an item's tokens and
// k_kv_prompt_join adds their results in order.
//
// Bound by the exponentials: 256 rows by 128 tokens take 4300 cycles, of which
// a tile's softmax is 2550 (exponentials 1630, at 10.6 cycles a warp each; the
// maxima 370; tensor memory 330) and its products 840 of the tensor core, the
// other tile's meanwhile; a CTA's start and end take another 10000 to 15000, a
// fifth of one with 17 tiles.  Measured: 8192 queries of 32 heads over 8 heads
// of 128, causal, 562 to 573 us by the machine, 0.98 PFLOP/s, 0.57 of the measured
// bf16 matrix rate, in calls whose inputs change (524 with the same inputs again, as in the
// trials below); 6 chunks of up to 1501 queries, window 2048, head_dim 64, 106 us; 8 x 448
// queries over up to 1500 tokens, 16 heads of 64, 32 us.  Slower: two threads
// a row (875 us), a polynomial for a quarter of the exponentials (642 against
// 631 without), the weights handed over in halves (625 against 629: no gain), 64
// tokens a turn with two score buffers a tile (602 against 541: an MMA of 64
// tokens takes as long as one of 128).
#include <math_constants.h>

#include "fos_kv.cuh"

namespace fos {
namespace {

constexpr int kRows = 256, kTileRows = 128, kTileTok = 128;
constexpr int kThreads = 512;
constexpr uint32_t kWaitLimit = 1u << 20;

template <int D>
struct Cfg {
  static constexpr int kHalf = kTileRows * 128;               // 64 values of 128 rows, 128-byte swizzle
  static constexpr int kOperand = (D / 64) * kHalf;           // a Q, K or V tile
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + 2 * kOperand;
  static constexpr int kOffV = kOffK + 2 * kOperand;
  static constexpr int kOffValid = kOffV + 2 * kOperand;      // visible-token masks, ring of 4 tiles x 128 bits
  static constexpr int kOffScale = kOffValid + 64;            // the rows' powers of two
  static constexpr int kOffBar = kOffScale + kRows * 4;
  static constexpr int kBars = 16;
  static constexpr int kOffMisc = kOffBar + 8 * kBars;        // tensor memory base, failure flag, the item
  static constexpr int kSmem = kOffMisc + 384 + 1024;         // + alignment slack
  // kind::f16, f32 accumulator, f16 operands; M = 128
  static constexpr uint32_t kIdescS = (1u << 4) | ((kTileTok / 8) << 17) | ((128 / 16) << 24);
  static constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((D / 8) << 17) | ((128 / 16) << 24);  // B MN-major
  static constexpr uint32_t kColS = 0, kColO = 256;           // + 128 * tile
};

enum { B_Q = 0, B_KFULL = 1, B_KEMPTY = 3, B_VFULL = 5, B_VEMPTY = 7, B_S = 9, B_P = 11, B_O = 13, B_DRAIN = 15 };

// Bounded wait; gives up at once when another warp has.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* fail) {
  for (uint32_t it = 0; it < kWaitLimit; ++it) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    if (done) return true;
    if (*fail) return false;
  }
  *fail = 1;
  return false;
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}

// Operand descriptors, 128-byte swizzle, as two words.  Low: the address and,
// for the MN-major values, the distance of its groups of 64 (unused, 1, for
// K-major).  High: 1024 bytes between groups of 8 rows (K-major) or tokens.
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return ((addr & 0x3FFFF) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr, uint32_t half) {
  return ((addr & 0x3FFFF) >> 4) | ((half >> 4) << 16);
}

// One lane of the (converged) warp, the same each time: commits cover the
// MMAs of the thread that issues them.  8192 causal queries: 530 us with a
// branch on elect.sync, 541 with each MMA predicated on lane 0, 5 % more again
// from a branch on lane 0.
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}"
      :: "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHi) : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}"
      :: "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHi) : "memory");
}

__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}

#define FOS_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
    "=r"(r[i + 6]), "=r"(r[i + 7])
#define FOS_I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
    "r"(r[i + 6]), "r"(r[i + 7])

// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : FOS_R8(r, 0), FOS_R8(r, 8), FOS_R8(r, 16), FOS_R8(r, 24) : "r"(addr));
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
      :: FOS_I8(r, 0), FOS_I8(r, 8), FOS_I8(r, 16), FOS_I8(r, 24), "r"(addr) : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Rows rt * 256 .. of sequence b, and the tokens [lo, hi) that any of them
// sees, `base` (a multiple of 16) on in tiles of 128.
struct Item {
  int b, rt, q0, n, len, lo, hi, base, tiles;
};

// The rows rt of a sequence whose q0, n and len are set.
__device__ __forceinline__ void set_rows(const KvAttnArgs& a, Item& it, int rt) {
  it.rt = rt;
  const int first = fdiv(it.rt * kRows, a.by_group);
  const int last = fdiv(min(it.n * a.group - 1, it.rt * kRows + kRows - 1), a.by_group);
  it.hi = query_hi(a, it.n, it.len, last);
  it.lo = query_lo(a, query_hi(a, it.n, it.len, first));
  it.base = it.lo & ~15;
  it.tiles = (it.hi - it.base + kTileTok - 1) / kTileTok;
}

// Item number `want` over all sequences (the last rows of a sequence, which
// see the most, first); every thread of the block takes part and has it in
// `it`.  False beyond the last item, and for all where the sequences have too
// many queries.  Up to 32 sequences: every warp by itself,
// a sequence for each lane, which saves the block two meetings of a start of
// 13000 cycles (2000 for the item, 1100 to meet); more: the block together,
// through shared memory, a sequence for each thread at once instead of 32 in turn.
__device__ __forceinline__ bool find_item(const KvAttnArgs& a, int want, int threads, Item& it, Item* shared,
                                          int* warp_sum, long long* block_sum, bool tell) {
  const int tid = threadIdx.x, lane = tid & 31;
  bool bad = false, ordered = true, wrong;
  if (a.batch <= 32) {
    int nrt = 0;
    if (lane < a.batch) {
      ordered = lengths_of(a, lane, it.q0, it.n, it.len, wrong);
      bad = wrong;
      nrt = (it.n * a.group + kRows - 1) / kRows;
    }
    if (!__all_sync(~0u, ordered)) {      // too many queries (too_many): halves of 16 bits, that the sums fit
      const unsigned n = nrt ? it.n : 0;
      if (((long long)__reduce_add_sync(~0u, n >> 16) << 16) + __reduce_add_sync(~0u, n & 0xffffu) > a.total_q) nrt = 0;
    }
    if (bad && tell && tid < 32 && a.status) atomicOr(a.status, FOS_STATUS_INDEX);
    int upto = nrt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += x;
    }
    const uint32_t beyond = __ballot_sync(~0u, want < upto);
    if (!beyond) return false;
    it.b = __ffs(beyond) - 1;
    it.q0 = __shfl_sync(~0u, it.q0, it.b);
    it.n = __shfl_sync(~0u, it.n, it.b);
    it.len = __shfl_sync(~0u, it.len, it.b);
    set_rows(a, it, __shfl_sync(~0u, upto, it.b) - 1 - want);
    return true;
  }
  const int per = (a.batch + threads - 1) / threads;
  const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
  int mine = 0;
  long long asked = 0;
  for (int b = b0; b < b1 && asked <= a.total_q; ++b) {
    ordered &= lengths_of(a, b, it.q0, it.n, it.len, wrong);
    bad |= wrong;
    asked += it.n;
    mine += (it.n * a.group + kRows - 1) / kRows;
  }
  if (bad && tell && a.status) atomicOr(a.status, FOS_STATUS_INDEX);
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) warp_sum[tid >> 5] = upto;
  if (tid == 0) shared->b = -1;
  const bool broken = __syncthreads_or(!ordered) && too_many(a, asked, block_sum);
  for (int w = 0; w < (tid >> 5); ++w) upto += warp_sum[w];
  int at = upto - mine;
  if (want >= at && want < upto && !broken)
    for (int b = b0; b < b1; ++b) {
      if (per > 1) lengths_of(a, b, it.q0, it.n, it.len, wrong);
      const int nrt = (it.n * a.group + kRows - 1) / kRows;
      if (want < at + nrt) {
        it.b = b;
        set_rows(a, it, nrt - 1 - (want - at));
        *shared = it;
        break;
      }
      at += nrt;
    }
  __syncthreads();
  it = *shared;
  return it.b >= 0;
}

// One 8-value word of codes times its block's scale -> 16 bytes
__device__ __forceinline__ uint4 word_f16(uint32_t w, uint32_t s) {
  uint32_t h[4];
  codes_h2x4(w, h);
  return make_uint4(hmul2(h[0], s), hmul2(h[1], s), hmul2(h[2], s), hmul2(h[3], s));
}

// The codes and scales of one token's head.
template <int D>
struct Raw {
  uint32_t w[D / 8], s[D / 64];
};

template <int D>
__device__ __forceinline__ void load_raw(Raw<D>& r, const uint8_t* codes, const uint8_t* scales, bool live) {
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
    const uint4 x = live ? __ldg(reinterpret_cast<const uint4*>(codes) + k) : make_uint4(0u, 0u, 0u, 0u);
    r.w[4 * k] = x.x; r.w[4 * k + 1] = x.y; r.w[4 * k + 2] = x.z; r.w[4 * k + 3] = x.w;
  }
#pragma unroll
  for (int k = 0; k < D / 64; ++k) r.s[k] = live ? __ldg(reinterpret_cast<const uint32_t*>(scales) + k) : 0u;
}

// Row `row` of an operand tile at `tile` (shared memory, generic address).
template <int D>
__device__ __forceinline__ void store_raw(const Raw<D>& r, uint8_t* tile, int row) {
#pragma unroll
  for (int b = 0; b < D / 16; ++b) {
    const uint32_t pair = scales_h2(b & 2 ? r.s[b >> 2] >> 16 : r.s[b >> 2] & 0xffffu);
    const uint32_t s = __byte_perm(pair, 0u, b & 1 ? 0x3232u : 0x1010u);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int w = 2 * b + e;
      *reinterpret_cast<uint4*>(tile + (w >> 3) * Cfg<D>::kHalf + row * 128 + (((w & 7) ^ (row & 7)) << 4)) =
          word_f16(r.w[w], s);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_kv_prompt(const KvAttnArgs a, float* part) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  const uint32_t sbase = smem_u32(smem), bar = sbase + C::kOffBar;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc);
  volatile uint32_t* fail = tmem_slot + 1;
  Item* item = reinterpret_cast<Item*>(smem + C::kOffMisc + 16);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    *fail = 0;
    auto init = [&](int b, int count) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar + 8 * b), "r"(count) : "memory");
    };
    init(B_Q, 8);
    for (int s = 0; s < 2; ++s) {
      init(B_KFULL + s, 4);
      init(B_KEMPTY + s, 1);
      init(B_VFULL + s, 4);
      init(B_VEMPTY + s, 1);
      init(B_S + s, 1);
      init(B_P + s, 4);
      init(B_O + s, 1);
    }
    init(B_DRAIN, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
                 :: "r"(smem_u32((const void*)tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  Item mine;
  const bool found = find_item(a, blockIdx.x / a.p.heads, kThreads, mine, item,
                               reinterpret_cast<int*>(smem + C::kOffMisc + 128),
                               reinterpret_cast<long long*>(smem + C::kOffMisc + 256),
                               blockIdx.x == 0 && blockIdx.y == 0);
  const int h = blockIdx.x % a.p.heads;
  const int here = found ? mine.n * a.group - mine.rt * kRows : 0;
  // The queries of a softmax warp's 32 rows, a row for D / 8 lanes at a time,
  // are on their way before the block meets.
  constexpr int kLanes = D / 8, kStep = 32 / kLanes;
  const int chunk = lane & (kLanes - 1);
  uint4 qw[kLanes];
  if (warp < 8 && (warp >> 2) * kTileRows < here) {
#pragma unroll
    for (int y = 0; y < kLanes; ++y) {
      const int rr = min(mine.rt * kRows + warp * 32 + y * kStep + lane / kLanes, mine.n * a.group - 1);
      const int i = (int)fdiv(rr, a.by_group);
      qw[y] = __ldg(reinterpret_cast<const uint4*>(a.q + (long long)(mine.q0 + i) * a.q_ld +
                                                   (long long)(h * a.group + (rr - i * a.group)) * D) + chunk);
    }
  }
  if (tid == 0) *item = mine;        // read again where it is used, to hold no registers
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  if (!found) {
    if (warp == 12)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
    return;
  }
  const Item it = *item;
  const int rows = it.n * a.group - it.rt * kRows;           // of this item, may exceed kRows
  const int nt = rows > kTileRows ? 2 : 1;                   // tiles with rows
  const int j0 = (int)((long long)it.tiles * blockIdx.y / gridDim.y);
  const int J = (int)((long long)it.tiles * (blockIdx.y + 1) / gridDim.y) - j0;
  const int tok_base = it.base + j0 * kTileTok;

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int t = warp >> 2, rl = (warp & 3) * 32 + lane;    // tile, row in it
    const int r = it.rt * kRows + t * kTileRows + rl;
    const bool live = r < it.n * a.group;
    const int qi = live ? (int)fdiv(r, a.by_group) : 0, hq = h * a.group + (live ? r - qi * a.group : 0);
    float vst = 0.0f;
    if (t >= nt && lane == 0) mbar_arrive(bar + 8 * B_Q);
    if (t < nt) {
      // the warp's 32 queries, scaled by a power of two (and the sign of the
      // softmax scale, so that larger scores are larger weights)
      const float kst = a.scale_log2 * __ldg(a.p.kst + h);
      vst = __ldg(a.p.vst + h);
      uint8_t* qt = smem + C::kOffQ + t * C::kOperand;
      float* scales = reinterpret_cast<float*>(smem + C::kOffScale) + t * kTileRows + (warp & 3) * 32;
      uint32_t tops[kLanes];
#pragma unroll
      for (int y = 0; y < kLanes; ++y) {
        const uint32_t x4[4] = {qw[y].x, qw[y].y, qw[y].z, qw[y].w};
        tops[y] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) tops[y] = max(tops[y], max((x4[e] & 0x7fffu) << 16, x4[e] & 0x7fff0000u));
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1)
#pragma unroll
        for (int y = 0; y < kLanes; ++y) tops[y] = max(tops[y], __shfl_xor_sync(~0u, tops[y], o));
#pragma unroll
      for (int r8 = 0; r8 < kLanes; ++r8) {
        const int x = r8 * kStep + lane / kLanes, row = (warp & 3) * 32 + x;
        const bool there = it.rt * kRows + t * kTileRows + row < it.n * a.group;
        const uint32_t top = tops[r8], x4[4] = {qw[r8].x, qw[r8].y, qw[r8].z, qw[r8].w};
        uint32_t y[4];
        const RowScale sc = row_scale(top);
        float up1 = there && sc.finite ? (kst < 0.0f ? -sc.up1 : sc.up1) : 0.0f;
        // one factor does unless the row's largest value is below 2^-113
        const bool tiny = __any_sync(~0u, top < (14u << 23));
        if (!tiny) up1 *= sc.up2;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo = bf_lo(x4[e]) * up1, hi = bf_hi(x4[e]) * up1;
          if (tiny) { lo *= sc.up2; hi *= sc.up2; }
          y[e] = sc.finite ? pack_h2(lo, hi) : 0u;
        }
        *reinterpret_cast<uint4*>(qt + (chunk >> 3) * C::kHalf + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)) =
            make_uint4(y[0], y[1], y[2], y[3]);
        if (chunk == 0) scales[x] = sc.finite ? fabsf(kst) * sc.down1 * sc.down2 : CUDART_NAN_F;
      }
      __syncwarp();
      const int hi = live ? query_hi(a, it.n, it.len, qi) : 0, lo = query_lo(a, hi);
      // never 0 (2^-120 leaves every score's weight at 1), and not NaN for a
      // row without keys: masked scores are -inf before they are scaled
      float rs = scales[lane];
      if (rs < 7.52316385e-37f || hi <= lo) rs = 7.52316385e-37f;
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + 8 * B_Q);

      int min_hi = live ? hi : 0x7fffffff, max_lo = lo;
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        min_hi = min(min_hi, __shfl_xor_sync(~0u, min_hi, o));
        max_lo = max(max_lo, __shfl_xor_sync(~0u, max_lo, o));
      }
      const uint32_t ts = tmem + ((uint32_t)((warp & 3) * 32) << 16) + C::kColS + 128 * t;
      const uint32_t to = tmem + ((uint32_t)((warp & 3) * 32) << 16) + C::kColO + 128 * t;
      float m = -CUDART_INF_F, l = 0.0f;     // the maximum of the scores as they are, before rs
      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < J; ++j) {
        if (!__all_sync(~0u, mbar_wait(bar + 8 * (B_S + t), j & 1, fail))) { ok = false; break; }
        fence_after();
        uint32_t s[128];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32(ts + 32 * k, s + 32 * k);
        const int tok0 = tok_base + j * kTileTok;
        const uint4 seen = *reinterpret_cast<const uint4*>(smem + C::kOffValid + (j & 3) * 16);
        tmem_wait_ld();
        if ((seen.x & seen.y & seen.z & seen.w) != ~0u || tok0 + kTileTok > min_hi || tok0 < max_lo) {
          const uint32_t v[4] = {seen.x, seen.y, seen.z, seen.w};
#pragma unroll
          for (int k = 0; k < 128; ++k)
            if (!((v[k >> 5] >> (k & 31)) & 1u) || tok0 + k >= hi || tok0 + k < lo) s[k] = 0xff800000u;
        }
        float xm[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          xm[c] = fmaxf(__uint_as_float(s[c]), __uint_as_float(s[c + 4]));
#pragma unroll
          for (int k = 8 + c; k < 128; k += 8)
            xm[c] = fmaxf(fmaxf(xm[c], __uint_as_float(s[k])), __uint_as_float(s[k + 4]));
        }
        const float x0 = fmaxf(fmaxf(xm[0], xm[1]), fmaxf(xm[2], xm[3]));
        const bool raise = x0 > m && (m == -CUDART_INF_F || (x0 - m) * rs > kSlack);
        if (__any_sync(~0u, raise)) {
          const float keep = !raise ? 1.0f : m == -CUDART_INF_F ? 0.0f : ex2((m - x0) * rs);
          if (raise) m = x0;
          l *= keep;
          if (j > 0) {
            // this tile's earlier output products are done (their commit came before these scores')
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
              uint32_t o[32];
              tmem_ld32(to + k, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
              tmem_st32(to + k, o);
            }
          }
        }
        const float off = m == -CUDART_INF_F ? 0.0f : kLift - m * rs;
        const float2 rs2 = make_float2(rs, rs), off2 = make_float2(off, off);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int k = 0; k < 64; ++k) {
          const float2 x = fma2(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), rs2, off2);
          const float2 p = make_float2(ex2(x.x), ex2(x.y));
          sum[k & 1] = add2(sum[k & 1], p);
          s[k] = pack_h2(p.x, p.y);
        }
        tmem_st32(ts, s);
        tmem_st32(ts + 32, s + 32);
        sum[0] = add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + 8 * (B_P + t));
      }
      if (J > 0 && ok) ok = __all_sync(~0u, mbar_wait(bar + 8 * (B_O + t), 0, fail));
      fence_after();
      // the output: a warp's rows through shared memory, each where the query of
      // its row was, so that whole rows are written at once.  No product reads the
      // queries any more, and a warp touches no bytes but its own queries': the
      // other warps may still be writing theirs when there are no tokens to wait for.
      const float msc = m == -CUDART_INF_F ? -CUDART_INF_F : m * rs;
      const bool split = gridDim.y > 1;
      const long long row = (long long)(it.q0 + qi) * a.q_heads + hq;
      const long long all = (long long)a.total_q * a.q_heads;
      const float f = l == 0.0f ? 0.0f : __fdividef(vst, l);
      const bool none = l == 0.0f || J == 0 || !ok;
      uint8_t* ot = smem + C::kOffQ + t * C::kOperand + (warp & 3) * 32 * 128;
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        uint32_t o[32];
        if (J > 0 && ok) {
          tmem_ld32(to + k, o);
          tmem_wait_ld();
        }
        if (split) {
          if (live && J > 0) {
            float4* dst = reinterpret_cast<float4*>(part + (blockIdx.y * all + row) * D + k);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                   __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(none ? 0.0f : __uint_as_float(o[8 * e + 2 * i]) * f,
                                                             none ? 0.0f : __uint_as_float(o[8 * e + 2 * i + 1]) * f);
              w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            const int c = k / 8 + e;
            *reinterpret_cast<uint4*>(ot + (c >> 3) * C::kHalf + lane * 128 + (((c & 7) ^ (lane & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();
      }
      if (!split) {
#pragma unroll
        for (int x = lane / kLanes; x < 32; x += kStep) {
          const int rr = it.rt * kRows + t * kTileRows + (warp & 3) * 32 + x;
          if (rr < it.n * a.group) {
            const int i = (int)fdiv(rr, a.by_group);
            reinterpret_cast<uint4*>(a.out + (long long)(it.q0 + i) * a.out_ld +
                                     (long long)(h * a.group + (rr - i * a.group)) * D)[chunk] =
                *reinterpret_cast<const uint4*>(ot + (chunk >> 3) * C::kHalf + x * 128 +
                                                (((chunk & 7) ^ (x & 7)) << 4));
          }
        }
      }
      if (live) {
        if (split) {
          float2* stat = reinterpret_cast<float2*>(part + (long long)gridDim.y * all * D);
          stat[blockIdx.y * all + row] = make_float2(msc, l);
        } else if (a.lse) {
          a.lse[row] = l == 0.0f ? -CUDART_INF_F : (msc - kLift + log2f(l)) * 0.69314718055994531f;
        }
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------ keys and values
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    const int row = tid - 256;
    const int32_t* pages = a.pages + (long long)it.b * a.max_pages;
    // this thread's token of a tile, two tiles ahead of the conversion: its
    // page's id; one ahead: where it is in the pools, and its codes and scales
    auto page_of = [&](int j) {
      const int tok = tok_base + j * kTileTok + row;
      int page = -1;
      if (j < J && tok >= it.lo && tok < it.hi) {
        page = __ldg(pages + (tok >> a.p.page_shift));
        if ((uint32_t)page >= (uint32_t)a.p.num_pages) {
          page = -1;
          if (a.status) atomicOr(a.status, FOS_STATUS_INDEX);
        }
      }
      return page;
    };
    unsigned long long co = 0, so = 0;
    bool seen = false;
    auto locate = [&](int j, int page) {
      const uint32_t r = ((uint32_t)h << a.p.page_shift) +
                         ((uint32_t)(tok_base + j * kTileTok + row) & ((1u << a.p.page_shift) - 1));
      seen = page >= 0;
      co = (unsigned long long)(uint32_t)page * a.p.codes_stride32 + r * (D / 2);
      so = (unsigned long long)(uint32_t)page * a.p.scales_stride32 + r * (D / 16);
    };
    Raw<D> k, v;
    bool seen_k = false;           // of the keys in k
    int page = -1;
    if (J > 0) {
      locate(0, page_of(0));
      seen_k = seen;
      load_raw<D>(k, a.p.kc + co, a.p.ks + so, seen);
      load_raw<D>(v, a.p.vc + co, a.p.vs + so, seen);
      page = page_of(1);
    }
#pragma unroll 1
    for (int j = 0; j < J; ++j) {
      const int s = j & 1;
      const uint32_t parity = ((j >> 1) & 1) ^ 1;
      locate(j + 1, page);
      page = page_of(j + 2);
      if (j >= 2 && !__all_sync(~0u, mbar_wait(bar + 8 * (B_KEMPTY + s), parity, fail))) break;
      const uint32_t mask = __ballot_sync(~0u, seen_k);
      if (lane == 0) reinterpret_cast<uint32_t*>(smem + C::kOffValid)[(j & 3) * 4 + (warp & 3)] = mask;
      store_raw<D>(k, smem + C::kOffK + s * C::kOperand, row);
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + 8 * (B_KFULL + s));
      load_raw<D>(k, a.p.kc + co, a.p.ks + so, seen);
      seen_k = seen;
      if (j >= 2 && !__all_sync(~0u, mbar_wait(bar + 8 * (B_VEMPTY + s), parity, fail))) break;
      store_raw<D>(v, smem + C::kOffV + s * C::kOperand, row);
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + 8 * (B_VFULL + s));
      load_raw<D>(v, a.p.vc + co, a.p.vs + so, seen);
    }
  } else {
    // ---------------------------------------------------------------- MMAs
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 12 && J > 0) {
      const uint32_t dq = desc_k(sbase + C::kOffQ), dk = desc_k(sbase + C::kOffK);
      const uint32_t dv = desc_mn(sbase + C::kOffV, C::kHalf);
      constexpr uint32_t kStep = C::kOperand >> 4;    // from one tile or stage to the next
      auto scores = [&](uint32_t t, uint32_t stage) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t at = ((i >> 2) * C::kHalf + (i & 3) * 32) >> 4;
          mma_ss(tmem + C::kColS + 128 * t, dq + t * kStep + at, dk + stage * kStep + at, C::kIdescS, i > 0);
        }
        commit(bar + 8 * (B_S + t));
      };
      // the warp stays together, a wait that gave up included
      auto wait = [&](int b, uint32_t parity) { return __all_sync(~0u, mbar_wait(bar + 8 * b, parity, fail)) != 0; };
      bool ok = wait(B_Q, 0) && wait(B_KFULL, 0);
      if (ok) {
        fence_after();
        if (elect()) {
          for (int t = 0; t < nt; ++t) scores(t, 0);
          commit(bar + 8 * B_KEMPTY);
        }
        __syncwarp();
      }
#pragma unroll 1
      for (int j = 0; ok && j < J; ++j) {
        const uint32_t s = j & 1, s1 = s ^ 1;
        // keys and values are there long before the weights as a rule
        ok = wait(B_VFULL + s, (j >> 1) & 1) && (j + 1 >= J || wait(B_KFULL + s1, ((j + 1) >> 1) & 1));
#pragma unroll 1
        for (int t = 0; ok && t < nt; ++t) {
          ok = wait(B_P + t, j & 1);
          if (!ok) break;
          fence_after();
          if (elect()) {
#pragma unroll
            for (int i = 0; i < kTileTok / 16; ++i)
              mma_ts(tmem + C::kColO + 128 * t, tmem + C::kColS + 128 * t + 8 * i, dv + s * kStep + (i * 2048 >> 4),
                     C::kIdescO, j > 0 || i > 0);
            if (j + 1 < J) scores(t, s1);
            else           commit(bar + 8 * (B_O + t));
          }
          __syncwarp();
        }
        // of tile j, all products; of tile j + 1, the scores
        if (elect()) {
          commit(bar + 8 * (B_VEMPTY + s));
          if (j + 1 < J) commit(bar + 8 * (B_KEMPTY + s1));
        }
        __syncwarp();
      }
      if (!ok) {   // let what was issued finish before the tensor memory is freed
        if (elect()) commit(bar + 8 * B_DRAIN);
        __syncwarp();
        for (uint32_t i = 0; i < kWaitLimit; ++i) {
          uint32_t done;
          asm volatile(
              "{\n\t.reg .pred p;\n\t"
              "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], 0;\n\t"
              "selp.u32 %0, 1, 0, p;\n\t}"
              : "=r"(done) : "r"(bar + 8 * B_DRAIN) : "memory");
          if (done) break;
        }
      }
    }
    __syncwarp();
  }
  fence_before();
  __syncthreads();
  if (warp == 12) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
  }
  if (tid == 0 && *fail && a.status) atomicOr(a.status, FOS_STATUS_TIMEOUT);
}

// Adds the results of the CTAs that shared an item's tokens; blockIdx.y: which
// 256 / (D / 4) of its rows.
template <int D>
__global__ void __launch_bounds__(256) k_kv_prompt_join(const KvAttnArgs a, const float* part, int splits) {
  __shared__ Item item;
  __shared__ int sums[8];
  __shared__ long long queries[8];
  Item it;
  const bool found = find_item(a, blockIdx.x / a.p.heads, 256, it, &item, sums, queries, false);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!found) return;
  const int h = blockIdx.x % a.p.heads;
  const long long all = (long long)a.total_q * a.q_heads;
  const float2* stat = reinterpret_cast<const float2*>(part + (long long)splits * all * D);
  constexpr int kLanes = D / 4;
  const int d = (threadIdx.x % kLanes) * 4;
  const int r = it.rt * kRows + blockIdx.y * (256 / kLanes) + threadIdx.x / kLanes;
  if (r >= it.n * a.group) return;
  const int qi = (int)fdiv(r, a.by_group), hq = h * a.group + (r - qi * a.group);
  const long long row = (long long)(it.q0 + qi) * a.q_heads + hq;
  float M = -CUDART_INF_F, L = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float2 ml = stat[s * all + row];
    const float4 v = ml.y == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)   // saw nothing: its output was not written
                                  : *reinterpret_cast<const float4*>(part + (s * all + row) * D + d);
    const float top = fmaxf(M, ml.x);
    const float f = M == top ? 1.0f : ex2(M - top), k = ml.x == top ? 1.0f : ex2(ml.x - top);
    L = L * f + ml.y * k;
    o.x = o.x * f + v.x * k; o.y = o.y * f + v.y * k; o.z = o.z * f + v.z * k; o.w = o.w * f + v.w * k;
    M = top;
  }
  const float f = L == 0.0f ? 0.0f : __fdividef(a.p.vst[h], L);
  const __nv_bfloat162 y = __floats2bfloat162_rn(o.x * f, o.y * f), z = __floats2bfloat162_rn(o.z * f, o.w * f);
  uint2 w;
  w.x = *reinterpret_cast<const uint32_t*>(&y);
  w.y = *reinterpret_cast<const uint32_t*>(&z);
  *reinterpret_cast<uint2*>(a.out + (long long)(it.q0 + qi) * a.out_ld + (long long)hq * D + d) = w;
  if (d == 0 && a.lse)
    a.lse[row] = L == 0.0f ? -CUDART_INF_F : (M - kLift + log2f(L)) * 0.69314718055994531f;
}

// Items that the grid has room for: the rows of every sequence in units of 256.
long long item_bound(long long total_q, long long batch, long long group) {
  return total_q * group / kRows + batch;
}

template <int D>
cudaError_t launch(const KvAttnArgs& a, int splits, float* part, cudaStream_t st) {
  using C = Cfg<D>;
  static KvDevices devices;
  int sms = 0;
  cudaError_t e = devices.get((const void*)k_kv_prompt<D>, C::kSmem, &sms);
  if (e != cudaSuccess) return e;
  const long long grid = item_bound(a.total_q, a.batch, a.group) * a.p.heads;
  k_kv_prompt<D><<<dim3((unsigned)grid, splits), kThreads, C::kSmem, st>>>(a, part);
  if ((e = cudaGetLastError()) != cudaSuccess || splits == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, kRows / (256 / (D / 4)));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_kv_prompt_join<D>, a, (const float*)part, splits);
}

}  // namespace

// CTAs that share an item's tokens: enough to fill 148 SMs (a B200's; workspaces
// are sized without asking a device) when the items do not, with four tiles of
// tokens for each at least, as the page table's width has it: where it is far
// above the lengths, CTAs without tokens and a join come with it.  max_q bounds
// the items more tightly than the grid does, which must hold whatever the offsets
// say.
int kv_prompt_splits(long long total_q, long long batch, long long group, long long heads, long long max_q,
                     long long max_kv) {
  const long long each = batch * ((max_q * group + kRows - 1) / kRows), all = item_bound(total_q, batch, group);
  const long long items = (each < all ? each : all) * heads;
  const long long tiles = (max_kv + kTileTok - 1) / kTileTok;
  long long s = items >= 148 ? 1 : 148 / items;
  if (s > tiles / 4) s = tiles / 4;
  // the workspace holds every row of q, those of no sequence too: at most four CTAs' rows for each SM
  const long long held = ((total_q * group + kRows - 1) / kRows) * heads;
  if (s > 4 * 148 / held) s = 4 * 148 / held;
  return s < 1 ? 1 : (int)s;
}

bool kv_prompt_fits(long long total_q, long long batch, long long group, long long heads) {
  return item_bound(total_q, batch, group) * heads <= 0x7fffffffll;
}

size_t kv_prompt_workspace_bytes(int dim, int splits, long long rows) {
  return splits > 1 ? (size_t)splits * rows * (dim + 2) * 4 : 0;
}

cudaError_t launch_kv_prompt(const KvAttnArgs& a, int splits, float* part, cudaStream_t st) {
  return a.p.dim == 128 ? launch<128>(a, splits, part, st) : launch<64>(a, splits, part, st);
}

}  // namespace fos
