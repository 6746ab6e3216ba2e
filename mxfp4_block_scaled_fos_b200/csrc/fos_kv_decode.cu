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
// A CTA has two groups of 4 warps, which take its tiles in turn; a warp has
// 32 tokens of a tile.
//   S^T = K Q^T runs on the FP4 tensor cores (tcgen05 kind::mxf4nvf4) on the
// codes and scales as the cache holds them: the 128 tokens are the rows of A.
// Queries become FP4 operands: a row is scaled by a power of two so that its
// largest value lies in [2^22, 2^23), rounded to integers (off by half a unit,
// 2^-23 of the row's largest value at most; a bf16 within 2^15 of it is exact),
// written in balanced base 8, and the digits -4 .. 4 are E2M1 values (halves).
// Digit j and digit j + 4 share column j of a row, as two products with scales
// 2^-6 and 2^6; a score is the sum of its 4 columns times 8^j.  So no key is
// converted in registers, where four codes take a conversion and a product each
// pair: that is left to the values, a third of the instructions of a tile.
//   O^T += V^T P^T runs on m16n8k16 with f16 operands: A = 16 output values
// of 16 tokens, B = the weights of 8 rows. A code times its E4M3 scale has 6
// significant bits between 2^-10 and 2688, exact in f16. A register holds one
// value of two tokens: nibbles of two tokens' words are zipped into bytes and
// converted together (cvt f16x2.e2m1x2). A warp reads the scores of its own
// tokens, a token for each lane, and only its own values, so the warps of a group
// meet at one barrier a tile, which only the warp that issues the next
// products waits for: the next tile's keys are there, this one's scores read.
// The next tile's scores are computed while this one's values are.
// The running maximum of a row is raised, and its sums rescaled, only when a
// score passes it by 2^8 (fos_kv.cuh).
//
// Measured: 64 sequences of up to 16384 tokens (598 MB of 8 heads of 128,
// pages of 16) 148 us with k_kv_join, 0.63 of the copy bandwidth; 4 of up to
// 131072 tokens (407 MB) 101 us, 0.62; one of 1000 tokens 12 us.  More than 8
// rows cost more (launch_kv_decode): 32 sequences of up to 16384 tokens, floor 48
// us, 90 us with 1 to 8 rows, 125 with 16, 225 with 32.  A CTA in the middle of
// a long item reads at 0.95 of it; beginning an item costs it 5 to 7 us (page
// ids, digits, the first scores, the warps' results joined), which the other CTA
// of the SM covers in part, and the plan 2 us.
#include <math_constants.h>

#include "fos_kv.cuh"

namespace fos {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kSlice = 16, kTile = 128;               // tokens of one copy, of a tile
constexpr int kStagesK = 2, kStagesV = 3;             // tiles of a group in shared memory
// What beginning an item costs, in tiles.  Without it a share of many short
// items takes far longer than its tiles say: 64 ragged contexts of up to
// 16384 tokens 209 us with 0, 154 with 4 to 8, 156 with 10; 48 windows of 1000
// tokens 47, 34, 32 (8) and 32 us.
constexpr int kOver = 8;
constexpr int kMaxCtas = 320;                         // shares: two CTAs on each of up to 160 SMs
constexpr float kNone = -1e30f;                       // the maximum of a row that has seen nothing
constexpr uint32_t kWaitLimit = 1u << 20;

template <int D, int NT>
struct Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kCtas = NT == 1 ? 2 : 1;                          // on an SM: 16 rows take all registers
  static constexpr int kCols = 4 * kRows;                                // score columns: row r, digits j: j * kRows + r
  static constexpr int kCodes = kTile * D / 2, kScales = kTile * D / 16; // bytes of a tile's keys (or values)
  static constexpr int kTile1 = kCodes + kScales;
  static constexpr int kGroup = (kStagesK + kStagesV) * kTile1;
  static constexpr int kLdO = D + 4;                                     // floats
  static constexpr int kMerge = kWarps * kRows * kLdO * 4;               // the warps' outputs, over the stages
  static constexpr int kOffQ = 2 * kGroup > kMerge ? 2 * kGroup : (kMerge + 1023) / 1024 * 1024;
  static constexpr int kQ = kCols * D / 2;                               // one set of digits
  static constexpr int kOffP = kOffQ + 2 * kQ;                           // weights, [warp][32 tokens][rows] f16
  static constexpr int kOffStat = kOffP + kWarps * 32 * kRows * 2;       // m, l [warps][rows]
  static constexpr int kOffRow = kOffStat + 2 * kWarps * kRows * 4;      // rs, hi, lo, query, head [rows]
  static constexpr int kOffBar = kOffRow + 5 * kRows * 4;                // of a group: scores done, keys ready
  static constexpr int kOffPlan = kOffBar + 2 * 16 + 16;
  static constexpr int kSmem = kOffPlan + 128 + 2 * kWarps * 8 + 1024;    // + alignment slack
  static constexpr int kPart = kRows * (D + 2);                          // floats of one partial result
  static constexpr uint32_t kTmemCols = NT == 1 ? 128 : 256;
  static constexpr uint32_t kColSFA = 2 * kCols, kColSFB = kColSFA + 16; // + 8 * group; 4 each for both digit sets
  // kind::mxf4nvf4, E2M1, K-major, E4M3 scales, M = 128, N = kCols
  static constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | ((uint32_t)(kCols >> 3) << 17) | ((128u >> 4) << 24);
  static_assert(kColSFB + 8 <= kTmemCols, "tensor memory");
  static_assert(kSmem <= 113 * 1024, "two CTAs on an SM");
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

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Copies straight to shared memory: 16 bytes, or 4, of which n are read and
// the others written as zeros.
__device__ __forceinline__ void copy16(uint32_t dst, unsigned long long src, uint32_t n) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, unsigned long long src, uint32_t n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}

// m ? a : b, bit by bit
__device__ __forceinline__ uint32_t select_bits(uint32_t m, uint32_t a, uint32_t b) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xca;" : "=r"(d) : "r"(m), "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                     uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb) : "memory");
}

// K-major operand whose rows are D / 2 bytes, swizzled over that width: 64
// bytes (D = 128) or 32; 8-row groups follow one another.
template <int D>
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(8 * (D / 2) >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)(D == 128 ? 4 : 6) << 61);
}

// A 512-byte scale atom (32 rows of 16 bytes, no swizzle) as a copy source.
__device__ __forceinline__ uint64_t desc_sf(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

// Byte b of row n of such an operand: the swizzle exchanges 16-byte chunks.
template <int D>
__device__ __forceinline__ int row_chunk(int n) {
  return D == 128 ? (n >> 1) & 3 : (n >> 2) & 1;
}
template <int D>
__device__ __forceinline__ int row_at(int n, int b) {
  return n * (D / 2) + (((b >> 4) ^ row_chunk<D>(n)) << 4) + (b & 15);
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[N]) {
  static_assert(N % 32 == 0, "");
#pragma unroll
  for (int k = 0; k < N; k += 32)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
        "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[k]), "=r"(r[k + 1]), "=r"(r[k + 2]), "=r"(r[k + 3]), "=r"(r[k + 4]), "=r"(r[k + 5]), "=r"(r[k + 6]),
          "=r"(r[k + 7]), "=r"(r[k + 8]), "=r"(r[k + 9]), "=r"(r[k + 10]), "=r"(r[k + 11]), "=r"(r[k + 12]),
          "=r"(r[k + 13]), "=r"(r[k + 14]), "=r"(r[k + 15]), "=r"(r[k + 16]), "=r"(r[k + 17]), "=r"(r[k + 18]),
          "=r"(r[k + 19]), "=r"(r[k + 20]), "=r"(r[k + 21]), "=r"(r[k + 22]), "=r"(r[k + 23]), "=r"(r[k + 24]),
          "=r"(r[k + 25]), "=r"(r[k + 26]), "=r"(r[k + 27]), "=r"(r[k + 28]), "=r"(r[k + 29]), "=r"(r[k + 30]),
          "=r"(r[k + 31])
        : "r"(addr + k));
}

// The token of index r of the second product's 16 tokens: lane c's tokens
// (2c, 2c + 1, 2c + 8, 2c + 9) are c of each group of four, which spreads its
// reads of values over the banks.
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
  int first = 0, last = n - 1;
  if (n * a.group > ROWS) {
    first = fdiv(rt * ROWS, a.by_group);
    last = fdiv(min(n * a.group - 1, rt * ROWS + ROWS - 1), a.by_group);
  }
  s.hi = query_hi(a, n, len, last);
  s.lo = query_lo(a, query_hi(a, n, len, first));
  s.base = s.lo & ~(kSlice - 1);
  s.tiles = max(1, (s.hi - s.base + kTile - 1) / kTile);
  return s;
}

// a / b for a >= 0, b > 0, short where both fit 32 bits
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (long long)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// Work is counted in tiles, with kOver of them before each item's first for
// what it costs to begin one.  Share s of `shares` begins at s * base +
// min(s, rest); a share that begins in an item's kOver begins with its tile 0.
struct Split {
  long long base;
  int rest;
  __device__ __forceinline__ Split(long long total, int shares) {
    base = quotient(total, shares);
    rest = (int)(total - base * shares);
  }
  __device__ __forceinline__ long long first(int s) const { return base * s + min(s, rest); }
  // the share that holds x
  __device__ __forceinline__ int of(long long x) const {
    const long long big = (base + 1) * rest;
    return x < big ? (int)quotient(x, base + 1) : rest + (int)quotient(x - big, base);
  }
};

// A row tile of a sequence and a key/value head; start: where its work begins.
struct Item {
  int b, rt, h, q0, n, len, nrt;
  Span s;
  long long start;
};

template <int ROWS>
__device__ __forceinline__ bool load_sequence(const KvAttnArgs& a, int b, Item& it, bool& wrong) {
  const bool ordered = lengths_of(a, b, it.q0, it.n, it.len, wrong);
  it.b = b;
  it.nrt = (it.n * a.group + ROWS - 1) / ROWS;
  return ordered;
}

// The item after `it`; false behind the last.
template <int ROWS>
__device__ __forceinline__ bool next_item(const KvAttnArgs& a, Item& it) {
  it.start += it.s.tiles + kOver;
  if (++it.h < a.p.heads) return true;
  it.h = 0;
  if (++it.rt == it.nrt) {
    it.rt = 0;
    bool wrong;
    do {
      if (++it.b >= a.batch) return false;
      load_sequence<ROWS>(a, it.b, it, wrong);
    } while (it.nrt == 0);
  }
  it.s = span_of<ROWS>(a, it.n, it.len, it.rt);
  return true;
}

// Where a share of the work begins: all of it, the share's first, its item.
struct Plan {
  long long total, first;
  Item it;
};

// Every thread of the block takes part.  The item is set unless the share is
// empty; all are where the sequences have too many queries.  warp_sum: two
// numbers for each warp.
template <int ROWS>
__device__ __forceinline__ void make_plan(const KvAttnArgs& a, int share, int shares, Plan* plan, long long* warp_sum,
                                          bool tell) {
  const int tid = threadIdx.x, per = (a.batch + kThreads - 1) / kThreads;
  const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
  long long mine = 0, asked = 0;
  bool bad = false, ordered = true, wrong;
  Item it;
  for (int b = b0; b < b1 && asked <= a.total_q; ++b) {
    ordered &= load_sequence<ROWS>(a, b, it, wrong);
    bad |= wrong;
    asked += it.n;
    long long tiles = 0;
    for (int rt = 0; rt < it.nrt; ++rt) tiles += span_of<ROWS>(a, it.n, it.len, rt).tiles + kOver;
    mine += tiles * a.p.heads;
  }
  if (bad && tell && a.status) atomicOr(a.status, FOS_STATUS_INDEX);
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(~0u, upto, o);
    if ((tid & 31) >= o) upto += x;
  }
  if ((tid & 31) == 31) warp_sum[tid >> 5] = upto;
  const bool broken = __syncthreads_or(!ordered) && too_many(a, asked, warp_sum + kWarps);
  long long before = 0, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < (tid >> 5)) before += warp_sum[w];
    total += warp_sum[w];
  }
  upto += before;
  if (broken) total = upto = mine = 0;
  const long long first = Split(total, shares).first(share);
  if (tid == 0) { plan->total = total; plan->first = first; }
  if (first >= upto - mine && first < upto) {
    long long x = upto - mine;
    for (int b = b0; b < b1; ++b) {
      if (per > 1) load_sequence<ROWS>(a, b, it, wrong);
      for (int rt = 0; rt < it.nrt; ++rt) {
        it.s = span_of<ROWS>(a, it.n, it.len, rt);
        const int each = it.s.tiles + kOver;
        const long long all = (long long)each * a.p.heads;
        if (first >= x && first < x + all) {
          it.rt = rt;
          it.h = (int)quotient(first - x, each);
          it.start = x + (long long)it.h * each;
          plan->it = it;
        }
        x += all;
      }
    }
  }
  __syncthreads();
}

// One row of a finished item: values d .. d + 3 and (lane 0 of the row) lse.
// No weight, no output: o may be 0 * NaN where the cache holds one that only
// other rows see.
__device__ __forceinline__ void write_row(const KvAttnArgs& a, int h, int t, int hq, int d, int D, float4 o, float M,
                                          float L) {
  if (L == 0.0f) o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float f = L == 0.0f ? 0.0f : __fdividef(a.p.vst[h], L);
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
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kCtas)
    k_kv_decode(const KvAttnArgs a, float* part) {
  using C = Cfg<D, NT>;
  constexpr int R = C::kRows, MT = D / 16;           // rows; 16-value tiles of the output
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int grp = warp >> 2, wq = warp & 3;          // group, and which 32 tokens of its tile
  Plan* plan = reinterpret_cast<Plan*>(smem + C::kOffPlan);
  float* stat = reinterpret_cast<float*>(smem + C::kOffStat);
  float* row_rs = reinterpret_cast<float*>(smem + C::kOffRow);
  int *row_hi = reinterpret_cast<int*>(row_rs + R), *row_lo = row_hi + R;
  int *row_t = row_lo + R, *row_hq = row_t + R;     // -1 for a row that there is not
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffPlan - 16);
  const uint32_t bar_s = sbase + C::kOffBar + 16 * grp, bar_r = bar_s + 8;
  const uint32_t off_k = sbase + grp * C::kGroup, off_v = off_k + kStagesK * C::kTile1;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // The page table and the queries on their way to L2, a line for each thread
  // of the grid, while the plan is made: 48 windows of 1000 tokens 34 -> 32 us.
  {
    const long long at = ((long long)blockIdx.x * kThreads + tid) * 128;
    const long long table = (long long)a.batch * a.max_pages * 4;
    const long long queries = ((long long)(a.total_q - 1) * a.q_ld + (long long)a.q_heads * D) * 2;
    if (at < table) asm volatile("prefetch.global.L2 [%0];" :: "l"(reinterpret_cast<const char*>(a.pages) + at));
    if (at < queries) asm volatile("prefetch.global.L2 [%0];" :: "l"(reinterpret_cast<const char*>(a.q) + at));
    if (tid == 0) {
      asm volatile("prefetch.global.L2 [%0];" :: "l"(a.p.kst));
      asm volatile("prefetch.global.L2 [%0];" :: "l"(a.p.vst));
    }
  }
  static_assert(sizeof(Plan) <= 128, "plan");
  if (warp == kWarps - 1 && lane == 0) {
    for (int b = 0; b < 4; ++b)   // scores: one commit; ready: an arrival from each warp of the group
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(sbase + C::kOffBar + 8 * b), "r"(b & 1 ? 4 : 1)
                   : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarps - 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(tmem_slot)), "r"(C::kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  make_plan<R>(a, blockIdx.x, gridDim.x, plan, reinterpret_cast<long long*>(smem + C::kOffPlan + 128), blockIdx.x == 0);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  if (grp == 0) {   // the digit sets' scales: 2^-6 and 2^6 everywhere
    const uint32_t lo = 0x08080808u, hi = 0x68686868u;
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %1, %1, %1, %2, %2, %2, %2};"
                 :: "r"(tmem + ((uint32_t)(32 * wq) << 16) + C::kColSFB), "r"(lo), "r"(hi) : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  const long long first = plan->first, last = Split(plan->total, gridDim.x).first(blockIdx.x + 1);
  Item it = plan->it;
  uint32_t ph_s = 0, ph_r = 0;  // parities of the next scores and of the next keys
  // what a lane reads of a tile's values: tokens c, 4 + (c ^ 1) and both + 8, of 16 (row_token)
  const uint32_t v_at0 = c * (D / 2) + (D / 16) * g, v_at1 = (4 + (c ^ 1)) * (D / 2) + (D / 16) * g;
  const uint32_t vs_at0 = c * (D / 16) + g * D / 128, vs_at1 = (4 + (c ^ 1)) * (D / 16) + g * D / 128;
  const uint32_t p_at = sbase + C::kOffP + warp * 32 * R * 2;   // this warp's weights
  const uint32_t p_ld = p_at + row_token(lane & 15) * 16;
  // where a lane's copies go in a tile: keys' codes (swizzled) and scales, values' codes and scales
  const uint32_t k_at = (32 * wq + lane / (D / 32)) * (D / 2) +
                        (((lane & (D / 32 - 1)) ^ row_chunk<D>(lane / (D / 32))) << 4);
  const uint32_t ks_at = C::kCodes + 4 * wq + 512 * (lane & (D / 64 - 1)) + (lane / (D / 64)) * 16;
  const uint32_t w_at = 32 * wq * (D / 2) + lane * 16, ws_at = C::kCodes + 32 * wq * (D / 16) + lane * 16;
  bool dead = false;            // a wait gave up
  bool more = first < last;
  for (long long pos = first; more && pos < last; more = next_item<R>(a, it)) {
    const int ta = (int)max(0ll, pos - it.start - kOver), tb = (int)min((long long)it.s.tiles, last - it.start - kOver);
    if (tb <= ta) break;         // the share ends before the item's first tile
    const long long seg_pos = pos;
    pos = it.start + kOver + it.s.tiles;
    const int h = it.h;
    const int mine = (tb - ta + 1 - grp) / 2;          // this group's tiles: ta + grp + 2 i
    const int32_t* ids_row = a.pages + (long long)it.b * a.max_pages;
    auto token0 = [&](int i) { return it.s.base + (ta + grp + 2 * i) * kTile; };

    // ---- a warp copies its own 32 tokens of a tile, 16 from one page at a
    // time: the keys' codes into the swizzled operand, their scales into the
    // atoms that go to tensor memory, the values as they are.  Page ids come
    // 16 tiles at once, a lane for each 16 tokens, and one such window ahead.
    auto load_ids = [&](int i0) {
      const int i = i0 + (lane >> 1), tok = token0(i) + 32 * wq + kSlice * (lane & 1);
      int page = -1;
      if (i < mine && tok < it.s.hi) {
        page = __ldg(ids_row + (tok >> a.p.page_shift));
        if ((uint32_t)page >= (uint32_t)a.p.num_pages) {
          page = -1;
          if (a.status) atomicOr(a.status, FOS_STATUS_INDEX);
        }
      }
      return page;
    };
    int ids = load_ids(0), ids_next = mine > 16 ? load_ids(16) : -1;
    const uint32_t in_page = (1u << a.p.page_shift) - 1;
    // this head's part of page 0: a lane's bytes of the keys' codes, the keys' scales
    const unsigned long long kc0 = (unsigned long long)a.p.kc + ((uint32_t)h << a.p.page_shift) * (D / 2) + lane * 16;
    const unsigned long long ks0 = (unsigned long long)a.p.ks + ((uint32_t)h << a.p.page_shift) * (D / 16);
    // The next tile to copy, its 32 tokens' first, and where it goes; which 16
    // tokens of it (bits 0, 1) and of the tiles before it were copied.
    uint32_t copy_tok = (uint32_t)token0(0) + 32 * wq, copy_k = off_k, copy_v = off_v, copied = 0;
    int copy_i = 0;
    auto issue = [&]() {
      copied <<= 2;
      if (copy_i < mine) {
        if ((copy_i & 15) == 0 && copy_i > 0) {
          ids = ids_next;
          ids_next = load_ids(copy_i + 16);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int page = __shfl_sync(~0u, ids, (2 * copy_i & 30) + half);
          const uint32_t n = page >= 0 ? 16u : 0u, p = (uint32_t)max(page, 0);
          copied |= (n >> 4) << half;
          const uint32_t r = (copy_tok + kSlice * half) & in_page;
          const unsigned long long kp = (unsigned long long)p * a.p.codes_stride32 + (kc0 + r * (D / 2));
          const unsigned long long sp = (unsigned long long)p * a.p.scales_stride32 + (ks0 + r * (D / 16));
#pragma unroll
          for (int e = 0; e < D / 64; ++e) {           // 16 tokens: 512 bytes at a time
            copy16(copy_k + k_at + kSlice * half * (D / 2) + 512 * e, kp + 512 * e, n);
            copy16(copy_v + w_at + kSlice * half * (D / 2) + 512 * e, kp + a.p.kv_codes + 512 * e, n);
          }
          // key scales: token t, 4 scales a word, word k at 512 k + 16 (t mod 32) + 4 (t / 32)
          if (D == 128 || lane < 16) copy4(copy_k + ks_at + kSlice * half * 16, sp + 4 * lane, n >> 2);
          if (lane < D / 16) copy16(copy_v + ws_at + kSlice * half * (D / 16), sp + a.p.kv_scales + 16 * lane, n);
        }
        copy_tok += 2 * kTile;
        copy_k = 2 * off_k + C::kTile1 - copy_k;
        copy_v = copy_v == off_v + 2 * C::kTile1 ? off_v : copy_v + C::kTile1;
        ++copy_i;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // the queries of rows warp, warp + 8, .. are on their way while the page ids are
    constexpr int E = D / 32;                            // values of a lane
    const float base_scale = a.scale_log2 * __ldg(a.p.kst + h);
    uint32_t qw[NT][E / 2];
#pragma unroll
    for (int rr = 0; rr < NT; ++rr) {
      const int row = it.rt * R + warp + 8 * rr, i = (int)fdiv(row, a.by_group);
      const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q + (long long)(it.q0 + i) * a.q_ld +
                                                              (long long)(h * a.group + (row - i * a.group)) * D) +
                            lane * (E / 2);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) qw[rr][e] = row < it.n * a.group ? __ldg(src + e) : 0u;
    }
    issue();
    issue();

    // ---- their digits
#pragma unroll
    for (int rr = 0; rr < NT; ++rr) {
      const int r = warp + 8 * rr, row = it.rt * R + r;
      const bool live = row < it.n * a.group;
      float v[E];
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        v[2 * e] = bf_lo(qw[rr][e]);
        v[2 * e + 1] = bf_hi(qw[rr][e]);
      }
      uint32_t top = 0;          // |values| as bits: ordered like the values, NaN and Inf above all
#pragma unroll
      for (int e = 0; e < E; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
      top = __reduce_max_sync(~0u, top);
      const RowScale sc = row_scale(top);                // below 2^15; 2^8 more for the digits
      uint32_t digits[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) digits[k] = 0;
      // n = sum of d_k 8^k with d_k in -4 .. 3 (the last one -4 .. 4): the octal
      // digits of n + 4 (8^7 - 1) / 7 less 4.  Codes of four values at once:
      // a permute looks the digits up in a table of bytes.
      int n[E];
#pragma unroll
      for (int e = 0; e < E; ++e) n[e] = (sc.finite ? __float2int_rn(v[e] * sc.up1 * sc.up2 * 256.0f) : 0) + 1198372;
#pragma unroll
      for (int k = 0; k < 7; ++k) {
        uint32_t pick = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) pick |= (((uint32_t)n[e] >> (3 * k)) & 7u) << (4 * e);
        const uint32_t b = __byte_perm(0x090a0b0cu, 0x03020100u, pick);
        digits[k] = __byte_perm(b | b >> 4, 0u, 0x4420u);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int d = n[e] >> 21;
        digits[7] |= (uint32_t)(d < 0 ? 8 - d : d) << (4 * e);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint8_t* dst = smem + C::kOffQ + (k >> 2) * C::kQ + row_at<D>((k & 3) * R + r, lane * (E / 2));
        if (E == 4) *reinterpret_cast<uint16_t*>(dst) = (uint16_t)digits[k];
        else *dst = (uint8_t)digits[k];
      }
      if (lane == 0) {
        const int hi = live ? query_hi(a, it.n, it.len, (int)fdiv(row, a.by_group)) : 0;
        // a digit is twice its E2M1 value, the low set's scale is 2^-6: 2^7; and the 2^8 from above
        row_rs[r] = sc.finite ? base_scale * sc.down1 * sc.down2 * 0.5f : CUDART_NAN_F;
        row_hi[r] = live ? hi : 0;
        row_lo[r] = live ? query_lo(a, hi) : 0;
        const int i = live ? (int)fdiv(row, a.by_group) : 0;
        row_t[r] = live ? it.q0 + i : -1;
        row_hq[r] = h * a.group + (row - i * a.group);
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    int min_hi = 0x7fffffff, max_lo = 0;
    {
      const int r = lane & (R - 1);
      if (it.rt * R + r < it.n * a.group) {
        min_hi = row_hi[r];
        max_lo = row_lo[r];
      }
      min_hi = __reduce_min_sync(~0u, min_hi);
      max_lo = __reduce_max_sync(~0u, max_lo);
    }

    // This thread's token is 32 wq + lane of the tile.  off = kLift - m, with m
    // the maximum of a row, the same in all lanes; l: sums of this lane's tokens.
    float2 rs[R / 2], off[R / 2], l[R / 2];
    float acc[MT][NT][4];
#pragma unroll
    for (int r = 0; r < R / 2; ++r) {
      rs[r] = make_float2(row_rs[2 * r], row_rs[2 * r + 1]);
      off[r] = make_float2(kLift - kNone, kLift - kNone);
      l[r] = make_float2(0.0f, 0.0f);
    }
#pragma unroll
    for (int k = 0; k < MT; ++k)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[k][nt][e] = 0.0f;

    // ---- the scores of tile i into tensor memory: every warp says when its
    // keys have landed and the scores before them have been read; warp i mod 4
    // waits for that and issues the products
    auto ready = [&]() {
      asm volatile("cp.async.wait_group 1;" ::: "memory");     // all tiles' copies but the newest's
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      asm volatile(
          "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %1, 0;\n\t"
          "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}"
          :: "r"(bar_r), "r"(lane) : "memory");
    };
    auto scores = [&](int i) {
      if (wq == (i & 3)) {
        if (!dead && !__all_sync(~0u, mbar_wait(bar_r, ph_r))) dead = true;
        if (lane == 0) {
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t sfa = tmem + C::kColSFA + 8 * grp, d = tmem + C::kCols * grp;
          const uint32_t k0 = off_k + (i & 1) * C::kTile1;
#pragma unroll
          for (int k = 0; k < D / 64; ++k)
            asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;"
                         :: "r"(sfa + 4 * k), "l"(desc_sf(k0 + C::kCodes + 512 * k)) : "memory");
#pragma unroll
          for (int set = 0; set < 2; ++set)
#pragma unroll
            for (int k = 0; k < D / 64; ++k)
              umma(d, desc_rows<D>(k0 + 32 * k), desc_rows<D>(sbase + C::kOffQ + set * C::kQ + 32 * k), C::kIdesc,
                   sfa + 4 * k, tmem + C::kColSFB + 4 * set, set | k);
          asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                       :: "r"(bar_s) : "memory");
        }
        __syncwarp();
      }
      ph_r ^= 1;
    };
    if (mine > 0) {
      ready();
      scores(0);
    }
    int sv = 0;                  // stage of this tile's values

#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
      // after a wait that gave up a warp waits no more
      if (!dead && !__all_sync(~0u, mbar_wait(bar_s, ph_s))) dead = true;
      ph_s ^= 1;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      uint32_t s[C::kCols];
      tmem_ld(tmem + C::kCols * grp + ((uint32_t)(32 * wq) << 16), s);
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
      float2 y[R / 2];           // the scores, before their row's scale
#pragma unroll
      for (int r = 0; r < R / 2; ++r) {
        auto col = [&](int j) {
          return make_float2(__uint_as_float(s[j * R + 2 * r]), __uint_as_float(s[j * R + 2 * r + 1]));
        };
        const float2 e8 = make_float2(8.0f, 8.0f);
        y[r] = fma2(fma2(fma2(col(3), e8, col(2)), e8, col(1)), e8, col(0));
      }
      // the keys of tile i have been read, this warp's values of tile i - 1 too
      issue();
      if (i + 1 < mine) ready();

      // ---- softmax
      const int tok0 = token0(i) + 32 * wq;
      const uint32_t live = copied >> 4;       // two tiles were issued after this one
      const bool edge = tok0 + 32 > min_hi || tok0 < max_lo || (live & 3u) != 3u;
      float2 x[R / 2];
      float over = -CUDART_INF_F;
#pragma unroll
      for (int r = 0; r < R / 2; ++r) x[r] = fma2(y[r], rs[r], off[r]);
      if (edge) {
        __syncwarp();            // a branch, not predicates: few tiles come here
        const int tok = tok0 + lane;
        const bool held = tok >= it.s.lo && tok < it.s.hi && ((live >> (lane >> 4)) & 1u);
#pragma unroll
        for (int r = 0; r < R / 2; ++r) {
          if (!held || tok >= row_hi[2 * r] || tok < row_lo[2 * r]) x[r].x = -CUDART_INF_F;
          if (!held || tok >= row_hi[2 * r + 1] || tok < row_lo[2 * r + 1]) x[r].y = -CUDART_INF_F;
        }
        // what lies outside the rows' tokens may be anything, NaN too: its scales become 0
        if (!held) {
#pragma unroll
          for (int k = 0; k < D / 64; ++k)
            *reinterpret_cast<uint32_t*>(smem + (off_v - sbase) + sv * C::kTile1 + C::kCodes +
                                         (32 * wq + lane) * (D / 16) + 4 * k) = 0;
        }
      }
#pragma unroll
      for (int r = 0; r < R / 2; ++r) over = fmaxf(over, fmaxf(x[r].x, x[r].y));
      if (__any_sync(~0u, over > kLift + kSlack)) {
        float keep0[NT], keep1[NT];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float& o = (r & 1) ? off[r / 2].y : off[r / 2].x;
          float& lr = (r & 1) ? l[r / 2].y : l[r / 2].x;
          float& xr = (r & 1) ? x[r / 2].y : x[r / 2].x;
          const float rsr = (r & 1) ? rs[r / 2].y : rs[r / 2].x, yr = (r & 1) ? y[r / 2].y : y[r / 2].x;
          const bool masked = xr == -CUDART_INF_F;
          float t = masked ? kNone : yr * rsr;
#pragma unroll
          for (int o2 = 16; o2; o2 >>= 1) t = fmaxf(t, __shfl_xor_sync(~0u, t, o2));
          const float was = o, keep = kLift - t < was ? ex2(kLift - t - was) : 1.0f;
          if (kLift - t < was) o = kLift - t;
          lr *= keep;
          if (!masked) xr = fmaf(yr, rsr, o);
          if (2 * c == (r & 7)) keep0[r >> 3] = keep;
          if (2 * c + 1 == (r & 7)) keep1[r >> 3] = keep;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < MT; ++k) {
            acc[k][nt][0] *= keep0[nt];
            acc[k][nt][1] *= keep1[nt];
            acc[k][nt][2] *= keep0[nt];
            acc[k][nt][3] *= keep1[nt];
          }
      }
      // the weights of 8 rows of a token are 16 bytes, [row tile][token]
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t ph[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 p = make_float2(ex2(x[4 * nt + e].x), ex2(x[4 * nt + e].y));
          l[4 * nt + e] = add2(l[4 * nt + e], p);
          ph[e] = pack_h2(p.x, p.y);
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                     :: "r"(p_at + nt * 512 + lane * 16), "r"(ph[0]), "r"(ph[1]), "r"(ph[2]), "r"(ph[3]) : "memory");
      }
      __syncwarp();

      // ---- output (the wait for this tile's keys was one for its values too)
      const uint32_t vbase = off_v + sv * C::kTile1 + 32 * wq * (D / 2);
      const uint32_t sbase_v = off_v + sv * C::kTile1 + C::kCodes + 32 * wq * (D / 16);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (half == 1 && i + 1 < mine) scores(i + 1);   // by now the other warps are ready as a rule
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
                       : "=r"(pf[nt][0]), "=r"(pf[nt][1]) : "r"(p_ld + nt * 512 + 256 * half) : "memory");
        constexpr int VW = D / 64;             // words of a token in a lane: 8 VW values from 8 VW g on
        uint32_t w[4][VW], sc[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t at = (t & 1 ? v_at1 : v_at0) + vbase + (16 * half + 8 * (t >> 1)) * (D / 2);
          if (VW == 2) {
            const uint2 y = lds64(at);
            w[t][0] = y.x;
            w[t][VW - 1] = y.y;
          } else {
            w[t][0] = lds32(at);
          }
          sc[t] = lds8((t & 1 ? vs_at1 : vs_at0) + sbase_v + (16 * half + 8 * (t >> 1)) * (D / 16));
        }
        const uint32_t s01 = scales_h2(sc[0] | sc[1] << 8), s23 = scales_h2(sc[2] | sc[3] << 8);
#pragma unroll
        for (int v = 0; v < VW; ++v) {
          const uint32_t e01 = select_bits(0x0f0f0f0fu, w[0][v], w[1][v] << 4);
          const uint32_t o01 = select_bits(0x0f0f0f0fu, w[0][v] >> 4, w[1][v]);
          const uint32_t e23 = select_bits(0x0f0f0f0fu, w[2][v], w[3][v] << 4);
          const uint32_t o23 = select_bits(0x0f0f0f0fu, w[2][v] >> 4, w[3][v]);
          uint32_t he01[4], ho01[4], he23[4], ho23[4];
          codes_h2x4(e01, he01);
          codes_h2x4(o01, ho01);
          codes_h2x4(e23, he23);
          codes_h2x4(o23, ho23);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t a0 = hmul2(he01[q], s01), a1 = hmul2(ho01[q], s01);
            const uint32_t a2 = hmul2(he23[q], s23), a3 = hmul2(ho23[q], s23);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma(acc[4 * v + q][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
          }
        }
      }
      __syncwarp();              // the values' stage and the weights may be written again
      sv = sv == 2 ? 0 : sv + 1;
    }

    // ---- join the warps' results through shared memory (over the stages: their copies have all landed)
    __syncthreads();
    float* om = reinterpret_cast<float*>(smem);
    // the sums over the lanes: each step halves the rows that a lane holds
    float ls[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      ls[r] = (r & 1) ? l[r / 2].y : l[r / 2].x;
      if (lane == r) stat[warp * R + r] = kLift - ((r & 1) ? off[r / 2].y : off[r / 2].x);
    }
#pragma unroll
    for (int mask = 16, left = R; mask; mask >>= 1) {
      if (left > 1) {
        left /= 2;
#pragma unroll
        for (int r = 0; r < left; ++r) {
          const float other = __shfl_xor_sync(~0u, lane & mask ? ls[r] : ls[r + left], mask);
          ls[r] = (lane & mask ? ls[r + left] : ls[r]) + other;
        }
      } else {
        ls[0] += __shfl_xor_sync(~0u, ls[0], mask);
      }
    }
    constexpr int kShift = NT == 1 ? 2 : 1;    // lane bits that no row needed
    if ((lane & ((1 << kShift) - 1)) == 0) stat[(kWarps + warp) * R + (lane >> kShift)] = ls[0];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        float* dst = om + (warp * R + 8 * nt + 2 * c + k2) * C::kLdO + (D / 8) * g;
#pragma unroll
        for (int i = 0; i < MT; ++i)
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
        if (row_t[r] >= 0) write_row(a, h, row_t[r], row_hq[r], d, D, o, M, L);
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
  }
  if (dead) {                    // let this warp's products finish before the tensor memory is freed
    if (lane == 0) {
      const uint32_t bar_d = sbase + C::kOffPlan + 128 + 8 * warp;   // the plan's sums, long read
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" :: "r"(bar_d) : "memory");
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                   :: "r"(bar_d) : "memory");
      mbar_wait(bar_d, 0);
      if (a.status) atomicOr(a.status, FOS_STATUS_TIMEOUT);
    }
    __syncwarp();
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == kWarps - 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(C::kTmemCols) : "memory");
  }
}

// Joins an item that several shares hold (3 us for one of 1000 tokens, begun
// before k_kv_decode has ended so that its plan costs nothing): the CTAs of those shares (but one
// that the item only ends) take its rows in turn.  The warps of a CTA take a
// row each, or several share a row's partial results; every sum is in the
// order of the tokens within a warp and over the warps in theirs.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads) k_kv_join(const KvAttnArgs a, const float* part) {
  using C = Cfg<D, NT>;
  constexpr int R = C::kRows;
  __shared__ Plan plan;
  __shared__ long long sums[2 * kWarps];
  __shared__ float4 s_o[kWarps][D / 4];
  __shared__ float2 s_ml[kWarps];
  make_plan<R>(a, blockIdx.x, gridDim.x, &plan, sums, false);
  const Split split(plan.total, gridDim.x);
  const long long first = plan.first, last = split.first(blockIdx.x + 1);
  const Item it = plan.it;
  bool mine = first < last;
  int c0 = 0, c1 = 0, lead = 0;
  if (mine) {
    c0 = split.of(it.start + kOver);
    c1 = split.of(it.start + kOver + it.s.tiles - 1);
    lead = split.first(c0) < it.start ? c0 + 1 : c0;   // the first share that begins with this item or inside it
    mine = c1 > c0 && (int)blockIdx.x >= lead;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!mine) return;
  const int ctas = c1 - lead + 1, n = c1 - c0 + 1;     // CTAs on the item, its partial results
  const int rows = (R + ctas - 1) / ctas;              // of this CTA: r = blockIdx.x - lead + ctas * k
  const int wide = rows >= 8 ? 8 : rows > 2 ? 4 : rows;   // rows at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int teams = kWarps / wide, team = warp / wide;
  const float* p0 = part + (long long)(2 * c0 + (lead > c0 ? 1 : 0)) * C::kPart;
  for (int k0 = 0; k0 < rows; k0 += wide) {
    const int r = blockIdx.x - lead + ctas * (k0 + warp % wide);
    const bool live = r < R && it.rt * R + r < it.n * a.group;
    float M = -CUDART_INF_F, L = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (live && lane < D / 4) {
#pragma unroll 4
      for (int s = team; s < n; s += teams) {
        const float* p = s ? part + (long long)(2 * (c0 + s)) * C::kPart : p0;
        const float4 v = *reinterpret_cast<const float4*>(p + r * D + 4 * lane);
        const float pm = p[R * D + r], pl = p[R * D + R + r], top = fmaxf(M, pm);
        const float f = M == top ? 1.0f : ex2(M - top), k = pm == top ? 1.0f : ex2(pm - top);
        L = L * f + pl * k;
        o.x = o.x * f + v.x * k; o.y = o.y * f + v.y * k; o.z = o.z * f + v.z * k; o.w = o.w * f + v.w * k;
        M = top;
      }
      s_o[warp][lane] = o;
      if (lane == 0) s_ml[warp] = make_float2(M, L);
    }
    __syncthreads();
    if (live && team == 0 && lane < D / 4) {
      for (int t = 1; t < teams && t < n; ++t) {
        const float2 ml = s_ml[warp + t * wide];
        const float4 v = s_o[warp + t * wide][lane];
        const float top = fmaxf(M, ml.x);
        const float f = M == top ? 1.0f : ex2(M - top), k = ml.x == top ? 1.0f : ex2(ml.x - top);
        L = L * f + ml.y * k;
        o.x = o.x * f + v.x * k; o.y = o.y * f + v.y * k; o.z = o.z * f + v.z * k; o.w = o.w * f + v.w * k;
        M = top;
      }
      const int row = it.rt * R + r, i = (int)fdiv(row, a.by_group);
      write_row(a, it.h, it.q0 + i, it.h * a.group + (row - i * a.group), 4 * lane, D, o, M, L);
    }
    __syncthreads();
  }
}

template <int D, int NT>
cudaError_t launch(const KvAttnArgs& a, float* part, cudaStream_t st) {
  using C = Cfg<D, NT>;
  static KvDevices devices;
  int sms = 0;
  cudaError_t e = devices.get((const void*)k_kv_decode<D, NT>, C::kSmem, &sms);
  if (e != cudaSuccess) return e;
  const int ctas = C::kCtas * sms < kMaxCtas ? C::kCtas * sms : kMaxCtas;
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

// More than 8 rows take one tile of 16 (one CTA on an SM) rather than two of 8
// that read the cache twice.  16 rows, 8 heads of 128, us: 32 ragged contexts of
// up to 16384 tokens 119 against 148, 16 of 4000 45 / 52, 16 of 1000 29 / 27, 64
// of 300 45 / 45.
cudaError_t launch_kv_decode(const KvAttnArgs& a, int rows, float* part, cudaStream_t st) {
  if (a.p.dim == 128) return rows <= 8 ? launch<128, 1>(a, part, st) : launch<128, 2>(a, part, st);
  return rows <= 8 ? launch<64, 1>(a, part, st) : launch<64, 2>(a, part, st);
}

}  // namespace fos
