// fos_kv_api.cu -- the C ABI of the key/value cache (argument checks, launch
// descriptors).  Declarations and semantics: include/fos.h.
#include <math.h>

#include "fos.h"
#include "fos_internal.h"
#include "fos_kv.h"

namespace fos {
namespace {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

fos_status check_pool(const fos_kv_cache* c, KvPool* p) {
  if (!c) return FOS_ERR_NULL;
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || !c->k_tensor_scale || !c->v_tensor_scale)
    return FOS_ERR_NULL;
  if (c->head_dim != 64 && c->head_dim != 128) return FOS_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return FOS_ERR_UNSUPPORTED;
  if (c->num_pages < 0 || c->num_pages > 0x7fffffff || c->heads < 1 || c->heads > 1024) return FOS_ERR_SHAPE;
  const int64_t rows = c->heads * c->page_size;
  if (c->codes_page_stride < rows * (c->head_dim / 2) || c->scales_page_stride < rows * (c->head_dim / 16))
    return FOS_ERR_SHAPE;
  if (c->codes_page_stride > 0xffffffffll || c->scales_page_stride > 0xffffffffll) return FOS_ERR_SHAPE;
  if (c->codes_page_stride % 16 || c->scales_page_stride % 16) return FOS_ERR_ALIGN;
  if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) ||
      !aligned(c->v_scales, 16) || !aligned(c->k_tensor_scale, 4) || !aligned(c->v_tensor_scale, 4))
    return FOS_ERR_ALIGN;
  p->kc = c->k_codes;
  p->ks = c->k_scales;
  p->vc = c->v_codes;
  p->vs = c->v_scales;
  p->kst = c->k_tensor_scale;
  p->vst = c->v_tensor_scale;
  p->codes_stride = c->codes_page_stride;
  p->scales_stride = c->scales_page_stride;
  p->codes_stride32 = (uint32_t)c->codes_page_stride;
  p->scales_stride32 = (uint32_t)c->scales_page_stride;
  p->kv_codes = (long long)((uintptr_t)c->v_codes - (uintptr_t)c->k_codes);
  p->kv_scales = (long long)((uintptr_t)c->v_scales - (uintptr_t)c->k_scales);
  p->num_pages = c->num_pages;
  p->page_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  p->heads = (int)c->heads;
  p->dim = (int)c->head_dim;
  return FOS_OK;
}

// rows of `heads` heads, `ld` elements apart
fos_status check_rows(const void* x, int64_t ld, int64_t heads, int64_t dim) {
  if (!aligned(x, 16) || ld % 8) return FOS_ERR_ALIGN;
  if (ld < heads * dim) return FOS_ERR_SHAPE;
  return FOS_OK;
}

// Which kernel a call of fos_kv_attention runs, from what the host knows.
// The kernel for few queries reads a sequence's cache again for every 16 rows
// (queries times heads of a group) but cuts the tokens as finely as it takes
// to fill the SMs; the one for many takes 256 rows at a time, computes 128
// whatever there are, and gives each CTA 512 tokens at least.  Measured (us,
// few / many, captured calls with nothing in L2) by sequences times heads, on
// each side of the rule; head_dim 128, then 64:
//     2,  4000 tokens: 128 rows 25 / 27, 256 rows 27 / 33;  23 / 23, 25 / 27
//     2, 16000 tokens: 128 rows 31 / 39, 256 rows 45 / 43;  29 / 33, 39 / 37
//     8,  4000 tokens:  64 rows 25 / 25,  96 rows 31 / 27;  23 / 23, 27 / 23
//     8, 16000 tokens:  64 rows 43 / 39,  96 rows 55 / 41;  37 / 35, 47 / 35
//    16,  4000 tokens:  32 rows 25 / 27,  48 rows 31 / 27;  23 / 23, 27 / 23
//    16,   500 tokens:  32 rows 20 / 23,  48 rows 20 / 23;  18 / 18, 20 / 18
//    64,  4000 tokens:  32 rows 47 / 49,  48 rows 59 / 49;  41 / 41, 51 / 41
//    64,   500 tokens:  32 rows 25 / 23,  48 rows 31 / 23;  23 / 18, 29 / 18
//   256,  4000 tokens:  32 rows 129 / 143, 48 rows 180 / 143; 106 / 115, 150 / 115
//   256,   500 tokens:  32 rows 47 / 41,  48 rows 62 / 41;  41 / 33, 53 / 33
// Over short tables 32 rows of many sequences would do better with the kernel
// for many, by a tenth to a quarter: the rule does not look at the lengths, which
// only the device knows (a table's width bounds them, and is often far above them).
// It is one choice for the call: see the note on max_q in fos.h.
struct AttnPlan {
  bool many;
  int rows, splits;
  size_t bytes;
};

AttnPlan attn_plan(const fos_kv_cache* c, int64_t total_q, int64_t batch, int64_t q_heads, int64_t max_q,
                   int64_t max_kv) {
  AttnPlan p{};
  const int64_t group = q_heads / c->heads, rows = max_q * group, items = batch * c->heads;
  p.many = rows > 32 && rows > 512 / (items > 0 ? items : 1) && kv_prompt_fits(total_q, batch, group, c->heads);
  if (p.many) {
    p.splits = kv_prompt_splits(total_q, batch, group, c->heads, max_q, max_kv);
    p.bytes = kv_prompt_workspace_bytes((int)c->head_dim, p.splits, total_q * q_heads);
  } else {
    p.rows = rows > 16 ? 16 : (int)rows;
    p.bytes = kv_decode_workspace_bytes((int)c->head_dim, p.rows);
  }
  return p;
}

}  // namespace
}  // namespace fos

using namespace fos;

extern "C" {

fos_status fos_kv_append(const fos_kv_cache* cache, int32_t fmt, const void* k, int64_t k_ld, const void* v,
                         int64_t v_ld, int64_t tokens, const int64_t* slots, const fos_rotary* rot,
                         const void* q, int64_t q_ld, void* q_out, int64_t q_out_ld, int64_t q_heads,
                         uint32_t* status, void* stream) {
  KvAppendArgs a{};
  fos_status e = check_pool(cache, &a.p);
  if (e != FOS_OK) return e;
  if (fmt < 0 || fmt > 2) return FOS_ERR_ARG;
  if (fmt == FOS_FMT_MXFP4) return FOS_ERR_UNSUPPORTED;
  if (tokens < 0 || tokens > (1 << 30)) return FOS_ERR_SHAPE;
  if (tokens == 0) return FOS_OK;  // buffers of no tokens may be NULL
  if (!k || !v || !slots) return FOS_ERR_NULL;
  if ((q != nullptr) != (q_out != nullptr)) return FOS_ERR_NULL;
  if (q && !rot) return FOS_ERR_ARG;
  if ((e = check_rows(k, k_ld, a.p.heads, a.p.dim)) != FOS_OK) return e;
  if ((e = check_rows(v, v_ld, a.p.heads, a.p.dim)) != FOS_OK) return e;
  if (!aligned(slots, 8)) return FOS_ERR_ALIGN;
  if (rot) {
    if (!rot->table || !rot->positions) return FOS_ERR_NULL;
    if (rot->dim < 16 || rot->dim % 16 || rot->dim > a.p.dim || rot->max_positions < 0) return FOS_ERR_SHAPE;
    if (rot->interleaved != 0 && rot->interleaved != 1) return FOS_ERR_ARG;
    if (!aligned(rot->table, 16) || !aligned(rot->positions, 4)) return FOS_ERR_ALIGN;
    a.table = rot->table;
    a.positions = rot->positions;
    a.max_positions = rot->max_positions;
    a.rot = rot->dim;
  }
  if (q) {
    if (q_heads < 1 || q_heads > 65536) return FOS_ERR_SHAPE;
    if ((e = check_rows(q, q_ld, q_heads, a.p.dim)) != FOS_OK) return e;
    if ((e = check_rows(q_out, q_out_ld, q_heads, a.p.dim)) != FOS_OK) return e;
    a.q = (const uint16_t*)q;
    a.q_out = (uint16_t*)q_out;
    a.q_heads = (int)q_heads;
  }
  a.k = (const uint16_t*)k;
  a.v = (const uint16_t*)v;
  a.k_ld = k_ld;
  a.v_ld = v_ld;
  a.q_ld = q_ld;
  a.q_out_ld = q_out_ld;
  a.slots = slots;
  a.tokens = (int)tokens;
  a.status = status;
  return launch_kv_append(a, fmt, rot && rot->interleaved, (cudaStream_t)stream) == cudaSuccess ? FOS_OK
                                                                                                : FOS_ERR_CUDA;
}

fos_status fos_kv_read(const fos_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k, void* v,
                       uint32_t* status, void* stream) {
  KvReadArgs a{};
  const fos_status e = check_pool(cache, &a.p);
  if (e != FOS_OK) return e;
  if (tokens < 0 || tokens > (1 << 30)) return FOS_ERR_SHAPE;
  if (tokens == 0) return FOS_OK;
  if (!slots || !k || !v) return FOS_ERR_NULL;
  if (!aligned(slots, 8) || !aligned(k, 16) || !aligned(v, 16)) return FOS_ERR_ALIGN;
  a.slots = slots;
  a.tokens = (int)tokens;
  a.k = (uint16_t*)k;
  a.v = (uint16_t*)v;
  a.status = status;
  return launch_kv_read(a, (cudaStream_t)stream) == cudaSuccess ? FOS_OK : FOS_ERR_CUDA;
}

size_t fos_kv_attention_workspace_size(const fos_kv_cache* cache, int64_t total_q, int64_t batch, int64_t q_heads,
                                       int64_t max_q, int64_t max_pages) {
  if (!cache || cache->heads < 1 || q_heads < cache->heads || q_heads > 65536 || total_q < 1 || total_q > (1 << 30) ||
      batch < 1 || batch > (1 << 20) || max_q < 0 || max_q > (1 << 30) || max_pages < 0 ||
      max_pages > (1ll << 31) || cache->page_size < 1 || cache->page_size > 128)
    return 0;
  return attn_plan(cache, total_q, batch, q_heads, max_q, max_pages * cache->page_size).bytes;
}

fos_status fos_kv_attention(const fos_kv_cache* cache, const void* q, int64_t q_ld, int64_t total_q,
                            int64_t q_heads, const int32_t* cu_q, int64_t batch, const int32_t* pages,
                            int64_t max_pages, const int32_t* kv_len, int64_t max_q, float scale, int32_t causal,
                            int64_t window, void* out, int64_t out_ld, float* lse, void* workspace,
                            size_t workspace_bytes, uint32_t* status, void* stream) {
  KvAttnArgs a{};
  fos_status e = check_pool(cache, &a.p);
  if (e != FOS_OK) return e;
  if (causal != 0 && causal != 1) return FOS_ERR_ARG;
  if (window < 0 || (window && !causal) || max_q < 0 || max_q > (1 << 30) || !isfinite(scale))
    return FOS_ERR_ARG;
  if (total_q < 0 || total_q > (1 << 30) || batch < 0 || batch > (1 << 20) || max_pages < 0) return FOS_ERR_SHAPE;
  if (q_heads < 1 || q_heads > 65536 || q_heads % a.p.heads) return FOS_ERR_SHAPE;
  // rows and tokens are 32-bit in the kernels, which count up to the end of a tile of rows, and some 8500
  // tokens past the last one of a sequence (page ids are asked for up to 32 tiles of a group ahead)
  if (total_q * (q_heads / a.p.heads) >= (1ll << 31) - 512 || max_pages > ((1ll << 31) - 65536) / cache->page_size)
    return FOS_ERR_SHAPE;
  if (batch == 0 || total_q == 0) return FOS_OK;  // buffers of nothing may be NULL
  if (!q || !cu_q || (!pages && max_pages) || !kv_len || !out) return FOS_ERR_NULL;
  if ((e = check_rows(q, q_ld, q_heads, a.p.dim)) != FOS_OK) return e;
  if ((e = check_rows(out, out_ld, q_heads, a.p.dim)) != FOS_OK) return e;
  if (!aligned(cu_q, 4) || !aligned(pages, 4) || !aligned(kv_len, 4) || (lse && !aligned(lse, 4)))
    return FOS_ERR_ALIGN;
  const AttnPlan plan = attn_plan(cache, total_q, batch, q_heads, max_q, max_pages * cache->page_size);
  if (plan.bytes) {
    if (!workspace || workspace_bytes < plan.bytes) return FOS_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return FOS_ERR_ALIGN;
  }
  a.q = (const uint16_t*)q;
  a.out = (uint16_t*)out;
  a.lse = lse;
  a.q_ld = q_ld;
  a.out_ld = out_ld;
  a.cu_q = cu_q;
  a.pages = pages;
  a.kv_len = kv_len;
  a.max_pages = max_pages;
  a.total_q = (int)total_q;
  a.batch = (int)batch;
  a.q_heads = (int)q_heads;
  a.group = (int)(q_heads / a.p.heads);
  a.by_group = make_fastdiv((uint32_t)a.group);
  a.causal = causal;
  a.window = window;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.status = status;
  const cudaError_t ce = plan.many ? launch_kv_prompt(a, plan.splits, (float*)workspace, (cudaStream_t)stream)
                                   : launch_kv_decode(a, plan.rows, (float*)workspace, (cudaStream_t)stream);
  return ce == cudaSuccess ? FOS_OK : FOS_ERR_CUDA;
}

}  // extern "C"
