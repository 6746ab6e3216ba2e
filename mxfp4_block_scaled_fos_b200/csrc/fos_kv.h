// fos_kv.h -- launch descriptors of the key/value cache's kernels (host
// side; no device code).  Semantics: include/fos.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "fos.h"
#include "fos_internal.h"

namespace fos {

// The pools of one cache; strides in bytes.
struct KvPool {
  uint8_t *kc, *ks, *vc, *vs;
  const float *kst, *vst;
  long long codes_stride, scales_stride;  // between pages, below 2^32
  uint32_t codes_stride32, scales_stride32;
  long long kv_codes, kv_scales;          // from the keys' pools to the values'
  long long num_pages;
  int page_shift;                         // log2(page_size)
  int heads, dim;
};

struct KvAppendArgs {
  KvPool p;
  const uint16_t *k, *v, *q;              // q nullable
  uint16_t* q_out;
  long long k_ld, v_ld, q_ld, q_out_ld;
  const int64_t* slots;
  const float* table;                     // nullable: no rotation
  const int32_t* positions;
  long long max_positions;
  int rot, tokens, q_heads;
  uint32_t* status;
  float neg_zero = -0.0f;                 // opaque -0 (see QuantArgs)
};

struct KvReadArgs {
  KvPool p;
  const int64_t* slots;
  int tokens;
  int token0;                             // of this launch
  uint16_t *k, *v;
  uint32_t* status;
};

struct KvAttnArgs {
  KvPool p;
  const uint16_t* q;
  uint16_t* out;
  float* lse;                             // nullable
  long long q_ld, out_ld;
  const int32_t *cu_q, *pages, *kv_len;
  long long max_pages;
  int total_q, batch, q_heads, group;     // group = q_heads / heads
  FastDiv by_group;                       // rows are below 2^31
  int causal;
  long long window;                       // 0: none
  float scale_log2;                       // scale * log2(e)
  uint32_t* status;
};

// What a launch asks of the current device, asked once for each: the SMs, and
// a kernel's shared memory above the default.
struct KvDevices {
  std::atomic<int> sms[64] = {};
  cudaError_t get(const void* kernel, int smem, int* out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int n = dev < 64 ? sms[dev].load(std::memory_order_acquire) : 0;
    if (n == 0) {
      if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
          (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
        return e;
      if (dev < 64) sms[dev].store(n, std::memory_order_release);
    }
    *out = n;
    return cudaSuccess;
  }
};

cudaError_t launch_kv_append(const KvAppendArgs& a, int fmt, bool interleaved, cudaStream_t st);
cudaError_t launch_kv_read(const KvReadArgs& a, cudaStream_t st);
// few queries; rows: the largest number of rows (queries times heads of a
// group) of a sequence, which chooses the row tile
size_t kv_decode_workspace_bytes(int dim, int rows);
cudaError_t launch_kv_decode(const KvAttnArgs& a, int rows, float* part, cudaStream_t st);
// many queries; splits: CTAs that share the tokens of 256 rows
int kv_prompt_splits(long long total_q, long long batch, long long group, long long heads, long long max_q,
                     long long max_kv);
bool kv_prompt_fits(long long total_q, long long batch, long long group, long long heads);   // in a grid
size_t kv_prompt_workspace_bytes(int dim, int splits, long long rows);
cudaError_t launch_kv_prompt(const KvAttnArgs& a, int splits, float* part, cudaStream_t st);

}  // namespace fos
