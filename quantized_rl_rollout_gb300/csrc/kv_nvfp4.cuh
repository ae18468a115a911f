// The paged NVFP4 key/value cache: its device view, the mapping from a call's
// rows to cache slots, and the launchers of its kernels (kv_nvfp4.cu,
// attention_nvfp4.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "attention_nvfp4_items.cuh"
#include "common.cuh"

namespace qrr {

// Pages [num_pages][Hkv][page] of rows; a row is D / 2 code bytes and D / 16
// scale bytes.  Token p of sequence b lives in page table[b][p / page], slot
// p % page (page a power of two of at least 16, so an aligned group of 16
// tokens never crosses pages).
struct KvNvfp4 {
  uint8_t *kc, *ks, *vc, *vs;
  const float *kg, *vg;  // [Hkv] global scales, null: 1
  const int32_t* table;  // [B][max_pages]
  int num_pages, Hkv, page_shift, D, B, max_pages;
  __host__ __device__ int64_t capacity() const { return static_cast<int64_t>(max_pages) << page_shift; }
};

// A call's rows: sequence b brings rows cu[b] .. cu[b + 1] - 1 (row b alone
// where cu is null), row cu[b] + i at position pos[b] + i.
struct KvRows {
  const int32_t* cu;
  const int32_t* pos;
  int64_t T;
};

// First row and number of rows of sequence b, clamped to the call's rows.
// Returns false if the offsets had to be clamped.
__device__ __forceinline__ bool kv_rows_of(const KvRows& r, int b, int& first, int& n) {
  if (!r.cu) {
    first = b;
    n = 1;
    return true;
  }
  const int lo = __ldg(r.cu + b), hi = __ldg(r.cu + b + 1);
  const int T = static_cast<int>(r.T);
  first = min(max(lo, 0), T);
  n = min(max(hi, first), T) - first;
  return first == lo && n == hi - lo;
}

// Row index (token row over all pages; below 2^32) of head h, slot `slot` of
// page `pg`.
__device__ __forceinline__ int64_t kv_row(const KvNvfp4& c, int pg, int h, int slot) {
  return ((static_cast<int64_t>(pg) * c.Hkv + h) << c.page_shift) + slot;
}

cudaError_t launch_kv_append_nvfp4(const KvNvfp4& c, const KvRows& r, const void* k, const void* v, int64_t ld_k,
                                   int64_t ld_v, int32_t* status, cudaStream_t stream);
cudaError_t launch_kv_read_nvfp4(const KvNvfp4& c, const KvRows& r, void* k, void* v, int32_t* status,
                                 cudaStream_t stream);

struct AttnNvfp4Args {
  KvNvfp4 c;
  KvRows r;
  const uint16_t* q;  // bf16, row t at q + t ld_q, Hq heads of D
  int64_t ld_q;
  int Hq, max_new;
  float scale;  // of the scores, > 0
  uint16_t* out;  // bf16 [T][Hq][D]
  float* lse;     // [T][Hq] or null
  uint8_t* ws;
  int32_t* status;
};

size_t attention_nvfp4_ws_bytes(int D, int B, int Hq, int Hkv, int64_t max_new);
cudaError_t launch_attention_nvfp4(const AttnNvfp4Args& a, cudaStream_t stream);

}  // namespace qrr
