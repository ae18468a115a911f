// Writing rows of keys and values into the paged NVFP4 cache, and reading
// them back as bf16.
//
// Write, per 16 consecutive values x of a row, with g the head's global scale:
//   s = e4m3_rne(amax / (6 g)),  d = fp32(s g),  code = e2m1_rne(x / d)
// (quotients correctly rounded in fp32; all-zero codes where d = 0): the
// weight quantizer's rule with g in the place of the tensor scale.
// Read: bf16_rn(fp32(e2m1(code) e4m3(s)) g).
//
// Both are bound by memory: 2 bytes a value on one side, 0.5625 on the other.
// One thread takes one block of 16 values (two 16-byte accesses of bf16, one
// 8-byte access of codes, one scale byte).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_nvfp4.cuh"

namespace qrr {

namespace {

constexpr int kThreads = 256;

// The sequence that row t belongs to (offsets ascending), -1 for a row behind
// the last sequence.
__device__ __forceinline__ int seq_of(const KvRows& r, int B, int t) {
  if (!r.cu) return t;
  int lo = 0, hi = B;  // the first b with cu[b + 1] > t is in [lo, hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(r.cu + mid + 1) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo < B && t >= __ldg(r.cu + lo) ? lo : -1;
}

// Cache row of call row t and head h; -1: no token (padding, a position below
// zero), -2: outside the table or its page outside the cache.
__device__ __forceinline__ int64_t place(const KvNvfp4& c, const KvRows& r, int t, int h) {
  const int b = seq_of(r, c.B, t);
  if (b < 0) return -1;
  const int64_t p = static_cast<int64_t>(__ldg(r.pos + b)) + (r.cu ? t - __ldg(r.cu + b) : 0);
  if (p < 0) return -1;
  if (p >= c.capacity()) return -2;
  const int pg = __ldg(c.table + static_cast<int64_t>(b) * c.max_pages + (p >> c.page_shift));
  if (pg < 0 || pg >= c.num_pages) return -2;
  return kv_row(c, pg, h, static_cast<int>(p) & ((1 << c.page_shift) - 1));
}

}  // namespace

__global__ void __launch_bounds__(kThreads) kv_append_nvfp4_kernel(const KvNvfp4 c, const KvRows r,
                                                                   const uint16_t* __restrict__ k,
                                                                   const uint16_t* __restrict__ v, int64_t ld_k,
                                                                   int64_t ld_v, int32_t* status) {
  const int bpr = c.D / 16, per_kind = c.Hkv * bpr;  // blocks of a row of one head, of a token's keys
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t t = idx / (2 * per_kind);
  if (t >= r.T) return;
  int rest = static_cast<int>(idx - t * 2 * per_kind);
  const bool is_v = rest >= per_kind;
  if (is_v) rest -= per_kind;
  const int h = rest / bpr, blk = rest % bpr;
  const int64_t row = place(c, r, static_cast<int>(t), h);
  if (row < 0) {
    if (row == -2) flag(status, QRR_DEV_BAD_INDEX);
    return;
  }
  const uint16_t* src = (is_v ? v + t * ld_v : k + t * ld_k) + static_cast<int64_t>(rest) * 16;
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(src)), b = __ldcs(reinterpret_cast<const uint4*>(src) + 1);
  uint32_t m = max(absmax_bits8(a), absmax_bits8(b));
  if (m >= 0x7F80u) {
    flag(status, QRR_DEV_NONFINITE);
    m = 0x7F7Fu;  // the scale written stays finite
  }
  const float* gp = is_v ? c.vg : c.kg;
  const float g = gp ? __ldg(gp + h) : 1.0f;
  const uint32_t s = cvt_e4m3x2(__fdiv_rn(bf16bits_to_f32(m), __fmul_rn(6.0f, g)), 0.0f) & 0xFFu;
  const float d = __fmul_rn(e4m3_to_f32(s), g);
  uint2 codes = make_uint2(0u, 0u);
  if (d > 0.0f) {
    const SharedDivisor2 div(d);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float q[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) div(bf16_lo(w[i]), bf16_hi(w[i]), q[2 * i], q[2 * i + 1]);
    const float lo[8] = {q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7]};
    const float hi[8] = {q[8], q[9], q[10], q[11], q[12], q[13], q[14], q[15]};
    codes = make_uint2(cvt_e2m1x8(lo), cvt_e2m1x8(hi));
  }
  reinterpret_cast<uint2*>(is_v ? c.vc : c.kc)[row * bpr + blk] = codes;
  (is_v ? c.vs : c.ks)[row * bpr + blk] = static_cast<uint8_t>(s);
}

__global__ void __launch_bounds__(kThreads) kv_read_nvfp4_kernel(const KvNvfp4 c, const KvRows r,
                                                                 uint16_t* __restrict__ k, uint16_t* __restrict__ v,
                                                                 int32_t* status) {
  const int bpr = c.D / 16, per_kind = c.Hkv * bpr;
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t t = idx / (2 * per_kind);
  if (t >= r.T) return;
  int rest = static_cast<int>(idx - t * 2 * per_kind);
  const bool is_v = rest >= per_kind;
  if (is_v) rest -= per_kind;
  const int h = rest / bpr, blk = rest % bpr;
  const int64_t row = place(c, r, static_cast<int>(t), h);
  uint4 o[2] = {};
  if (row >= 0) {
    const uint2 codes = __ldg(reinterpret_cast<const uint2*>(is_v ? c.vc : c.kc) + row * bpr + blk);
    const float s = e4m3_to_f32(__ldg((is_v ? c.vs : c.ks) + row * bpr + blk));
    const float* gp = is_v ? c.vg : c.kg;
    const float g = gp ? __ldg(gp + h) : 1.0f;
    const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t f[4], p[4];
      f16x2x4_from_e2m1x8(w[i], f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&f[j]));
        const __nv_bfloat162 y = __floats2bfloat162_rn(__fmul_rn(__fmul_rn(e.x, s), g), __fmul_rn(__fmul_rn(e.y, s), g));
        p[j] = *reinterpret_cast<const uint32_t*>(&y);
      }
      o[i] = make_uint4(p[0], p[1], p[2], p[3]);
    }
  } else if (row == -2) {
    flag(status, QRR_DEV_BAD_INDEX);
  }
  uint4* dst = reinterpret_cast<uint4*>((is_v ? v : k) + (t * per_kind + rest) * 16);
  __stcs(dst, o[0]);
  __stcs(dst + 1, o[1]);
}

namespace {

unsigned blocks_for(const KvNvfp4& c, int64_t T) {
  return static_cast<unsigned>((T * 2 * c.Hkv * (c.D / 16) + kThreads - 1) / kThreads);
}

}  // namespace

cudaError_t launch_kv_append_nvfp4(const KvNvfp4& c, const KvRows& r, const void* k, const void* v, int64_t ld_k,
                                   int64_t ld_v, int32_t* status, cudaStream_t stream) {
  if (r.T == 0 || c.Hkv == 0) return cudaSuccess;
  kv_append_nvfp4_kernel<<<blocks_for(c, r.T), kThreads, 0, stream>>>(
      c, r, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), ld_k, ld_v, status);
  return cudaGetLastError();
}

cudaError_t launch_kv_read_nvfp4(const KvNvfp4& c, const KvRows& r, void* k, void* v, int32_t* status,
                                 cudaStream_t stream) {
  if (r.T == 0 || c.Hkv == 0) return cudaSuccess;
  kv_read_nvfp4_kernel<<<blocks_for(c, r.T), kThreads, 0, stream>>>(c, r, static_cast<uint16_t*>(k),
                                                                   static_cast<uint16_t*>(v), status);
  return cudaGetLastError();
}

}  // namespace qrr
