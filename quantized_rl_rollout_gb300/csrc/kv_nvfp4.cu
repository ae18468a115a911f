// Writing rows of keys and values into the paged NVFP4 cache, and reading
// them back as bf16.
//
// Write, per 16 consecutive values x of a row, with g the head's global scale:
//   s = e4m3_rne(amax / (6 g)),  d = fp32(s g),  code = e2m1_rne(x / d)
// (quotients correctly rounded in fp32; all-zero codes where d = 0): the
// weight quantizer's rule with g in the place of the tensor scale.
// Read: bf16_rn(fp32(e2m1(code) e4m3(s)) g).
//
// Both are bound by memory: 2 bytes a value on one side, 0.5625 on the other.  A
// CTA takes some tokens; it finds their places first (a thread a token).  Then,
// to write, its threads take units of 32 values of them in turn: 64 bytes of
// bf16, 16 of codes, two scales.  To read, its warps take kHeads groups of heads
// of a token at a time, keys and values: a lane a word of 8 codes, so that a
// store of the warp is one stretch of 512 bytes.
//
// Measured, 8 heads of 128: writing 4 x 30000..32768 tokens 116 us, 5.2 TB/s (issue
// slots 58 % busy, DRAM 66 %: the encoding of the values and the tail); reading
// 32 x 2048..4096 tokens 89 us, 5.8 TB/s (DRAM).
//
// The correctly rounded quotients are not formed where they cannot matter: with
// y near 1 / d, x / d lies between x y (1 - 2^-20) and x y (1 + 2^-20), and where
// both round to the same code, so does the quotient (rounding is monotonic).
// Only blocks with a value that near a midpoint of the grid take the division.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "kv_nvfp4.cuh"

namespace qrr {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokensCta = 256;
constexpr int kHeads = 4;  // rows of keys, and of values, a lane reads at a time

// The sequence that row t belongs to (offsets ascending), -1 for a row behind
// the last sequence; its first row and the one behind its last.
__device__ __forceinline__ int seq_of(const KvRows& r, int B, int t, int& first, int& end) {
  first = t, end = t + 1;
  if (!r.cu) return t;
  int lo = 0, hi = B;  // the first b with cu[b + 1] > t is in [lo, hi]
  first = __ldg(r.cu);
  while (lo < hi) {
    const int mid = (lo + hi) >> 1, x = __ldg(r.cu + mid + 1);
    if (x > t) hi = mid, end = x;
    else lo = mid + 1, first = x;
  }
  return lo < B && t >= first ? lo : -1;
}

constexpr uint32_t kNoToken = 0xFFFFFFFFu;   // padding, a position below zero
// outside the table, its page outside the cache, or of a sequence whose offsets leave the call's rows
constexpr uint32_t kBadToken = 0xFFFFFFFEu;

// Cache row of call row t and head 0.
__device__ __forceinline__ uint32_t place(const KvNvfp4& c, const KvRows& r, int t) {
  int first, end;
  const int b = seq_of(r, c.B, t, first, end);
  if (b < 0) return kNoToken;
  if (first < 0 || end > r.T) return kBadToken;
  const int64_t p = static_cast<int64_t>(__ldg(r.pos + b)) + (t - first);
  if (p < 0) return kNoToken;
  if (p >= c.capacity()) return kBadToken;
  const int pg = __ldg(c.table + static_cast<int64_t>(b) * c.max_pages + (p >> c.page_shift));
  if (pg < 0 || pg >= c.num_pages) return kBadToken;
  return static_cast<uint32_t>(kv_row(c, pg, 0, static_cast<int>(p) & ((1 << c.page_shift) - 1)));
}

// A CTA's tokens, and a token's units.
struct Units {
  int tokens;
  FastDiv units;
};

// One unit of a token: kind, head, chunk of 32 values of the head's row.
struct Unit {
  bool value;
  int h, chunk;
  __device__ __forceinline__ Unit(const KvNvfp4& c, int u, int units) {
    value = u >= units / 2;
    if (value) u -= units / 2;
    const int shift = c.D == 128 ? 2 : 1;
    h = u >> shift;
    chunk = u & ((1 << shift) - 1);
  }
};

// The places of the CTA's tokens t0 .. t0 + n - 1, in shared memory.  Offsets that
// leave the call's rows or descend are told whether they name a row or not.
__device__ __forceinline__ int find_places(const KvNvfp4& c, const KvRows& r, const Units& un, int t0, uint32_t* at,
                                           int32_t* status) {
  const int n = min(un.tokens, static_cast<int>(r.T) - t0);
  if (r.cu && blockIdx.x == 0)
    for (int b = threadIdx.x; b < c.B; b += kThreads) {
      int first, rows;
      if (!kv_rows_of(r, b, first, rows)) flag(status, QRR_DEV_BAD_INDEX);
    }
  for (int i = threadIdx.x; i < n; i += kThreads) {
    at[i] = place(c, r, t0 + i);
    if (at[i] == kBadToken) flag(status, QRR_DEV_BAD_INDEX);
  }
  __syncthreads();
  return n;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}

// E2M1 codes of 8 values times y.
__device__ __forceinline__ uint32_t codes_of(const uint64_t (&x)[4], uint64_t y) {
  const float2 a = unpair(mul2(x[0], y)), b = unpair(mul2(x[1], y)), c = unpair(mul2(x[2], y)), d = unpair(mul2(x[3], y));
  const float v[8] = {a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
  return cvt_e2m1x8(v);
}

__device__ __forceinline__ float rcp_near(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kUnder = 1.0f - 0x1p-20f, kOver = 1.0f + 0x1p-20f;

// The scale byte and the codes of one block of 16 values.
__device__ __forceinline__ uint32_t quantize_block(const uint4 (&x)[2], float g, uint2& codes, int32_t* status) {
  uint32_t m = max(absmax_bits8(x[0]), absmax_bits8(x[1]));
  if (m >= 0x7F80u) {
    flag(status, QRR_DEV_NONFINITE);
    m = 0x7F7Fu;  // the scale written stays finite
  }
  const float amax = bf16bits_to_f32(m), g6 = __fmul_rn(6.0f, g);
  const float near = amax * rcp_near(g6);
  const uint32_t both = cvt_e4m3x2(near * kUnder, near * kOver);
  uint32_t s = both & 0xFFu;
  // (a divisor whose reciprocal leaves the normal range takes the division too)
  if (s != both >> 8 || !(g6 > 0x1p-100f && g6 < 0x1p100f)) s = cvt_e4m3x2(__fdiv_rn(amax, g6), 0.0f) & 0xFFu;
  const float d = __fmul_rn(e4m3_to_f32_cvt(s), g);
  codes = make_uint2(0u, 0u);
  if (d > 0.0f) {
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    uint64_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = pair(bf16_lo(w[i]), bf16_hi(w[i]));
      hi[i] = pair(bf16_lo(w[i + 4]), bf16_hi(w[i + 4]));
    }
    const float y = rcp_near(d);
    const uint64_t under = pair(y * kUnder, y * kUnder), over = pair(y * kOver, y * kOver);
    codes = make_uint2(codes_of(lo, under), codes_of(hi, under));
    if (codes.x != codes_of(lo, over) || codes.y != codes_of(hi, over) || !(d > 0x1p-100f && d < 0x1p100f)) {
      const SharedDivisor2 div(d);
      float q[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) div(bf16_lo(w[i]), bf16_hi(w[i]), q[2 * i], q[2 * i + 1]);
      const float a[8] = {q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7]};
      const float b[8] = {q[8], q[9], q[10], q[11], q[12], q[13], q[14], q[15]};
      codes = make_uint2(cvt_e2m1x8(a), cvt_e2m1x8(b));
    }
  }
  return s;
}

// The 8 values of a word of codes, as bf16 (code x scale is exact in f16).
__device__ __forceinline__ uint4 values_of(uint32_t codes, uint32_t scale, float g) {
  uint32_t f[4], p[4], s2;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(s2) : "r"(scale | scale << 8));
  f16x2x4_from_e2m1x8(codes, f);
  const uint64_t g2 = pair(g, g);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(f[j]) : "r"(s2));
    const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&f[j])), y = unpair(mul2(pair(e.x, e.y), g2));
    const __nv_bfloat162 b = __floats2bfloat162_rn(y.x, y.y);
    p[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(p[0], p[1], p[2], p[3]);
}

}  // namespace

__global__ void __launch_bounds__(kThreads) kv_append_nvfp4_kernel(const KvNvfp4 c, const KvRows r, const Units un,
                                                                   const uint16_t* __restrict__ k,
                                                                   const uint16_t* __restrict__ v, int64_t ld_k,
                                                                   int64_t ld_v, int32_t* status) {
  __shared__ uint32_t at[kMaxTokensCta];
  const int t0 = blockIdx.x * un.tokens, units = static_cast<int>(un.units.d);
  const int n = find_places(c, r, un, t0, at, status);
  for (int i = threadIdx.x; i < n * units; i += kThreads) {
    const int t = un.units.div(i);
    const Unit u(c, i - t * units, units);
    const uint32_t row0 = at[t];
    if (row0 >= kBadToken) continue;
    const uint16_t* src = (u.value ? v + (t0 + t) * ld_v : k + (t0 + t) * ld_k) + u.h * c.D + u.chunk * 32;
    uint4 x[2][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j >> 1][j & 1] = __ldcs(reinterpret_cast<const uint4*>(src) + j);
    const float* gp = u.value ? c.vg : c.kg;
    const float g = gp ? __ldg(gp + u.h) : 1.0f;
    uint2 a, b;
    const uint32_t s0 = quantize_block(x[0], g, a, status), s1 = quantize_block(x[1], g, b, status);
    const int64_t row = static_cast<int64_t>(row0) + (static_cast<int64_t>(u.h) << c.page_shift);
    *reinterpret_cast<uint4*>((u.value ? c.vc : c.kc) + row * (c.D / 2) + u.chunk * 16) = make_uint4(a.x, a.y, b.x, b.y);
    *reinterpret_cast<uint16_t*>((u.value ? c.vs : c.ks) + row * (c.D / 16) + u.chunk * 2) = static_cast<uint16_t>(s0 | s1 << 8);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_read_nvfp4_kernel(const KvNvfp4 c, const KvRows r, const Units un,
                                                                 uint16_t* __restrict__ k, uint16_t* __restrict__ v,
                                                                 int32_t* status) {
  constexpr int kWords = D / 8, kRows = 32 / kWords;  // of a row; rows of a warp
  __shared__ uint32_t at[kMaxTokensCta];
  const int t0 = blockIdx.x * un.tokens, groups = static_cast<int>(un.units.d);
  const int n = find_places(c, r, un, t0, at, status);
  const int lane = threadIdx.x & 31, word = lane % kWords, sub = lane / kWords;
  for (int i = threadIdx.x >> 5; i < n * groups; i += kThreads / 32) {
    const int t = un.units.div(i), h0 = (i - t * groups) * kHeads * kRows + sub;
    const uint32_t row0 = at[t];
    uint32_t w[2][kHeads] = {}, s[2][kHeads] = {};
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      const int h = h0 + u * kRows;
      if (row0 >= kBadToken || h >= c.Hkv) continue;
      const int64_t row = static_cast<int64_t>(row0) + (static_cast<int64_t>(h) << c.page_shift);
      w[0][u] = __ldg(reinterpret_cast<const uint32_t*>(c.kc) + row * kWords + word);
      w[1][u] = __ldg(reinterpret_cast<const uint32_t*>(c.vc) + row * kWords + word);
      s[0][u] = __ldg(c.ks + row * (D / 16) + (word >> 1));
      s[1][u] = __ldg(c.vs + row * (D / 16) + (word >> 1));
    }
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      const int h = h0 + u * kRows;
      if (h >= c.Hkv) continue;
      const int64_t to = (static_cast<int64_t>(t0 + t) * c.Hkv + h) * kWords + word;
      __stcs(reinterpret_cast<uint4*>(k) + to, values_of(w[0][u], s[0][u], c.kg ? __ldg(c.kg + h) : 1.0f));
      __stcs(reinterpret_cast<uint4*>(v) + to, values_of(w[1][u], s[1][u], c.vg ? __ldg(c.vg + h) : 1.0f));
    }
  }
}

namespace {

// Tokens a CTA: enough units for its threads (or warps) to take several each,
// but CTAs for every SM.
Units units_for(int64_t T, int units, int want) {
  int dev = 0, sms = kSMs;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t most = std::min(kMaxTokensCta, std::max(1, want / units)), spread = (T + 4 * sms - 1) / (4 * sms);
  return Units{static_cast<int>(std::max<int64_t>(1, std::min(most, spread))), FastDiv(static_cast<uint32_t>(units))};
}

}  // namespace

cudaError_t launch_kv_append_nvfp4(const KvNvfp4& c, const KvRows& r, const void* k, const void* v, int64_t ld_k,
                                   int64_t ld_v, int32_t* status, cudaStream_t stream) {
  if (r.T == 0 || c.Hkv == 0) return cudaSuccess;
  const Units un = units_for(r.T, 2 * c.Hkv * (c.D / 32), 8 * kThreads);
  kv_append_nvfp4_kernel<<<static_cast<unsigned>((r.T + un.tokens - 1) / un.tokens), kThreads, 0, stream>>>(
      c, r, un, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), ld_k, ld_v, status);
  return cudaGetLastError();
}

cudaError_t launch_kv_read_nvfp4(const KvNvfp4& c, const KvRows& r, void* k, void* v, int32_t* status,
                                 cudaStream_t stream) {
  if (r.T == 0 || c.Hkv == 0) return cudaSuccess;
  const int heads = kHeads * 256 / c.D;  // of a warp's step
  const Units un = units_for(r.T, (c.Hkv + heads - 1) / heads, 8 * kThreads / 32);
  const unsigned grid = static_cast<unsigned>((r.T + un.tokens - 1) / un.tokens);
  uint16_t *kb = static_cast<uint16_t*>(k), *vb = static_cast<uint16_t*>(v);
  if (c.D == 128) kv_read_nvfp4_kernel<128><<<grid, kThreads, 0, stream>>>(c, r, un, kb, vb, status);
  else kv_read_nvfp4_kernel<64><<<grid, kThreads, 0, stream>>>(c, r, un, kb, vb, status);
  return cudaGetLastError();
}

}  // namespace qrr
