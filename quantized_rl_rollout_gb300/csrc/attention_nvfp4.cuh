// What the two kernels of attention over the paged NVFP4 cache share: few rows a
// sequence (attention_nvfp4.cu) and many (attention_nvfp4_tc.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kv_nvfp4.cuh"
#include "once_per_device.cuh"
#include "tc.cuh"

namespace qrr {

namespace attn4 {

constexpr int kMaxSms = 160;       // of the workspace's size; grids are capped to it
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -1.0e30f;  // reference of a row that has seen nothing
// a new reference lies kLift under the largest score (many rows: kLift to kLift + 1,
// a whole number) and moves when a score exceeds it by kRoom
constexpr float kLift = 7.0f, kRoom = 15.0f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row's factor of its weighted sum, and its log-sum-exp, from its reference and its
// sum of weights: 0 and -inf where it has seen nothing (a NaN comes through).
__device__ __forceinline__ float row_factor(float vg, float l) { return l == 0.0f ? 0.0f : __fdividef(vg, l); }
__device__ __forceinline__ float row_lse(float m, float l) { return l == 0.0f ? -INFINITY : (m + lg2(l)) * kLn2; }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two E4M3 bytes -> f16x2 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The exponent e that brings a row whose largest |bf16| has the bits mx into
// f16: mx 2^-e in [2^14, 2^15) (0 for a zero or a non-finite row).
__device__ __forceinline__ int query_exp(uint32_t mx) {
  if (mx == 0u || mx >= 0x7F80u) return 0;
  return (mx >= 0x80u ? static_cast<int>(mx >> 7) - 127 : 31 - __clz(static_cast<int>(mx)) - 133) - 14;
}

// An item that crosses ranges.  Piece 2 k is range k's first when it continues
// an item, piece 2 k + 1 its last when it starts one that the next ranges
// continue.
struct Record {
  int pieces;           // 0: there is nothing to join
  int range;            // that the item starts in
  int rt, h, first, n;  // its row tile, KV head, the sequence's rows
};

struct Params {
  KvNvfp4 c;
  KvRows r;
  const uint16_t* q;
  int64_t ld_q;
  int Hq, G, max_new;
  FastDiv byG;
  float scale;
  uint16_t* out;
  float* lse;
  Record* rec;
  float *pm, *pl, *po;  // [piece][row], [piece][row], [piece][row][D]
  int32_t* status;
};

__device__ __forceinline__ Seq seq_of(const Params& p, int b) {
  int first, n;
  if (!kv_rows_of(p.r, b, first, n) || n > p.max_new) flag(p.status, QRR_DEV_BAD_INDEX);
  const int cap = static_cast<int>(p.c.capacity());
  const Seq s = seq_at(first, min(n, p.max_new), __ldg(p.r.pos + b), cap);
  if (s.n > 0 && s.pos + (s.n - 1) >= cap) flag(p.status, QRR_DEV_BAD_INDEX);
  return s;
}

// Output row of row `row` (token row / G, head of the group row % G).
__device__ __forceinline__ int64_t out_row(const Params& p, int first, int h, int row) {
  return static_cast<int64_t>(first + p.byG.div(row)) * p.Hq + h * p.G + p.byG.mod(row);
}

// Weights of up to 32 pieces of a row, piece i in lane i (the rest: none), brought to
// the row's new reference m; `old` brings what the row has so far there.
__device__ __forceinline__ float piece_weight(float mi, float li, float& m, float& l, float& old) {
  float top = mi;
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
  top = fmaxf(top, m);
  old = ex2(m - top);
  m = top;
  const float a = ex2(mi - top);
  float sum = a * li;
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
  l = l * old + sum;
  return a;
}

__device__ __forceinline__ uint2 bf16x4(const float (&o)[4], float f) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(o[0] * f, o[1] * f), b = __floats2bfloat162_rn(o[2] * f, o[3] * f);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

__device__ __forceinline__ int64_t piece_row(const Record& rec, int i, int rt) {
  return static_cast<int64_t>(i == 0 ? 2 * rec.range + 1 : 2 * (rec.range + i)) * rt;
}

// Launches a kernel as the programmatic dependent of the one before it in the
// stream: its CTAs may be placed while that one still runs, and wait for it
// (griddep_wait) before they touch anything.
template <class... A>
cudaError_t launch_dependent(void (*kernel)(A...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The current device and its SMs.
inline cudaError_t device_of(int& dev, int& sms) {
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
}

// Workspace of `ranges` ranges whose pieces have `rt` rows, and their records.
inline size_t align256(size_t v) { return (v + 255) / 256 * 256; }
inline size_t ws_bytes(int D, int ranges, int rt, int64_t records) {
  const size_t rows = static_cast<size_t>(2) * ranges * rt;
  return align256(sizeof(Record) * records) + 2 * align256(rows * 4) + align256(rows * D * 4);
}
inline Params make_params(const AttnNvfp4Args& a, uint8_t* w, int ranges, int rt, int64_t records) {
  const int G = a.Hq / a.c.Hkv;
  Params p{a.c, a.r, a.q, a.ld_q, a.Hq, G, a.max_new, FastDiv(static_cast<uint32_t>(G)), a.scale, a.out, a.lse};
  const size_t rows = static_cast<size_t>(2) * ranges * rt;
  p.rec = reinterpret_cast<Record*>(w);
  w += align256(sizeof(Record) * records);
  p.pm = reinterpret_cast<float*>(w);
  w += align256(rows * 4);
  p.pl = reinterpret_cast<float*>(w);
  w += align256(rows * 4);
  p.po = reinterpret_cast<float*>(w);
  p.status = a.status;
  return p;
}

}  // namespace attn4

// Many rows a sequence (attention_nvfp4_tc.cu); ws: its own part; beside: the
// launch before it in the stream is the other kernel's.
size_t attention_nvfp4_tc_ws_bytes(int D);
cudaError_t launch_attention_nvfp4_tc(const AttnNvfp4Args& a, uint8_t* ws, bool beside, cudaStream_t stream);

}  // namespace qrr
