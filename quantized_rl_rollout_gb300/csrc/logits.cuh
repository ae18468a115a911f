// Rows of logits: what the losses (logits_loss.cu) and the verification of drafts (verify_drafts.cu) share.
//
// A row starts anywhere its element type allows (an odd vocabulary, a slice of padded rows), so it is read in granules of
// 16 aligned bytes: granule i holds the elements i kN - lead .. i kN - lead + kN - 1, lead being the elements between the
// 16-byte boundary at or before the row's start and that start. The first and the last granule may be cut; what they hold
// beside the row reads -inf.
#pragma once

#include <cuda_bf16.h>

#include "linear.cuh"
#include "tc.cuh"

namespace qrr {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kAll = 0xFFFFFFFFu;

// Element types: Bf16 keeps its bits as uint16_t.
using Bf16 = uint16_t;
template <class E>
constexpr int kPer = 16 / static_cast<int>(sizeof(E));  // elements of a granule

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float to_f32(Bf16 x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ Bf16 from_f32(float x, Bf16) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
__device__ __forceinline__ float from_f32(float x, float) { return x; }

__device__ __forceinline__ void unpack(uint4 g, float (&x)[8]) {
  x[0] = bf16_lo(g.x), x[1] = bf16_hi(g.x), x[2] = bf16_lo(g.y), x[3] = bf16_hi(g.y);
  x[4] = bf16_lo(g.z), x[5] = bf16_hi(g.z), x[6] = bf16_lo(g.w), x[7] = bf16_hi(g.w);
}
__device__ __forceinline__ void unpack(uint4 g, float (&x)[4]) {
  x[0] = __uint_as_float(g.x), x[1] = __uint_as_float(g.y), x[2] = __uint_as_float(g.z), x[3] = __uint_as_float(g.w);
}

__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

template <int N>
__device__ __forceinline__ float max_of(const float (&x)[N]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
  return m;
}

// Elements between the 16-byte boundary at or before `row` and it, and the granules of a row of V.
template <class E>
__device__ __forceinline__ int lead_of(const E* row) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u) / static_cast<int>(sizeof(E));
}
template <class E>
__host__ __device__ __forceinline__ int granules_of(int lead, int V) {
  return (lead + V + kPer<E> - 1) / kPer<E>;
}

// A cut granule: first element e0 (below 0, or with its end behind the row), -inf outside the row.
template <class E>
__device__ __noinline__ uint4 load_cut(const E* row, int e0, int V) {
  float x[kPer<E>];
#pragma unroll
  for (int u = 0; u < kPer<E>; ++u) x[u] = e0 + u >= 0 && e0 + u < V ? to_f32(row[e0 + u]) : -INFINITY;
  return pack(x);
}

// ---- sums of e^{x / t} ----------------------------------------------------------
//
// With c = log2(e) / t, a sum is kept as s = sum 2^{c x - r} for a reference r = rint(c m), m one of the logits. fp32's
// exponents reach far enough that m need not be the largest: it is the largest of the first values that a thread sees, and
// the values behind them cost a multiply-add, an exponential and an addition each, no comparison. A sum that gets near
// the end of the range is taken again with the largest of all (add_largest). References are whole numbers so that a sum
// moves to another by a power of two, and c x - r is rounded once.
// c is held in two parts: rounded to one, the exponents of a row would be off by up to 2^-24 of themselves, which is 1e-6 of a
// probability where logits reach 20. The second part costs half an instruction an element, beside an exponential's
// eight cycles.
// A reference of more than 2^20 (rows at their type's lowest value, say, where c m itself may overflow) takes the
// difference of the logits first: r = c m in effect, 2^{c (x - m)}.

__device__ __forceinline__ uint64_t f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f32x2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// t and 1 / t, and log2(e) / t in two parts, c rounded down and lo > 0: of a logit of -inf both products are -inf.
struct Scale {
  float t, inv_t, c, lo;
  __device__ __forceinline__ operator float() const { return c; }
  __device__ __forceinline__ float exponent(float x, float r) const { return fmaf(x, lo, fmaf(x, c, -r)); }
};
inline Scale scale_of(double t) {
  const double k = 1.4426950408889634 / t;
  float c = static_cast<float>(k);
  if (c >= k) c = nextafterf(c, 0.0f);
  return Scale{static_cast<float>(t), static_cast<float>(1.0 / t), c, static_cast<float>(k - c)};
}

// A number in two parts, and sums of such.
struct Two {
  float high = 0.0f, low = 0.0f;
  __device__ __forceinline__ void add(Two x) {
    const float sum = high + x.high, part = sum - high;
    low = (low + x.low) + ((high - (sum - part)) + (x.high - part));
    high = sum;
  }
  __device__ __forceinline__ void add_warp() {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) add(Two{__shfl_xor_sync(kAll, high, o), __shfl_xor_sync(kAll, low, o)});
  }
};

// 2^(x + lo) for a small lo, in two parts: the hardware's is 2 ulps off, which is seen where few values make up a sum. 2^f by
// its series, |f| <= 1/2.
__device__ __forceinline__ Two pow2(float x, float lo) {
  const float n = rintf(fminf(fmaxf(x, -200.0f), 200.0f)), f = (x - n) + lo;
  float p = 1.52527338e-5f;  // ln(2)^7 / 7!
  p = fmaf(p, f, 1.54035304e-4f);
  p = fmaf(p, f, 1.33335581e-3f);
  p = fmaf(p, f, 9.61812911e-3f);
  p = fmaf(p, f, 5.55041087e-2f);
  p = fmaf(p, f, 2.40226507e-1f);
  p = fmaf(p, f, 6.93147181e-1f);
  const float high = fmaf(p, f, 1.0f), low = fmaf(p, f, 1.0f - high);
  const int e = static_cast<int>(n);
  return x < -200.0f ? Two{} : Two{ldexpf(high, e), ldexpf(low, e)};
}

// The reference that a logit m makes (m = -inf: 0, for sums without a value).
struct Ref {
  float m, r;
  bool far;
  __device__ __forceinline__ Ref(float m_, Scale c) : m(m_ == -INFINITY ? 0.0f : m_) {
    r = rintf(m * c);
    far = !(fabsf(r) <= 0x1p20f);
  }
  __device__ __forceinline__ float operator()(float x, Scale c) const {
    return ex2_approx(far ? (x - m) * c : c.exponent(x, r));
  }
  // Where a sum stands, in base 2, is c m if it is far and r if not, which is up to half a power of two from c m. What m has
  // above that, and how far this stands above another.
  __device__ __forceinline__ float offset(Scale c) const { return far ? 0.0f : c.exponent(m, r); }
  __device__ __forceinline__ float above(const Ref& other, Scale c) const {
    return far || other.far ? (m - other.m) * c + (other.offset(c) - offset(c)) : r - other.r;
  }
  __device__ __forceinline__ Two exactly(float x, Scale c) const {
    if (far || !(fabsf(x) < 1e30f)) return Two{(*this)(x, c), 0.0f};
    const float high = __fmul_rn(x, c);  // (not contracted: what it is off by is added)
    return pow2(high - r, fmaf(x, c, -high) + x * c.lo);
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
// The largest of a warp's values (NaN aside).
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

struct Sum {
  float m = -INFINITY, s = 0.0f;

  // What a sum at m is worth at another reference, not below it.
  __device__ __forceinline__ static float moved(float m, const Ref& to, Scale c) {
    return m == -INFINITY ? 0.0f : ex2_approx(Ref(m, c).above(to, c));
  }
  // A sum without values has s = 0 and m = -inf; a NaN in s stays.
  __device__ __forceinline__ void merge(float m2, float s2, Scale c) {
    const Ref to(fmaxf(m, m2), c);
    s = s * moved(m, to, c) + s2 * moved(m2, to, c);
    m = fmaxf(m, m2);
  }
  // Of a warp's sums, the same in every lane: one move each, to the largest reference. (Far ones are rare: in line, their
  // moves cost the verification of 64 x 8 drafts 0.7 us of 53.)
  __device__ __forceinline__ void merge_warp(Scale c) {
    const float to = warp_max(m);
    const Ref from(m, c);
    if (__any_sync(kAll, from.far)) s = moved_far(m, s, to, c);
    else s *= m == -INFINITY ? 0.0f : ex2_approx(from.r - Ref(to, c).r);
    m = to;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  }
  static __device__ __noinline__ float moved_far(float m, float s, float to, Scale c) { return s * moved(m, Ref(to, c), c); }
  // Values with their largest: the reference follows it.
  template <int N>
  __device__ __forceinline__ void add_largest(const float (&x)[N], float largest, Scale c) {
    if (largest > m) {
      s *= moved(m, Ref(largest, c), c);
      m = largest;
    }
    const Ref ref(m, c);
#pragma unroll
    for (int u = 0; u < N; ++u) s += ref(x[u], c);
  }
};

// A thread's sum at a reference that stays, in two accumulators of two values.
template <class E>
struct FixedSum {
  uint64_t c2, lo2, nr2, a0, a1;
  __device__ __forceinline__ void start(const Ref& ref, Scale c) {
    c2 = f32x2(c, c);
    lo2 = f32x2(c.lo, c.lo);
    nr2 = f32x2(-ref.r, -ref.r);
    a0 = a1 = 0;
  }
  __device__ __forceinline__ void add(uint4 g) {
    float x[kPer<E>];
    unpack(g, x);
#pragma unroll
    for (int u = 0; u < kPer<E>; u += 4) {
      float e0, e1, e2, e3;
      const uint64_t x0 = f32x2(x[u], x[u + 1]), x1 = f32x2(x[u + 2], x[u + 3]);
      f32x2(fma2(x0, lo2, fma2(x0, c2, nr2)), e0, e1);
      f32x2(fma2(x1, lo2, fma2(x1, c2, nr2)), e2, e3);
      a0 = add2(a0, f32x2(ex2_approx(e0), ex2_approx(e1)));
      a1 = add2(a1, f32x2(ex2_approx(e2), ex2_approx(e3)));
    }
  }
  __device__ __forceinline__ float total() const {
    float x, y;
    f32x2(add2(a0, a1), x, y);
    return x + y;
  }
};

// A sum s = sum 2^{c x - r} (and a low part of it) as a power of two and a small logarithm: log2 of it and its reference =
// whole + part, |part| <= 1/2.
struct Log2 {
  float whole, part;
  __device__ __forceinline__ Log2(const Ref& ref, float s, float low = 0.0f) {
    int e;
    float f = frexpf(s, &e);
    if (f < 0.70710678f) f += f, --e;
    part = log2f(f);
    if (low != 0.0f) part = fmaf(low / s, kLog2e, part);
    whole = ref.r + static_cast<float>(e);  // exact
  }
};

// ln of e^{x / t} / s: what is left of c x behind the whole powers of two is rounded as the small number that it is.
__device__ __forceinline__ float ln_share(float x, const Ref& ref, float s, const Log2& log2, Scale c) {
  // c x may overflow where x / t does not, and beside such numbers the sum's own power of two is nothing
  if (ref.far || !(fabsf(x) < 1e30f)) return (x - ref.m) * c.inv_t - logf(s);
  return (c.exponent(x, log2.whole) - log2.part) * kLn2;
}

// L2's treatment of what is read: once, or again soon.
__device__ __forceinline__ uint64_t read_once() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t read_again() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// (Of memory that the kernel may write: it stays where it stands among stores.)
__device__ __forceinline__ uint4 load_hint(const uint4* p, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy)
               : "memory");
  return v;
}

// use(i, load(i)) for i = first, first + step, .. below end, kInFlight loads at a time.
template <int kInFlight, class Load, class Use>
__device__ __forceinline__ void stream(int first, int end, int step, Load load, Use use) {
  int i = first;
  for (; i + (kInFlight - 1) * step < end; i += kInFlight * step) {
    uint4 g[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) g[u] = load(i + u * step);
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) use(i + u * step, g[u]);
  }
  uint4 g[kInFlight];
#pragma unroll
  for (int u = 0; u < kInFlight; ++u)
    if (i + u * step < end) g[u] = load(i + u * step);
#pragma unroll
  for (int u = 0; u < kInFlight; ++u)
    if (i + u * step < end) use(i + u * step, g[u]);
}

// ---- clusters ---------------------------------------------------------------

// To the same variable of CTA `rank`.
__device__ __forceinline__ void st_cluster(const float2* p, uint32_t rank, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(cluster_addr(p, rank)), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void st_cluster(const uint64_t* p, uint32_t rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_addr(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// ---- host -------------------------------------------------------------------

constexpr double kMinTemperature = 1e-6, kMaxTemperature = 1e6;

// Launch on clusters of `cluster` CTAs along x.
template <class... K, class... A>
cudaError_t launch_clusters(void (*kernel)(K...), unsigned grid, int cluster, int threads, size_t smem, cudaStream_t stream,
                            A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<A&&>(args)...);
}

// ---- arguments ----------------------------------------------------------------

// A call of logits_loss.cu: the rows, the teacher or the tokens, and the outputs.
struct LogitsLossArgs {
  const void* logits;
  int64_t ld, T;
  int V, fp32;
  Scale scale;  // of the logits (policy gradient: at temperature 1)
  // distillation
  const int32_t* ids;  // [T][k]
  const float* top;    // [T][k]
  const float* top_lse;
  int k;
  double temperature;  // its scale is set by the launch, as verify's
  const float* grad;
  const float* stats_in;
  float* loss;
  float* stats;
  // policy gradient
  const int32_t* tokens;
  const float* advantages;
  const float* rollout_logp;
  float cap;
  float* logp;
  float* w;
  void* dlogits;
  int64_t ldd;
  int32_t* status;
};
enum class LossMode { kLoss, kGrad, kBackward, kPolicy };
constexpr int kMaxTop = 1024;
cudaError_t launch_logits_loss(LogitsLossArgs a, LossMode mode, cudaStream_t stream);

struct VerifyArgs {
  const void* target;  // [T + B][V]
  int64_t ld_target;
  const void* draft;  // [T][V] or null
  int64_t ld_draft;
  int64_t T;
  int B, V, fp32;
  const int32_t* drafts;  // [T]
  const int32_t* cu;      // [B + 1] or null
  const float* uniforms;  // [T]
  const float* noise;     // [B][V]
  int64_t ld_noise;
  double temperature;  // 0: the likeliest token
  Scale scale;
  int32_t* tokens;    // [T + B]
  int32_t* accepted;  // [B]
  float* logp;        // [T + B]
  void* workspace;    // verify_drafts_ws_bytes
  int32_t* status;
};
constexpr int64_t kMaxDrafts = 1 << 24;  // drafts and sequences of a call
size_t verify_drafts_ws_bytes(int64_t T, int64_t B, int64_t V, int fp32);
cudaError_t launch_verify_drafts(VerifyArgs a, cudaStream_t stream);

}  // namespace qrr
