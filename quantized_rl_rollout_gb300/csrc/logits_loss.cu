// Losses over rows of logits with their gradients: distillation from a teacher's top logits, and the policy gradient of the
// tokens that a rollout took.
//
// Distillation, x a row of V logits, t the temperature, q = softmax(x / t), the teacher's top logits y_j at the ids i_j:
//   without a tail   p_j = e^{y_j / t} / sum_i e^{y_i / t},  L = sum_j p_j (ln p_j - ln q_{i_j})
//   with a tail      p_j = e^{y_j / t - lse_teacher}, p_r = 1 - sum_j p_j, q_r = 1 - sum_j q_{i_j},
//                    L = sum_j p_j (ln p_j - ln q_{i_j}) + p_r (ln p_r - ln q_r)
//   dL/dx_v = (q_v - p_v) / t; with a tail, outside the ids, e^{x_v / t - lse_r} (q_r - p_r) / t, lse_r the log-sum-exp of
//   the logits outside. Slots that name one id are one outcome: their p_j add up. Where all p_j add up to more than 1 (the
//   teacher's log-sum-exp is not of these slots), q is weighed with that: (q_v sum_j p_j - p_v) / t.
// Policy gradient of token a with advantage A: logp = x_a - lse, w = min(e^{logp - logp_rollout}, cap),
//   d(-A w logp)/dx_v = A w (q_v - [v = a]), w held fixed: the same form with p_a = 1 and the factor A w.
//
// Bound by memory: a logit is read from it once and its gradient written once (the loss alone only reads). The sums of a row
// are known when all of it has been read, so the gradient reads it again, from L2: a CTA takes a whole row, two CTAs an SM
// (78 MB of rows of 128256 bf16, of which half is still wanted, in 129 MB), and a row is read again before others push it
// out. Where there are few rows, a cluster of CTAs takes one, a contiguous part each, and joins sums over distributed
// shared memory.
//
// With a tail, the logits at the teacher's ids are left out of the sum (their granules are passed over and added without
// them), so that the sum outside them is one of positive terms, not a difference. Sums are fp32; e^x is the hardware's base-2 approximation
// (about 2^-22 relative) where it is taken a logit. What makes up most of a row and of a loss is the ids, a few terms whose
// errors do not average out: their exponentials are within an ulp and summed in two parts (without a tail they replace what
// the hardware made of them), and a logarithm's difference is rounded as the small number that it is. A loss of 0.1 is off by
// 2.6e-8 so (root mean square; 6.3e-8 without), the log-sum-exps by their own rounding.
//
// Measured, rows of 128256 bf16: loss alone, 2048 rows, 77 us (81% of a copy's rate); loss and gradient of 4096, 349 us (82%);
// policy gradient of 4096, 328 us (88%); 2048 rows' gradient from known log-sum-exps 142 us (98%). What is rare is called
// with copies of what it needs: closures by reference put the hot loops' variables on the stack (389 us for the 349, 351 for
// the 328).
#include <float.h>

#include <algorithm>

#include "logits.cuh"
#include "once_per_device.cuh"

namespace qrr {

namespace {

constexpr int kMaxThreads = 512, kMaxParts = 8;
constexpr int kBackwardThreads = 256;
// A rest of the teacher's that is no more than the rounding of its log-sum-exp and of the sum of p_j: beside a student
// without any, it is none.
constexpr float kDust = 1.0f / 65536;

// Part `rank` of a row: `per` granules, elements e0 .. e1 - 1; element e stands at e - base of the CTA's tile.
template <class E>
struct Part {
  const E* row;
  int V, lead, g0, g1, base, e0, e1;

  __device__ __forceinline__ Part(const E* row_, int V_, int rank, int per) : row(row_), V(V_), lead(lead_of(row_)) {
    const int granules = granules_of<E>(lead, V);
    g0 = min(rank * per, granules);
    g1 = min(g0 + per, granules);
    base = g0 * kPer<E> - lead;
    e0 = max(base, 0);
    e1 = min(g1 * kPer<E> - lead, V);
  }
  __device__ __forceinline__ bool has(int id) const { return id >= e0 && id < e1; }
  __device__ __forceinline__ int granule_of(int id) const { return has(id) ? g0 + (id - base) / kPer<E> : -1; }  // -1: not here
  // the granules that lie in the row as a whole
  __device__ __forceinline__ int whole0() const { return base < 0 ? g0 + 1 : g0; }
  __device__ __forceinline__ int whole1() const { return g1 > g0 && g1 * kPer<E> - lead > V ? g1 - 1 : g1; }
  // f(granule number) for the cut ones, by a thread each.
  template <class F>
  __device__ __forceinline__ void cut(int tid, int threads, F f) const {
    const int w0 = whole0(), w1 = whole1();
    if (g0 == g1) return;
    if (tid == 0 && w0 > g0) f(g0);
    if (tid == threads - 1 && w1 < g1 && (w1 > g0 || w0 == g0)) f(w1);
  }
  // Bulk copies of the whole granules to a tile, counted on `bar` with its one arrival (by one thread).
  __device__ __forceinline__ void copy(uint4* tile, uint64_t* bar) const {
    const int w0 = whole0(), w1 = whole1();
    const uint32_t bytes = w1 > w0 ? 16u * static_cast<uint32_t>(w1 - w0) : 0u;
    mbar_arrive_expect_tx(bar, bytes);
    constexpr uint32_t kChunk = 16 << 10;
    const uint8_t* const src = reinterpret_cast<const uint8_t*>(granules() + w0);
    for (uint32_t at = 0; at < bytes; at += kChunk)
      bulk_load(reinterpret_cast<uint8_t*>(tile + (w0 - g0)) + at, src + at, min(kChunk, bytes - at), bar);
  }
  __device__ __forceinline__ const uint4* granules() const { return reinterpret_cast<const uint4*>(row - lead); }
  __device__ __forceinline__ uint4 load_cut(int i) const { return qrr::load_cut(row, i * kPer<E> - lead, V); }
};

// The teacher's slots of a row, in shared memory.
struct Slots {
  int* id;   // -1: unused
  float* y;  // the teacher's logit
  float* p;  // its probability
  float* x;  // the row's logit
  int k;
  __device__ __forceinline__ Slots(uint8_t* at, int k_) : k(k_) {
    id = reinterpret_cast<int*>(at);
    y = reinterpret_cast<float*>(id + k);
    p = y + k;
    x = p + k;
  }
  // False: unused.
  __device__ __forceinline__ bool set(int j, int given, float logit, int V, int32_t* status) const {
    if (given >= V) flag(status, QRR_DEV_BAD_INDEX);
    const bool used = given >= 0 && given < V;
    id[j] = used ? given : -1;
    y[j] = logit;
    return used;
  }
  // Whether slot j is the first of its id.
  __device__ __forceinline__ bool first(int j) const {
    for (int i = 0; i < j; ++i)
      if (id[i] == id[j]) return false;
    return true;
  }
  // What the teacher gives the id of slot j by the slots from `from` on: j if it is the id's first.
  __device__ __forceinline__ float all(int j, int from) const {
    float sum = 0.0f;
    for (int i = from; i < k; ++i) sum += id[i] == id[j] ? p[i] : 0.0f;
    return sum;
  }
};

// mass = sum_j p_j, rest = p_r, and the log-sum-exp that the teacher's logits are measured from: y_sum = sum 2^{c y - r} at
// the reference of y_max (without a tail) or lse.
struct Teacher {
  float mass, mass_low, rest, y_max, y_sum, y_low, lse;
  // With a tail: 1, or more if the log-sum-exp is not of these slots.
  __device__ __forceinline__ float all() const { return fmaxf(mass + mass_low, 1.0f); }
};

// A log-sum-exp in base 2, in two parts.
struct Lse {
  float lse, high, low;
  __device__ __forceinline__ explicit Lse(float lse_) : lse(lse_) {
    constexpr float kHigh = 1.44269502162933350f, kLow = 1.92596299e-8f;  // log2(e)
    high = __fmul_rn(lse, kHigh);
    low = fmaf(lse, kHigh, -high) + lse * kLow;
  }
  __device__ __forceinline__ bool small(float y) const { return fabsf(lse) < 1e30f && fabsf(y) < 1e30f; }
  // The base-2 logarithm of e^{y / t - lse}, and the number.
  __device__ __forceinline__ Two exponent(float y, Scale c) const {
    const float h = __fmul_rn(y, c);
    return Two{h - high, fmaf(y, c, -h) + (y * c.lo - low)};
  }
  __device__ __forceinline__ Two share(float y, Scale c) const {
    if (!small(y)) return Two{expf(fmaf(y, c.inv_t, -lse)), 0.0f};
    const Two l = exponent(y, c);
    return pow2(l.high, l.low);
  }
  __device__ __forceinline__ float ln_share(float y, Scale c) const {
    const Two l = exponent(y, c);
    return small(y) ? (l.high + l.low) * kLn2 : fmaf(y, c.inv_t, -lse);
  }
};

// By a warp; the slots' p_j are written.
__device__ __forceinline__ Teacher teach(const LogitsLossArgs& a, float top_lse, const Slots& s, Scale c, int lane) {
  Teacher r{0.0f, 0.0f, 0.0f, 0.0f, 1.0f, 0.0f, 0.0f};
  if (a.top_lse) {
    r.lse = top_lse;
  } else {
    r.y_max = -INFINITY;
    for (int j = lane; j < s.k; j += 32)
      if (s.id[j] >= 0) r.y_max = fmaxf(r.y_max, s.y[j]);
    r.y_max = warp_max(r.y_max);
    if (r.y_max == -INFINITY) r.y_max = 0.0f;
    const Ref ref(r.y_max, c);
    Two sum;
    for (int j = lane; j < s.k; j += 32) {
      Two p;
      if (s.id[j] >= 0) p = ref.far ? Two{expf((s.y[j] - ref.m) * c.inv_t), 0.0f} : ref.exactly(s.y[j], c);
      s.p[j] = p.high;
      sum.add(p);
    }
    sum.add_warp();
    r.y_sum = sum.high, r.y_low = sum.low;
  }
  const float norm = 1.0f / r.y_sum;
  const Lse lse(r.lse);
  Two mass;  // (what it leaves of 1 may be little)
  for (int j = lane; j < s.k; j += 32) {
    Two p;
    if (s.id[j] >= 0) p = a.top_lse ? lse.share(s.y[j], c) : Two{__fmul_rn(s.p[j], norm), 0.0f};
    mass.add(p);
    s.p[j] = p.high;
  }
  mass.add_warp();
  r.mass = mass.high, r.mass_low = mass.low;
  r.rest = a.top_lse ? fmaxf((1.0f - mass.high) - mass.low, 0.0f) : 0.0f;
  return r;
}

template <class E>
__device__ __forceinline__ void store_zeros(E* out, const Part<E>& part, int tid, int threads) {
  constexpr int N = kPer<E>;
  if (part.e0 >= part.e1) return;
  const int lead = lead_of(out), last = (part.e1 + lead + N - 1) / N;
  for (int g = (part.e0 + lead) / N + tid; g < last; g += threads) {
    const int f = g * N - lead;
    if (f >= part.e0 && f + N <= part.e1) {
      __stcs(reinterpret_cast<uint4*>(out + f), make_uint4(0, 0, 0, 0));
    } else {
      for (int e = max(f, part.e0); e < min(f + N, part.e1); ++e) out[e] = from_f32(0.0f, E{});
    }
  }
}

// The gradient outside the ids: e^{x / t} over that at `at`, times `scale`.
struct Gradient {
  Ref at;
  Scale c;
  float scale;
  __device__ __forceinline__ float operator()(float x) const { return at(x, c) * scale; }
  template <int N>
  __device__ __forceinline__ uint4 block(float (&x)[N]) const {
    if (!at.far) {
      const uint64_t c2 = f32x2(c, c), lo2 = f32x2(c.lo, c.lo), nr2 = f32x2(-at.r, -at.r), scale2 = f32x2(scale, scale);
#pragma unroll
      for (int u = 0; u < N; u += 2) {
        float y, z;
        const uint64_t both = f32x2(x[u], x[u + 1]);
        f32x2(fma2(both, lo2, fma2(both, c2, nr2)), y, z);
        f32x2(mul2(f32x2(ex2_approx(y), ex2_approx(z)), scale2), x[u], x[u + 1]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < N; ++u) x[u] = (*this)(x[u]);
    }
    return pack(x);
  }
};

// Whether a NaN or +inf is among logits, from a maximum that a NaN comes through.
struct NoWatch {
  __device__ __forceinline__ void add(uint4) {}
  __device__ __forceinline__ void add(float) {}
};
template <class E>
struct Watch {
  uint32_t top = sizeof(E) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -inf
  static __device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (sizeof(E) == 2) {
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    } else {
      float f;
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
      r = __float_as_uint(f);
    }
    return r;
  }
  __device__ __forceinline__ void add(uint4 g) { top = max_nan(top, max_nan(max_nan(g.x, g.y), max_nan(g.z, g.w))); }
  __device__ __forceinline__ void add(float x) {
    top = max_nan(top, sizeof(E) == 2 ? __float_as_uint(x) | 0xFF80u : __float_as_uint(x));  // (beside it: -inf)
  }
  __device__ __forceinline__ bool finite() const {
    if constexpr (sizeof(E) == 2) return bf16_lo(top) < INFINITY && bf16_hi(top) < INFINITY;
    else return __uint_as_float(top) < INFINITY;
  }
};

// The N elements of two granules from element r on.
template <class E>
__device__ __forceinline__ uint4 window(uint4 a, uint4 b, int r) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const int words = r * static_cast<int>(sizeof(E)) / 4;
  if (words & 2) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (words & 1) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (sizeof(E) == 2 && (r & 1)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The gradient of a part to its row of it, by load(granule), from a whole granule of the logits each. Where the two rows do
// not start alike, a granule of the gradient comes of two of the logits, the second from the next lane.
template <int kInFlight, class E, class W, class Load>
__device__ __forceinline__ void store_gradient(E* out, const Part<E>& part, const Gradient& of, W& watch, int tid, int threads,
                                               Load load) {
  constexpr int N = kPer<E>;
  const int lead = lead_of(out);
  // Element e0 .. of a granule, inside the part.
  auto some = [&](int e, uint4 g) {
    float x[N];
    unpack(g, x);
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (e + u >= part.e0 && e + u < part.e1) {
        watch.add(x[u]);
        out[e + u] = from_f32(of(x[u]), E{});
      }
  };
  auto whole = [&](int e, uint4 g) {
    watch.add(g);
    float x[N];
    unpack(g, x);
    __stcs(reinterpret_cast<uint4*>(out + e), of.block(x));
  };
  if (lead == part.lead) {
    stream<kInFlight>(part.whole0() + tid, part.whole1(), threads, load, [&](int i, uint4 g) { whole(i * N - lead, g); });
    part.cut(tid, threads, [&](int i) { some(i * N - lead, part.load_cut(i)); });
    return;
  }
  if (part.e0 >= part.e1) return;
  constexpr int kPairs = (kInFlight + 1) / 2;
  const int lane = tid & 31, w0 = part.whole0(), w1 = part.whole1();
  const int back = part.lead < lead ? 1 : 0, r = part.lead - lead + back * N;
  auto granule = [&](int i) {
    if (i >= w0 && i < w1) return load(i);
    return i >= part.g0 && i < part.g1 ? part.load_cut(i) : make_uint4(0, 0, 0, 0);
  };
  const int last = (part.e1 + lead + N - 1) / N;
  for (int g = (part.e0 + lead) / N + tid - lane; g < last; g += kPairs * threads) {
    uint4 a[kPairs], b[kPairs];
#pragma unroll
    for (int u = 0; u < kPairs; ++u) {
      const int i = g + u * threads + lane - back;
      a[u] = granule(i);
      b[u] = lane == 31 ? granule(i + 1) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kPairs; ++u) {
      const uint4 next = make_uint4(__shfl_down_sync(kAll, a[u].x, 1), __shfl_down_sync(kAll, a[u].y, 1),
                                    __shfl_down_sync(kAll, a[u].z, 1), __shfl_down_sync(kAll, a[u].w, 1));
      const uint4 x = window<E>(a[u], lane == 31 ? b[u] : next, r);
      const int e = (g + u * threads + lane) * N - lead;
      if (e >= part.e0 && e + N <= part.e1) whole(e, x);
      else some(e, x);
    }
  }
}

// And at the ids of this part, behind it: factor (q_j - p_j).
template <class E>
__device__ __forceinline__ void store_ids(E* out, const Part<E>& part, const Slots& s, bool twice, const Ref& ref, Scale c, float inv_s,
                                          float factor, int tid, int threads) {
  for (int j = tid; j < s.k; j += threads) {
    if (!part.has(s.id[j]) || (twice && !s.first(j))) continue;
    const float p = twice ? s.all(j, j) : s.p[j];
    out[s.id[j]] = from_f32(factor * (ref(s.x[j], c) * inv_s - p), E{});
  }
}

// What a CTA's threads tell one another about a row.
struct RowInfo {
  Teacher teacher;
  float m_top;               // the largest logit at the ids, the reference of the row's sums
  float weight, rollout;     // the gradient's, or the advantage; the token's log-probability in the rollout
  int again;                 // whether the sums are to be taken once more
  int twice;                 // whether slots share an id
  // references and sums of the whole row (and a low part of it), and of its logits outside the ids (with a tail); the sum at
  // the ids, -1 if it is not at m
  float m, s, s_low, s_top, m_out, s_out;
  float m_at, scale;         // the gradient outside the ids
  float inv_s, factor;       // and at them (q as it is weighed)
  float lse, lse_at;         // kBackward: known, of m and m_at
};

// To a row's loss, of slots that share an id: what p ln p of their sum has above the sum of theirs, each slot its part. (Rare, and
// behind the rest: within it, it puts the hot loops' variables of loss and gradient on the stack, 358 us for 350.)
__device__ __noinline__ void add_shared_ids(float* loss, const Slots s, int lane) {
  float more = 0.0f;
  for (int j = lane; j < s.k; j += 32)
    if (s.id[j] >= 0 && s.p[j] > 0.0f) more += s.p[j] * logf(fminf(s.all(j, 0) / s.p[j], FLT_MAX));
  more = warp_sum(more);
  if (lane == 0) *loss += more;
}

// The loss of a row, by a warp.
template <LossMode M>
__device__ __forceinline__ void write_loss(const LogitsLossArgs& a, int64_t t, const Slots& s, const RowInfo& info, Scale c, int lane) {
  const bool empty = info.m == -INFINITY, none = info.m_out == -INFINITY;
  const float sum = empty ? 1.0f : info.s, inv_t = c.inv_t;
  const Ref ref(info.m, c), ref_out(info.m_out, c), ref_y(info.teacher.y_max, c);
  const Log2 log2(ref, sum, empty ? 0.0f : info.s_low), log2_y(ref_y, info.teacher.y_sum, info.teacher.y_low);
  const Teacher& y = info.teacher;
  // ln p - ln q of one id is rounded as the small number that it mostly is: (y - x) / t less what the log-sum-exps differ by.
  const Lse teacher_lse(y.lse);
  const float apart = a.top_lse ? (teacher_lse.high - log2.whole) + (teacher_lse.low - log2.part)
                                : (log2_y.whole - log2.whole) + (log2_y.part - log2.part);
  const bool near = !ref.far && !ref_y.far && fabsf(y.lse) < 1e30f;
  float loss = 0.0f;
  for (int j = lane; j < s.k; j += 32)
    if (s.id[j] >= 0 && s.p[j] > 0.0f) {
      if (near && fabsf(s.x[j]) < 1e30f && fabsf(s.y[j]) < 1e30f) {
        loss += s.p[j] * (c.exponent(s.y[j] - s.x[j], apart) * kLn2);
        continue;
      }
      const float ln_p = a.top_lse ? teacher_lse.ln_share(s.y[j], c) : ln_share(s.y[j], ref_y, y.y_sum, log2_y, c);
      // (a share of a logit over t that is beyond fp32's range may be within)
      if (ref.far || !(fabsf(s.x[j]) < 1e30f)) loss += s.p[j] * (ln_p + logf(sum)) - s.p[j] * (s.x[j] - ref.m) * inv_t;
      else loss += s.p[j] * (ln_p - ln_share(s.x[j], ref, sum, log2, c));
    }
  loss = warp_sum(loss);
  if (lane != 0) return;
  float lse = ref.far ? ref.m * inv_t + logf(sum) : fmaf(log2.whole, kLn2, log2.part * kLn2), lse_out = lse;
  if (empty) lse = lse_out = -INFINITY;
  if (a.top_lse) {
    const Log2 log2_out(ref_out, none ? 1.0f : info.s_out);
    lse_out = none ? -INFINITY : ref_out.far ? ref_out.m * inv_t + logf(info.s_out) : fmaf(log2_out.whole, kLn2, log2_out.part * kLn2);
    if (y.rest > (none ? kDust : 0.0f)) {
      const bool far = ref.far || ref_out.far;
      const float ln_q = none  ? -INFINITY
                         : far ? logf(info.s_out) - logf(sum) + (ref.offset(c) - ref_out.offset(c)) * kLn2
                               : ((log2_out.whole - log2.whole) + (log2_out.part - log2.part)) * kLn2;
      if (far && !none) loss -= y.rest * (ref_out.m - ref.m) * inv_t;
      // Where most is outside the ids for both, ln (p_r / q_r) is that of 1 and little: (1 - mass) / (1 - q at the ids).
      const float q_top = info.s_top >= 0.0f ? info.s_top / sum : 1.0f;
      loss += y.rest * (q_top < 0.5f && y.mass < 0.5f ? log1pf(((q_top - y.mass) - y.mass_low) / (1.0f - q_top)) : logf(y.rest) - ln_q);
    }
  }
  a.loss[t] = loss;
  if constexpr (M == LossMode::kLoss) {
    a.stats[2 * t] = lse;
    a.stats[2 * t + 1] = lse_out;
  }
  if (!(fabsf(ref.m) < INFINITY) || !(sum < INFINITY) || !(y.mass < INFINITY)) flag(a.status, QRR_DEV_NONFINITE);
}

// The sum at the ids, each once, by a warp. `less`: less what the hardware's exponential made of them.
__device__ __forceinline__ Two sum_at_ids(const Slots& slots, const RowInfo& info, bool less, Scale c, int lane) {
  Two top;
  const Ref ref(info.m_top, c);
  for (int j = lane; j < slots.k; j += 32)
    if (slots.id[j] >= 0 && (!info.twice || slots.first(j))) {
      top.add(ref.exactly(slots.x[j], c));
      if (less) top.add(Two{-ref(slots.x[j], c), 0.0f});
    }
  top.add_warp();
  return top;
}

// What follows from the references and sums of the row (and a low part) and (with a tail) outside the ids, whose sum at the
// row's reference is q_rest. By a warp; `writes`: of the row's parts, this one writes what is the row's.
template <bool kPolicy>
__device__ __forceinline__ void conclude(const LogitsLossArgs& a, int64_t t, const Slots& slots, RowInfo& info, const Sum& all,
                                         float low, float top, const Sum& outside, float q_rest, bool tail, Scale c, int lane, bool writes) {
  const Ref ref(all.m, c);
  const bool bare = all.m == -INFINITY, none = outside.m == -INFINITY;
  const float sum = bare ? 1.0f : all.s;  // a row of -inf alone has no probabilities: q = 0
  float factor = info.weight * c.inv_t;
  if constexpr (kPolicy) {
    const float lp = ln_share(slots.x[0], ref, sum, Log2(ref, sum, low), c);
    float w = 1.0f;
    if (a.rollout_logp) {
      w = expf(lp - info.rollout);
      if (a.cap > 0.0f && w > a.cap) w = a.cap;  // (a NaN stays one)
    }
    factor *= w;
    if (writes && lane == 0) {
      a.logp[t] = lp;
      if (a.w) a.w[t] = w;
      if (!(fabsf(ref.m) < INFINITY) || !(sum < INFINITY) || !(w < INFINITY)) flag(a.status, QRR_DEV_NONFINITE);
    }
  }
  if (lane == 0) {
    const float inv_s = 1.0f / sum;
    info.m = all.m, info.s = all.s, info.s_low = low, info.s_top = top, info.m_out = outside.m, info.s_out = outside.s;
    info.m_at = tail ? outside.m : all.m;
    const float all_by_s = tail ? info.teacher.all() * inv_s : inv_s;
    info.scale = !tail ? factor * inv_s : none ? 0.0f : factor * (q_rest * all_by_s - info.teacher.rest) / outside.s;
    info.inv_s = all_by_s;
    info.factor = factor;
  }
}

// From sums at the reference of the ids. False if that served badly: the sums that are divided by have to be there, far
// from the ends of fp32's range.
template <bool kPolicy>
__device__ __forceinline__ bool conclude_first(const LogitsLossArgs& a, int64_t t, const Slots& slots, RowInfo& info, const Two& top,
                                               float total, bool tail, Scale c, int lane, bool writes) {
  auto served = [](float x) { return x > 0x1p-60f && x < 0x1p64f; };
  Two sum{total, 0.0f};
  sum.add(top);
  const Sum outside{info.m_top, tail ? total : sum.high}, all{info.m_top, sum.high};
  if (!served(all.s) || (tail && !served(total)) || all.m == -INFINITY) return false;
  conclude<kPolicy>(a, t, slots, info, all, sum.low, top.high, outside, total, tail, c, lane, writes);
  return true;
}

// From sums at the largest logits.
template <bool kPolicy>
__device__ __forceinline__ void conclude_largest(const LogitsLossArgs& a, int64_t t, const Slots& slots, RowInfo& info, const Two& top,
                                                 const Sum& outside, bool tail, Scale c, int lane, bool writes) {
  Sum all = outside;
  if (tail) all.merge(info.m_top, top.high, c);
  conclude<kPolicy>(a, t, slots, info, all, 0.0f, -1.0f, outside, outside.s * Sum::moved(outside.m, Ref(all.m, c), c), tail, c, lane, writes);
}

// The reference of a known log-sum-exp, a whole number too, and the factor of its row's shares that is left.
__device__ __forceinline__ Ref known_ref(float lse, Scale c) {
  Ref ref(lse * c.t, c);
  if (!ref.far && lse > -INFINITY) ref.r = rintf(Lse(lse).high);
  return ref;
}
__device__ __forceinline__ float known_share(float lse, Scale c) {
  const Ref ref = known_ref(lse, c);
  const Lse parts(lse);
  return !ref.far && lse > -INFINITY ? pow2(ref.r - parts.high, -parts.low).high : 1.0f;
}

// From known log-sum-exps. By one thread.
__device__ __forceinline__ void conclude_known(const LogitsLossArgs& a, int64_t t, RowInfo& info, Scale c) {
  const bool tail = a.top_lse;
  const float lse = __ldg(a.stats_in + 2 * t), lse_out = __ldg(a.stats_in + 2 * t + 1);
  info.lse = lse;
  info.lse_at = tail ? lse_out : lse;
  info.factor = info.weight * c.inv_t;
  const float all = tail ? info.teacher.all() : 1.0f;
  info.inv_s = known_share(lse, c) * all;
  info.scale = !tail                  ? info.factor * info.inv_s
               : lse_out == -INFINITY ? 0.0f
                                      : info.factor * (ex2_approx((lse_out - lse) * kLog2e) * all - info.teacher.rest) *
                                            known_share(lse_out, c);
  if (!(info.teacher.mass < INFINITY) || !(lse < INFINITY) || !(info.lse_at < INFINITY)) flag(a.status, QRR_DEV_NONFINITE);
}

// Granule g without the marked elements.
template <class E>
__device__ __forceinline__ uint4 without(uint4 g, uint32_t marked) {
  if (marked == 0) return g;
  float x[kPer<E>];
  unpack(g, x);
#pragma unroll
  for (int u = 0; u < kPer<E>; ++u)
    if (marked >> u & 1u) x[u] = -INFINITY;
  return pack(x);
}

// The granules of a part that have ids, in shared memory: a table of a power of two of places, at most half of them used. Of
// each the elements at ids (a bit each) and its first slot.
struct Marked {
  int* granule;  // -1: an empty place
  uint32_t* bits;
  int* slot;
  int places;
  static __host__ __device__ __forceinline__ int places_for(int k) {
    int n = 32;
    while (n < 2 * k) n *= 2;
    return n;
  }
  static __host__ __device__ __forceinline__ int bytes_for(int k) { return 12 * places_for(k); }
  __device__ __forceinline__ Marked(uint8_t* at, int k) : granule(reinterpret_cast<int*>(at)), places(places_for(k)) {
    bits = reinterpret_cast<uint32_t*>(granule + places);
    slot = reinterpret_cast<int*>(bits + places);
  }
  __device__ __forceinline__ void clear(int tid, int threads) const {
    for (int i = tid; i < places; i += threads) granule[i] = -1, bits[i] = 0, slot[i] = kMaxTop;
  }
  __device__ __forceinline__ int start(int g) const {  // multiplicative hashing, by the golden ratio
    return static_cast<int>(static_cast<uint32_t>(g) * 2654435769u >> 16) & (places - 1);
  }
  // True if the element was marked before, which is another slot's doing.
  __device__ __forceinline__ bool mark(int g, int element, int j) const {
    int i = start(g);
    for (;; i = (i + 1) & (places - 1)) {
      const int was = atomicCAS(&granule[i], -1, g);
      if (was == -1 || was == g) break;
    }
    atomicMin(&slot[i], j);
    return atomicOr(&bits[i], 1u << element) >> element & 1u;
  }
  // Its place, -1 if it has no ids.
  __device__ __forceinline__ int find(int g) const {
    for (int i = start(g);; i = (i + 1) & (places - 1)) {
      if (granule[i] == g) return i;
      if (granule[i] == -1) return -1;
    }
  }
};

// Granule i of a part without the elements at ids.
template <class E>
__device__ __forceinline__ uint4 without_ids(const Marked& marked, int i, uint4 g) {
  const int at = marked.find(i);
  return at < 0 ? g : without<E>(g, marked.bits[at]);
}

// A warp's sum of a part, outside the ids if that is wanted, once more at its largest logits.
template <class E>
__device__ __noinline__ Sum sum_again(const Part<E> part, const Marked marked, bool outside, int tid, int threads, Scale c) {
  Sum sum;
  auto add = [&](int i, uint4 g) {
    if (outside) g = without_ids<E>(marked, i, g);
    float x[kPer<E>];
    unpack(g, x);
    sum.add_largest(x, max_of(x), c);
  };
  for (int i = part.whole0() + tid; i < part.whole1(); i += threads) add(i, part.granules()[i]);
  part.cut(tid, threads, [&](int i) { add(i, part.load_cut(i)); });
  sum.merge_warp(c);
  return sum;
}

// Bytes that say which granules a thread passes over, one for `in_flight` of them.
__host__ __device__ __forceinline__ int skip_bytes(int per, int threads, int in_flight) {
  return (per + threads * in_flight - 1) / (threads * in_flight) * threads;
}

// ---- losses -------------------------------------------------------------------------
//
// A CTA takes part blockIdx.x % parts of row blockIdx.x / parts: `per` granules. The parts of a row are a cluster.
//
// The gradient may be written over the logits, which are therefore read by plain loads, not by those of constant memory.
//
// A gradient reads its row again, so what counts is that it is still in L2: two CTAs of 512 threads an SM with eight
// granules a thread under way (three and four CTAs of 256 threads: 375 us became 400 and 419 for loss and gradient of 4096 rows).
// A loss alone reads once: four CTAs of 256 threads hide one another's ends (2048 rows of 128256 bf16: 76 us; six with four
// granules 77, eight of 128 threads 78, two of 512 87). Rows cut between CTAs where one each would do: 90 us and more.
template <LossMode M>
struct Shape {
  static constexpr bool kTwice = M != LossMode::kLoss;
  static constexpr int kThreads = kTwice ? 512 : 256, kCtas = kTwice ? 2 : 4, kInFlight = 8;
};

template <class E, LossMode M>
__global__ void __launch_bounds__(Shape<M>::kThreads, Shape<M>::kCtas) logits_loss_kernel(const LogitsLossArgs a, const int parts,
                                                                                              const int per) {
  constexpr int N = kPer<E>;
  constexpr bool kPolicy = M == LossMode::kPolicy, kWrites = M != LossMode::kLoss;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads / 32;
  const int64_t t = blockIdx.x / parts;
  const int rank = blockIdx.x % parts, k = kPolicy ? 1 : a.k;
  const Part<E> part(static_cast<const E*>(a.logits) + t * a.ld, a.V, rank, per);
  E* const out = kWrites ? static_cast<E*>(a.dlogits) + t * a.ldd : nullptr;
  const Scale c = a.scale;
  const bool tail = !kPolicy && a.top_lse;

  constexpr int kInFlight = Shape<M>::kInFlight;
  extern __shared__ __align__(16) uint8_t smem[];
  const Slots slots(smem, k);
  const Marked marked(smem + 16 * k, k);
  // a byte for each kInFlight granules of a thread, a bit a granule
  uint32_t* const skips = reinterpret_cast<uint32_t*>(smem + 16 * k + Marked::bytes_for(k));
  const int w0 = part.whole0(), w1 = part.whole1();
  __shared__ RowInfo info;
  __shared__ float2 sums[kMaxThreads / 32];
  __shared__ float2 shares[2][kMaxParts];  // of every part: sum and whether slots share an id; the second time reference and sum

  float weight = 0.0f, rollout = 0.0f;
  if (kWrites) weight = __ldg((kPolicy ? a.advantages : a.grad) + t);
  if (kPolicy && a.rollout_logp) rollout = __ldg(a.rollout_logp + t);
  const float top_lse = tail ? __ldg(a.top_lse + t) : 0.0f;
  bool any = false;
  for (int j = tid; j < k; j += threads)
    any |= slots.set(j, __ldg(kPolicy ? a.tokens + t : a.ids + t * k + j), kPolicy ? 0.0f : __ldg(a.top + t * k + j), a.V, a.status);
  if constexpr (!kPolicy) {
    marked.clear(tid, threads);
    for (int i = tid; i < skip_bytes(per, threads, kInFlight) / 16; i += threads)
      reinterpret_cast<uint4*>(skips)[i] = make_uint4(0, 0, 0, 0);
  }
  if (tid == 0) {
    info.weight = weight;
    info.rollout = rollout;
    info.twice = 0;
    if constexpr (kPolicy) slots.p[0] = 1.0f;
  }
  if (parts > 1) cluster_arrive();  // this CTA runs
  if (!__syncthreads_or(any)) {     // nothing to learn: the whole cluster ends here
    if constexpr (kWrites) store_zeros(out, part, tid, threads);
    if (rank == 0 && tid == 0) {
      if constexpr (M == LossMode::kLoss || M == LossMode::kGrad) a.loss[t] = 0.0f;
      if constexpr (M == LossMode::kLoss) a.stats[2 * t] = a.stats[2 * t + 1] = 0.0f;
      if constexpr (kPolicy) {
        a.logp[t] = 0.0f;
        if (a.w) a.w[t] = 0.0f;
      }
    }
    if (parts > 1) cluster_wait();
    return;
  }

  // The logits at the ids, and marks of their granules here. No part writes a gradient before all have been here, as sums are
  // joined in between. With a tail, a granule with an id is left to the thread of its first slot: the others have one byte to
  // look at for kInFlight granules. (With a mark for every element, and a byte a granule to look at by the thread that comes to
  // it: 388 us in the place of 349 for loss and gradient of 4096 rows.)
  const uint4* const granules = part.granules();
  uint4 mine = make_uint4(0, 0, 0, 0);  // of this thread's first slot
  for (int j = tid; j < k; j += threads) {
    const int id = slots.id[j];
    if (id < 0) continue;
    slots.x[j] = to_f32(part.row[id]);
    const int g = kPolicy ? -1 : part.granule_of(id);
    if (g < 0) continue;
    if (marked.mark(g, (id - part.base) % N, j)) info.twice = 1;
    if (tail && g >= w0 && g < w1) {
      if (j == tid) mine = granules[g];
      const int n = (g - w0) / threads, at = n / kInFlight * threads + (g - w0) % threads;
      atomicOr(&skips[at / 4], 1u << (8 * (at % 4) + n % kInFlight));
    }
  }
  __syncthreads();
  float m_top = -INFINITY;
  for (int j = lane; j < k; j += 32)
    if (slots.id[j] >= 0) m_top = fmaxf(m_top, slots.x[j]);
  m_top = warp_max(m_top);
  if (tid == 0) info.m_top = m_top;
  {
    const Ref ref(m_top, c);
    constexpr uint32_t kNothing = sizeof(E) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -inf
    const uint4 nothing = make_uint4(kNothing, kNothing, kNothing, kNothing);
    const uint64_t hint = kWrites ? read_again() : read_once();
    auto load = [&](int i) { return load_hint(granules + i, hint); };
    FixedSum<E> fixed;
    fixed.start(ref, c);
    if (!kPolicy && tail)
      for (int j = tid; j < k; j += threads) {
        const int id = slots.id[j], g = part.granule_of(id);
        if (g < w0 || g >= w1) continue;
        const int at = marked.find(g);
        if (marked.slot[at] == j) fixed.add(without<E>(j == tid ? mine : load(g), marked.bits[at]));
      }
    const uint8_t* skip = reinterpret_cast<const uint8_t*>(skips) + tid;
    for (int i = w0 + tid; i < w1; i += kInFlight * threads, skip += threads) {
      uint4 g[kInFlight];
      if (i + (kInFlight - 1) * threads < w1) {
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) g[u] = load(i + u * threads);
      } else {
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
          g[u] = nothing;
          if (i + u * threads < w1) g[u] = load(i + u * threads);
        }
      }
      if (!kPolicy && tail) {
        const uint32_t not_here = *skip;
        if (not_here != 0) {
#pragma unroll
          for (int u = 0; u < kInFlight; ++u)
            if (not_here >> u & 1u) g[u] = nothing;
        }
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) fixed.add(g[u]);
    }
    part.cut(tid, threads, [&](int i) {
      const uint4 g = part.load_cut(i);
      fixed.add(!kPolicy && tail ? without_ids<E>(marked, i, g) : g);
    });
    const float mine = warp_sum(ref.far ? INFINITY : fixed.total());
    if (lane == 0) sums[warp] = make_float2(mine, 0.0f);
    if (!kPolicy && warp == warps - 1) {
      const Teacher y = teach(a, top_lse, slots, c, lane);
      if (lane == 0) info.teacher = y;
    }
    __syncthreads();

    // What warp 0 has of all parts: each one's `of` in the lane of its number.
    auto exchange = [&](int round, float2 of) {
      if (parts == 1) return lane == 0 ? of : make_float2(round ? -INFINITY : 0.0f, 0.0f);
      if (round == 0) cluster_wait();  // every CTA runs
      if (warp == 0 && lane < parts) st_cluster(&shares[round][rank], lane, of);
      cluster_arrive();
      cluster_wait();
      return lane < parts ? shares[round][lane] : make_float2(round ? -INFINITY : 0.0f, 0.0f);
    };
    float2 of = make_float2(0.0f, 0.0f);
    if (warp == 0) of = make_float2(warp_sum(lane < warps ? sums[lane].x : 0.0f), info.twice ? 1.0f : 0.0f);
    of = exchange(0, of);
    Two top;  // at the ids, the largest terms mostly: with a tail they are not in the sum, without they are put right
    if (warp == 0) {
      const float total = warp_sum(of.x);
      const bool twice = __any_sync(kAll, of.y != 0.0f);
      if (lane == 0) info.twice = twice;
      __syncwarp();
      top = sum_at_ids(slots, info, !tail, c, lane);
      const bool served = conclude_first<kPolicy>(a, t, slots, info, top, total, tail, c, lane, rank == 0);
      if (lane == 0) info.again = !served;
    }
    __syncthreads();
    if (info.again) {
      const Sum largest = sum_again<E>(part, marked, !kPolicy && tail, tid, threads, c);
      if (lane == 0) sums[warp] = make_float2(largest.m, largest.s);
      __syncthreads();
      Sum outside;
      if (warp == 0) {
        if (lane < warps) outside = Sum{sums[lane].x, sums[lane].y};
        outside.merge_warp(c);
      }
      of = exchange(1, make_float2(outside.m, outside.s));
      if (warp == 0) {
        outside = Sum{of.x, of.y};
        outside.merge_warp(c);
        conclude_largest<kPolicy>(a, t, slots, info, top, outside, tail, c, lane, rank == 0);
      }
      __syncthreads();
    }
  }

  if constexpr (kWrites) {
    const uint64_t hint = read_once();
    NoWatch none;  // (the sums have seen them all)
    store_gradient<Shape<M>::kInFlight>(out, part, Gradient{Ref(info.m_at, c), c, info.scale}, none, tid, threads,
                                        [&](int i) { return load_hint(granules + i, hint); });
    __syncthreads();
    store_ids(out, part, slots, info.twice, Ref(info.m, c), c, info.inv_s, info.factor, tid, threads);
  }
  if ((M == LossMode::kLoss || M == LossMode::kGrad) && rank == 0 && warp == warps - 1) {
    write_loss<M>(a, t, slots, info, c, lane);
    if (info.twice) add_shared_ids(a.loss + t, slots, lane);
  }
}

// ---- the gradient from known log-sum-exps ------------------------------------------
//
// Part blockIdx.x % parts of row blockIdx.x / parts, with nothing to exchange: a tile by bulk copies, three CTAs an SM.
template <class E>
__global__ void __launch_bounds__(kBackwardThreads) logits_backward_kernel(const LogitsLossArgs a, const int parts, const int per) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, k = a.k;
  const int64_t t = blockIdx.x / parts;
  E* const out = static_cast<E*>(a.dlogits) + t * a.ldd;
  const Part<E> part(static_cast<const E*>(a.logits) + t * a.ld, a.V, blockIdx.x % parts, per);
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* const tile = reinterpret_cast<uint4*>(smem);
  E* const held = reinterpret_cast<E*>(smem);
  const Slots slots(smem + 16 * per, k);
  __shared__ uint64_t loaded;
  __shared__ int abort;
  __shared__ RowInfo info;
  const Scale c = a.scale;
  const float top_lse = a.top_lse ? __ldg(a.top_lse + t) : 0.0f;
  if (tid == 0) {
    mbar_init(&loaded, 1);
    fence_barrier_init();
    abort = 0;
  }
  bool any = false;
  for (int j = tid; j < k; j += threads) {
    any |= slots.set(j, __ldg(a.ids + t * k + j), __ldg(a.top + t * k + j), a.V, a.status);
  }
  if (!__syncthreads_or(any)) {
    store_zeros(out, part, tid, threads);
    return;
  }
  if (tid == 0) part.copy(tile, &loaded);
  part.cut(tid, threads, [&](int i) { tile[i - part.g0] = part.load_cut(i); });
  Watch<E> watch;
  for (int j = tid; j < k; j += threads)
    if (part.has(slots.id[j])) watch.add(slots.x[j] = to_f32(part.row[slots.id[j]]));
  if (warp == 0) {
    const Teacher y = teach(a, top_lse, slots, c, lane);
    if (lane == 0) {
      info.teacher = y;
      info.weight = __ldg(a.grad + t);
      conclude_known(a, t, info, c);
    }
  }
  mbar_wait(&loaded, 0, &abort, a.status);
  __syncthreads();
  // Slots that name one id find out by writing their numbers to its place, which store_ids fills in the end (small numbers, as
  // `watch` sees them).
  bool twice = false;
  for (int j = tid; j < k; j += threads)
    if (part.has(slots.id[j])) {
      if constexpr (sizeof(E) == 2) held[slots.id[j] - part.base] = static_cast<E>(j);
      else held[slots.id[j] - part.base] = __int_as_float(j);
    }
  __syncthreads();
  for (int j = tid; j < k; j += threads)
    if (part.has(slots.id[j])) {
      if constexpr (sizeof(E) == 2) twice |= held[slots.id[j] - part.base] != j;
      else twice |= __float_as_int(held[slots.id[j] - part.base]) != j;
    }
  twice = __syncthreads_or(twice);

  const Ref ref = known_ref(info.lse, c);
  const Gradient of{known_ref(info.lse_at, c), c, info.scale};
  store_gradient<1>(out, part, of, watch, tid, threads, [&](int i) { return tile[i - part.g0]; });
  if (!watch.finite()) flag(a.status, QRR_DEV_NONFINITE);
  __syncthreads();
  store_ids(out, part, slots, twice, ref, c, info.inv_s, info.factor, tid, threads);
}

constexpr int kMaxSmem = 220 << 10;  // of a CTA, beside what is declared

cudaError_t device(int& dev, int& sms) {
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
}

template <class E, LossMode M>
cudaError_t launch(const LogitsLossArgs& a, cudaStream_t stream) {
  int dev = 0, sms = kSMs;
  cudaError_t e = device(dev, sms);
  if (e != cudaSuccess) return e;
  const int granules = granules_of<E>(kPer<E> - 1, a.V);
  int parts = 1;  // more where rows do not fill the SMs
  while (parts < kMaxParts && a.T * parts < sms && granules > parts * 256) parts *= 2;
  const int per = (granules + parts - 1) / parts;
  // Threads: few rows are done with the soonest by many; where CTAs follow one another, more of them hide what each does
  // beside its granules, so a thread has 32 of these (16 without a teacher). 3174 rows of 32000 bf16: loss and gradient 93 us,
  // loss 51, policy gradient 66; with 512 (loss: 256) threads 134, 59 and 81. 300 rows of 32003: 12.6 us, with 256 threads 12.8.
  int threads = per >= 2048 ? 512 : per >= 1024 ? 256 : per >= 256 ? 128 : 64;
  if (a.T > 2 * sms) {
    threads = 64;
    while (threads < 512 && per > threads * (M == LossMode::kPolicy ? 16 : 32)) threads *= 2;
  }
  threads = std::min(threads, Shape<M>::kThreads);
  size_t smem = 16;
  if (M != LossMode::kPolicy) smem = 16 * static_cast<size_t>(a.k) + Marked::bytes_for(a.k) + skip_bytes(per, threads, Shape<M>::kInFlight);
  static OncePerDevice limit;
  e = limit(dev, [] { return cudaFuncSetAttribute(logits_loss_kernel<E, M>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem); });
  if (e != cudaSuccess) return e;
  return launch_clusters(logits_loss_kernel<E, M>, static_cast<unsigned>(a.T * parts), parts, threads, smem, stream, a, parts, per);
}

template <class E>
cudaError_t launch_backward(const LogitsLossArgs& a, cudaStream_t stream) {
  int dev = 0, sms = kSMs;
  cudaError_t e = device(dev, sms);
  if (e != cudaSuccess) return e;
  constexpr int kPartBytes = 64 << 10;
  const int granules = granules_of<E>(kPer<E> - 1, a.V);
  int parts = 1;
  while (parts < 32 && (granules * 16 > parts * kPartBytes || (a.T * parts < sms && granules > parts * 256))) parts *= 2;
  const int per = (granules + parts - 1) / parts;
  const int threads = per >= 1024 ? 256 : per >= 256 ? 128 : 64;
  static OncePerDevice limit;
  e = limit(dev, [] { return cudaFuncSetAttribute(logits_backward_kernel<E>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem); });
  if (e != cudaSuccess) return e;
  logits_backward_kernel<E><<<static_cast<unsigned>(a.T * parts), threads, 16 * static_cast<size_t>(per + a.k), stream>>>(a, parts, per);
  return cudaGetLastError();
}

template <class E>
cudaError_t launch(const LogitsLossArgs& a, LossMode mode, cudaStream_t stream) {
  switch (mode) {
    case LossMode::kLoss: return launch<E, LossMode::kLoss>(a, stream);
    case LossMode::kGrad: return launch<E, LossMode::kGrad>(a, stream);
    case LossMode::kBackward: return launch_backward<E>(a, stream);
    default: return launch<E, LossMode::kPolicy>(a, stream);
  }
}

}  // namespace

cudaError_t launch_logits_loss(LogitsLossArgs a, LossMode mode, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  a.scale = scale_of(mode == LossMode::kPolicy ? 1.0 : a.temperature);
  return a.fp32 ? launch<float>(a, mode, stream) : launch<Bf16>(a, mode, stream);
}

}  // namespace qrr
