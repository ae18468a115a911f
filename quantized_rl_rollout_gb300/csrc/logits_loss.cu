// Losses over rows of logits with their gradients: distillation from a teacher's top logits, and the policy gradient of the
// tokens that a rollout took.
//
// Distillation, x a row of V logits, t the temperature, q = softmax(x / t), the teacher's top logits y_j at the ids i_j:
//   without a tail   p_j = e^{y_j / t} / sum_i e^{y_i / t},  L = sum_j p_j (ln p_j - ln q_{i_j})
//   with a tail      p_j = e^{y_j / t - lse_teacher}, p_r = 1 - sum_j p_j, q_r = 1 - sum_j q_{i_j},
//                    L = sum_j p_j (ln p_j - ln q_{i_j}) + p_r (ln p_r - ln q_r)
//   dL/dx_v = (q_v - p_v) / t; with a tail, outside the ids, e^{x_v / t - lse_r} (q_r - p_r) / t, lse_r the log-sum-exp of
//   the logits outside. Slots that name one id add up.
// Policy gradient of token a with advantage A: logp = x_a - lse, w = min(e^{logp - logp_rollout}, cap),
//   d(-A w logp)/dx_v = A w (q_v - [v = a]), w held fixed: the same form with p_a = 1 and the factor A w.
//
// Bound by memory: a logit is read once and its gradient written once (the loss alone only reads). The two sums of a row are
// known when all of it has been read, so it stays on chip until then: a cluster of CTAs holds it in shared memory, a
// contiguous part each, and joins maxima and sums over distributed shared memory.
//
// The logits at the teacher's ids are taken out of the held row (-inf in their place), so that the sum outside them is one
// of positive terms, not a difference. Sums are fp32; e^x is the hardware's base-2 approximation (about 2^-22 relative)
// where it is taken a logit and expf where it is taken an id; a loss is a small difference of large logarithms, and its k
// terms are added in 64 bits.
#include "logits.cuh"
#include "once_per_device.cuh"

namespace qrr {

namespace {

constexpr int kMaxThreads = 256;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kLn2 = 0.6931471805599453f;
// A rest of the teacher's that is no more than the rounding of its log-sum-exp and of the sum of p_j: beside a student
// without any, it is none.
constexpr float kDust = 1.0f / 65536;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// out[e0 .. e1) of a row = value(e), whole granules at once: block(e) gives those of kPer elements from e on.
template <class E, class Block, class One>
__device__ __forceinline__ void store_range(E* out, int e0, int e1, Block block, One one) {
  constexpr int N = kPer<E>;
  const int lead = lead_of(out);
  const int first = (e0 + lead) / N, last = (e1 + lead + N - 1) / N;
  for (int g = first + threadIdx.x; g < last; g += blockDim.x) {
    const int f = g * N - lead;
    if (f >= e0 && f + N <= e1) {
      __stcs(reinterpret_cast<uint4*>(out + f), block(f));
    } else {
      for (int e = max(f, e0); e < min(f + N, e1); ++e) out[e] = one(e);
    }
  }
}

// A CTA takes part rank of `parts` of row blockIdx.x / parts: `per` granules. In every mode but kBackward, whose sums are
// known, the parts of a row are a cluster.
//
// A part's life is a chain of short steps (ids, row, sum, exchange, gradient), and several parts an SM hide one
// another's: what does not need the row (the teacher, the logits at its ids, read beside the row by every part) is done
// while the row is on its way, and the exchange writes a part's sum into the other CTAs ahead of the barrier, so that
// behind it everything is at hand.
template <class E, LossMode M>
__global__ void __launch_bounds__(kMaxThreads) logits_loss_kernel(const LogitsLossArgs a, const int parts, const int per) {
  constexpr int N = kPer<E>;
  constexpr bool kPolicy = M == LossMode::kPolicy, kWrites = M != LossMode::kLoss, kSums = M != LossMode::kBackward;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const int64_t t = blockIdx.x / parts;
  const int rank = blockIdx.x % parts, k = kPolicy ? 1 : a.k, V = a.V;
  const E* const row = static_cast<const E*>(a.logits) + t * a.ld;
  E* const out = kWrites ? static_cast<E*>(a.dlogits) + t * a.ldd : nullptr;

  extern __shared__ __align__(16) uint8_t smem[];
  uint4* const tile = reinterpret_cast<uint4*>(smem);
  E* const held = reinterpret_cast<E*>(smem);
  int* const sid = reinterpret_cast<int*>(tile + per);  // id of a slot, -1: unused
  float* const sy = reinterpret_cast<float*>(sid + k);  // the teacher's logit
  float* const sp = sy + k;                             // its probability
  float* const sx = sp + k;                             // the row's logit
  __shared__ uint64_t loaded;
  __shared__ float4 shares[8 * kMaxThreads / 32];  // of every part's warps: reference and sum outside the ids, whether slots share one
  __shared__ int abort, twice_here;

  const int lead = lead_of(row), granules = granules_of<E>(lead, V);
  const int g0 = min(rank * per, granules), g1 = min(g0 + per, granules), base = g0 * N - lead;
  const int e0 = max(base, 0), e1 = min(g1 * N - lead, V);  // this part's elements

  if (tid == 0) {
    mbar_init(&loaded, 1);
    fence_barrier_init();
    abort = twice_here = 0;
  }
  bool any = false;
  for (int j = tid; j < k; j += threads) {
    int id = __ldg(kPolicy ? a.tokens + t : a.ids + t * k + j);
    if constexpr (!kPolicy) sy[j] = __ldg(a.top + t * k + j);
    if (id >= V) {
      flag(a.status, QRR_DEV_BAD_INDEX);
      id = -1;
    }
    sid[j] = id;
    any |= id >= 0;
  }
  if (kSums && parts > 1) cluster_arrive();  // this CTA runs
  if (!__syncthreads_or(any)) {              // nothing to learn: the whole cluster ends here
    if constexpr (kWrites)
      if (e0 < e1)
        store_range(out, e0, e1, [](int) { return make_uint4(0, 0, 0, 0); }, [](int) { return from_f32(0.0f, E{}); });
    if (rank == 0 && tid == 0) {
      if constexpr (M == LossMode::kLoss || M == LossMode::kGrad) a.loss[t] = 0.0f;
      if constexpr (M == LossMode::kLoss) a.stats[2 * t] = a.stats[2 * t + 1] = 0.0f;
      if constexpr (kPolicy) {
        a.logp[t] = 0.0f;
        if (a.w) a.w[t] = 0.0f;
      }
    }
    if (kSums && parts > 1) cluster_wait();
    return;
  }

  // The part's whole granules by bulk copies, the row's cut ones by a thread each.
  const int whole0 = base < 0 ? g0 + 1 : g0, whole1 = g1 > g0 && g1 * N - lead > V ? g1 - 1 : g1;
  if (tid == 0) {
    const uint32_t bytes = whole1 > whole0 ? 16u * static_cast<uint32_t>(whole1 - whole0) : 0u;
    mbar_arrive_expect_tx(&loaded, bytes);
    constexpr uint32_t kChunk = 16 << 10;
    const uint8_t* const src = reinterpret_cast<const uint8_t*>(row + (whole0 * N - lead));
    for (uint32_t at = 0; at < bytes; at += kChunk)
      bulk_load(reinterpret_cast<uint8_t*>(tile + (whole0 - g0)) + at, src + at, min(kChunk, bytes - at), &loaded);
  }
  if (tid == threads - 1 && g0 < g1) {
    if (whole0 > g0) tile[0] = load_cut(row, base, V);
    if (whole1 < g1 && (whole1 > g0 || whole0 == g0)) tile[whole1 - g0] = load_cut(row, whole1 * N - lead, V);
  }
  // The logits at the ids: of every id (no part writes a gradient over them before the exchange); without an exchange, of
  // this part's alone. Each thread's first is on its way until it is wanted.
  auto wanted = [&](int j) { return j < k && (kSums ? sid[j] >= 0 : sid[j] >= e0 && sid[j] < e1); };
  const E x_first = wanted(tid) ? row[sid[tid]] : E{};
  for (int j = tid + threads; j < k; j += threads)
    if (wanted(j)) sx[j] = to_f32(row[sid[j]]);

  // The teacher, by every warp on its own: mass = sum_j p_j, and the log-sum-exp that its logits are measured from as
  // y_max / t + ln y_sum (without a tail) or lse_teacher.
  const float inv_t = kPolicy ? 1.0f : 1.0f / a.temperature, c = kLog2e * inv_t;
  const bool tail = !kPolicy && a.top_lse;
  float mass = 1.0f, y_max = 0.0f, y_sum = 1.0f, lse_teacher = 0.0f;
  if constexpr (kPolicy) {
    if (tid == 0) sp[0] = 1.0f;
  } else {
    if (tail) {
      lse_teacher = __ldg(a.top_lse + t);
    } else {
      y_max = -INFINITY;
      for (int j = lane; j < k; j += 32)
        if (sid[j] >= 0) y_max = fmaxf(y_max, sy[j]);
      y_max = warp_max(y_max);
      if (y_max == -INFINITY) y_max = 0.0f;
      y_sum = 0.0f;
      for (int j = lane; j < k; j += 32)
        if (sid[j] >= 0) y_sum += expf((sy[j] - y_max) * inv_t);
      y_sum = warp_sum(y_sum);
    }
    mass = 0.0f;
    const float norm = 1.0f / y_sum;
    for (int j = lane; j < k; j += 32) {
      float p = 0.0f;
      if (sid[j] >= 0) p = tail ? expf(fmaf(sy[j], inv_t, -lse_teacher)) : expf((sy[j] - y_max) * inv_t) * norm;
      mass += p;
      if (warp == 0) sp[j] = p;
    }
    mass = warp_sum(mass);
  }
  const float rest = tail ? fmaxf(1.0f - mass, 0.0f) : 0.0f;  // p_r

  // The ids' logits are taken out of the part. Slots that name one id find out by writing their numbers to its place.
  mbar_wait(&loaded, 0, &abort, a.status);
  auto number = [](int j) {
    if constexpr (sizeof(E) == 2) return static_cast<E>(j);
    else return __int_as_float(j);
  };
  auto bits = [](E x) {
    if constexpr (sizeof(E) == 2) return static_cast<int>(x);
    else return __float_as_int(x);
  };
  if (wanted(tid)) sx[tid] = to_f32(x_first);
  __syncthreads();  // the cut granules
  for (int j = tid; j < k; j += threads)
    if (sid[j] >= e0 && sid[j] < e1) held[sid[j] - base] = number(j);
  __syncthreads();
  for (int j = tid; j < k; j += threads)
    if (sid[j] >= e0 && sid[j] < e1) {
      if (bits(held[sid[j] - base]) != j) twice_here = 1;
      held[sid[j] - base] = minus_inf<E>();
    }
  __syncthreads();

  // Of the whole row: references and sums outside the ids and at them.
  float m_out, s_out, m, s, known = 0.0f, known_out = 0.0f;
  bool twice = twice_here;
  // the first slot of its id, where some share one
  auto first = [&](int j) {
    for (int i = 0; i < j; ++i)
      if (sid[i] == sid[j]) return false;
    return true;
  };
  if constexpr (kSums) {
    Sum mine;
    const int n = (g1 - g0 - tid + threads - 1) / threads;  // granules of this thread (0 or below: none)
    if (n > 0) {
      auto load = [&](int i) { return tile[tid + i * threads]; };
      float x[N];
      unpack(load(0), x);
      mine.m = max_of(x);
      const Ref ref(mine.m, c);
      FixedSum<E> sum;
      sum.start(ref, c);
#pragma unroll 4
      for (int i = 0; i < n; ++i) sum.add(load(i));
      mine.s = sum.total();
      if (ref.far || !mine.served()) mine = sum_largest<E>(n, load, c);
    }
    mine.merge_warp(c);
    const int warps = threads / 32;
    const float4 share = make_float4(mine.m, mine.s, twice ? 1.0f : 0.0f, 0.0f);
    if (parts > 1) {
      cluster_wait();  // every CTA runs
      if (lane < parts) st_cluster(shares + rank * warps + warp, lane, share);
      cluster_arrive();
    } else if (lane == 0) {
      shares[warp] = share;
    }
    // meanwhile the sum at the ids, by every warp on its own
    auto at_ids = [&](bool once) {
      Sum top;
      for (int j = lane; j < k; j += 32)
        if (sid[j] >= 0) top.m = fmaxf(top.m, sx[j]);
      top.m = warp_max(top.m);
      const Ref ref(top.m, c);
      for (int j = lane; j < k; j += 32)
        if (sid[j] >= 0 && (!once || first(j))) top.s += ref(sx[j], c);
      top.s = warp_sum(top.s);
      return top;
    };
    Sum top = at_ids(false);
    if (parts > 1) cluster_wait();
    else __syncthreads();
    Sum outside;
    for (int i = lane; i < parts * warps; i += 32) {
      const float4 of = shares[i];
      outside.merge(of.x, of.y, c);
      twice |= of.z != 0.0f;
    }
    outside.merge_warp(c);
    twice = __any_sync(kAll, twice);
    m_out = outside.m, s_out = outside.s;
    if (twice) top = at_ids(true);
    Sum all{m_out, s_out};
    all.merge(top.m, top.s, c);
    m = all.m, s = all.s;
  } else {
    known = __ldg(a.stats_in + 2 * t);
    known_out = __ldg(a.stats_in + 2 * t + 1);
    m = known * a.temperature;
    m_out = known_out * a.temperature;
    s = s_out = 1.0f;
  }
  const bool empty = m == -INFINITY;  // a row of -inf alone has no probabilities: q = 0
  if (empty) m = 0.0f, s = 1.0f;
  const bool none = m_out == -INFINITY;
  if (none) m_out = 0.0f, s_out = 1.0f;
  // of the whole row and of its logits outside the ids; known log-sum-exps are references themselves
  Ref ref(m, c), ref_out(m_out, c);
  if constexpr (!kSums) {
    ref.r = empty ? 0.0f : known * kLog2e;
    ref_out.r = none ? 0.0f : known_out * kLog2e;
  }

  float factor;
  if constexpr (kPolicy) {
    float lp;
    if (ref.far) {
      lp = (sx[0] - m) - logf(s);
    } else {  // s = 2^e f: r + e is exact, and what is left is rounded as the small number that it is
      int e;
      const float f = frexpf(s, &e);
      lp = (fmaf(sx[0], c, -(ref.r + static_cast<float>(e))) - log2f(f)) * kLn2;
    }
    float w = 1.0f;
    if (a.rollout_logp) {
      w = expf(lp - __ldg(a.rollout_logp + t));
      if (a.cap > 0.0f) w = fminf(w, a.cap);
    }
    if (rank == 0 && tid == 0) {
      a.logp[t] = lp;
      if (a.w) a.w[t] = w;
      if (!(s < INFINITY)) flag(a.status, QRR_DEV_NONFINITE);
    }
    factor = w * __ldg(a.advantages + t);
  } else {
    if (rank == 0 && tid == 0 && (!(fabsf(m) < INFINITY) || !(s < INFINITY) || !(mass < INFINITY))) flag(a.status, QRR_DEV_NONFINITE);
    factor = kWrites ? __ldg(a.grad + t) * inv_t : 0.0f;
  }

  if constexpr (kWrites) {
    const float inv_s = 1.0f / s;
    // outside the ids: e^{x / t} over that at `at` times `scale`
    const Ref at = tail ? ref_out : ref;
    float scale = factor * inv_s;
    if (tail) {
      const float up = !kSums ? (known_out - known) * kLog2e : ref.far || ref_out.far ? (m_out - m) * c : ref_out.r - ref.r;
      const float q_rest = s_out * ex2_approx(up) * inv_s;
      scale = none ? 0.0f : factor * (q_rest - rest) / s_out;
    }
    if (e0 < e1) {
      const int shift = -base;  // of an element in `held`
      const bool same = lead_of(out) == lead;
      const uint64_t c2 = f32x2(c, c), nr2 = f32x2(-at.r, -at.r), scale2 = f32x2(scale, scale);
      store_range(
          out, e0, e1,
          [&](int e) {
            float x[N];
            if (same) {
              unpack(*reinterpret_cast<const uint4*>(held + e + shift), x);
            } else {
#pragma unroll
              for (int u = 0; u < N; ++u) x[u] = to_f32(held[e + shift + u]);
            }
            if (!at.far) {
#pragma unroll
              for (int u = 0; u < N; u += 2) {
                float y, z;
                f32x2(fma2(f32x2(x[u], x[u + 1]), c2, nr2), y, z);
                f32x2(mul2(f32x2(ex2_approx(y), ex2_approx(z)), scale2), x[u], x[u + 1]);
              }
            } else {
#pragma unroll
              for (int u = 0; u < N; ++u) x[u] = at(x[u], c) * scale;
            }
            return pack(x);
          },
          [&](int e) { return from_f32(at(to_f32(held[e + shift]), c) * scale, E{}); });
    }
    __syncthreads();
    for (int j = tid; j < k; j += threads) {
      const int id = sid[j];
      if (id < e0 || id >= e1) continue;
      float p = sp[j];
      if (twice) {
        if (!first(j)) continue;
        p = 0.0f;
        for (int i = j; i < k; ++i) p += sid[i] == id ? sp[i] : 0.0f;
      }
      out[id] = from_f32(factor * (ref(sx[j], c) * inv_s - p), E{});
    }
  }
  // The loss, by the last warp: sum_j p_j ((y_j - (x_j - m)) / t - (lse_teacher - (lse - m / t))), its few terms in 64 bits.
  if (kSums && !kPolicy && rank == 0 && warp == threads / 32 - 1) {
    double cross = 0.0, sum_p = 0.0;
    for (int j = lane; j < k; j += 32)
      if (sid[j] >= 0 && sp[j] > 0.0f) {
        const double p = sp[j], y = sy[j], x = sx[j];
        cross += p * (y - (x - static_cast<double>(m)));
        sum_p += p;
      }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      cross += __shfl_xor_sync(kAll, cross, o);
      sum_p += __shfl_xor_sync(kAll, sum_p, o);
    }
    if (lane == 0) {
      const double inv = 1.0 / static_cast<double>(a.temperature);
      // of a sum's log-sum-exp, what it is above m / t
      auto above = [&](const Ref& r, float sum) {
        const double ln = log(static_cast<double>(sum));
        if (r.far) return ln;
        const double back = inv / static_cast<double>(c);  // from powers of 2 at this c
        return (static_cast<double>(r.r) - static_cast<double>(r.m) * static_cast<double>(c) + ln * 1.4426950408889634) * back;
      };
      const double ln_s = above(ref, s);
      const double lse_y = tail ? static_cast<double>(lse_teacher) : static_cast<double>(y_max) * inv + log(static_cast<double>(y_sum));
      double loss = cross * inv - sum_p * (lse_y - ln_s), lse = static_cast<double>(m) * inv + ln_s, lse_out = lse;
      if (tail) {
        const double ln_out = none ? -INFINITY : above(ref_out, s_out);
        lse_out = static_cast<double>(m_out) * inv + ln_out;
        if (rest > (none ? kDust : 0.0f))
          loss += static_cast<double>(rest) * (log(static_cast<double>(rest)) -
                                               ((static_cast<double>(m_out) - static_cast<double>(m)) * inv + ln_out - ln_s));
      }
      a.loss[t] = static_cast<float>(loss);
      if constexpr (M == LossMode::kLoss) {
        a.stats[2 * t] = empty ? -INFINITY : static_cast<float>(lse);
        a.stats[2 * t + 1] = empty ? -INFINITY : static_cast<float>(lse_out);
      }
    }
  }
}

// Bytes of a row that a CTA holds, at most, where fewer parts would do.
constexpr int kPartBytes = 64 << 10;

template <class E, LossMode M>
cudaError_t launch(const LogitsLossArgs& a, cudaStream_t stream) {
  int dev = 0, sms = kSMs;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int granules = granules_of<E>(kPer<E> - 1, a.V);
  int parts = 1;
  while (parts < 8 && (granules * 16 > parts * kPartBytes || (a.T * parts < sms && granules > parts * 256))) parts *= 2;
  const int per = (granules + parts - 1) / parts;
  const int threads = per >= 1024 ? 256 : per >= 256 ? 128 : 64;
  const size_t smem = static_cast<size_t>(per) * 16 + static_cast<size_t>(M == LossMode::kPolicy ? 1 : a.k) * 16;
  static OncePerDevice limit;
  e = limit(dev, [] {
    return cudaFuncSetAttribute(logits_loss_kernel<E, M>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kMaxLossRowBytes / 8 + 32 + 16 * kMaxTop));
  });
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(a.T * parts);
  return launch_clusters(logits_loss_kernel<E, M>, grid, M == LossMode::kBackward ? 1 : parts, threads, smem, stream, a, parts, per);
}

template <class E>
cudaError_t launch(const LogitsLossArgs& a, LossMode mode, cudaStream_t stream) {
  switch (mode) {
    case LossMode::kLoss: return launch<E, LossMode::kLoss>(a, stream);
    case LossMode::kGrad: return launch<E, LossMode::kGrad>(a, stream);
    case LossMode::kBackward: return launch<E, LossMode::kBackward>(a, stream);
    default: return launch<E, LossMode::kPolicy>(a, stream);
  }
}

}  // namespace

cudaError_t launch_logits_loss(const LogitsLossArgs& a, LossMode mode, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  return a.fp32 ? launch<float>(a, mode, stream) : launch<Bf16>(a, mode, stream);
}

}  // namespace qrr
