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
// A rest of the teacher's that is no more than the rounding of its log-sum-exp and of the sum of p_j: beside a student
// without any, it is none.
constexpr float kDust = 1.0f / 65536;

// What a CTA tells the others of its part of the row.
struct Part {
  float m_out, s_out;  // logits outside the ids
  float m_top, s_top;  // at the ids
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
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
  float* const sx = reinterpret_cast<float*>(sid + k);  // its logit, where it lies in this part or this is the first
  float* const sp = sx + k;                             // the teacher's probability
  int* const sown = reinterpret_cast<int*>(sp + k);     // of the slots with one id, the one that speaks for them
  __shared__ float2 sums[kMaxThreads / 32];
  __shared__ Part part, whole;

  const int lead = lead_of(row), granules = granules_of<E>(lead, V);
  const int g0 = min(rank * per, granules), g1 = min(g0 + per, granules), base = g0 * N - lead;
  const int e0 = max(base, 0), e1 = min(g1 * N - lead, V);  // this part's elements

  bool any = false;
  for (int j = tid; j < k; j += threads) {
    int id = __ldg(kPolicy ? a.tokens + t : a.ids + t * k + j);
    if (id >= V) {
      flag(a.status, QRR_DEV_BAD_INDEX);
      id = -1;
    }
    sid[j] = id;
    any |= id >= 0;
    // the first part takes the loss, so it wants the logits of all ids (before another part writes over its own)
    if (kSums && (rank == 0 || kPolicy) && id >= 0) sx[j] = to_f32(row[id]);
  }
  if (!__syncthreads_or(any)) {  // nothing to learn: the whole cluster ends here
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
    return;
  }

  for (int g = g0 + tid; g < g1; g += threads) {
    const int e = g * N - lead;
    if (e >= 0 && e + N <= V) cp_async16(tile + (g - g0), row + e);
    else tile[g - g0] = load_cut(row, e, V);
  }

  // The teacher, by every warp on its own: mass = sum_j p_j, and the log-sum-exp that its logits are measured from as
  // y_max / t + ln y_sum (without a tail) or lse_teacher.
  const float inv_t = kPolicy ? 1.0f : 1.0f / a.temperature, c = kLog2e * inv_t;
  const bool tail = !kPolicy && a.top_lse;
  float mass = 1.0f, y_max = 0.0f, y_sum = 1.0f, lse_teacher = 0.0f;
  if constexpr (kPolicy) {
    if (tid == 0) sp[0] = 1.0f;
  } else {
    const float* const top = a.top + t * k;
    if (tail) {
      lse_teacher = __ldg(a.top_lse + t);
    } else {
      y_max = -INFINITY;
      for (int j = lane; j < k; j += 32)
        if (sid[j] >= 0) y_max = fmaxf(y_max, __ldg(top + j));
      y_max = warp_max(y_max);
      if (y_max == -INFINITY) y_max = 0.0f;
      y_sum = 0.0f;
      for (int j = lane; j < k; j += 32)
        if (sid[j] >= 0) y_sum += expf((__ldg(top + j) - y_max) * inv_t);
      y_sum = warp_sum(y_sum);
    }
    mass = 0.0f;
    const float norm = 1.0f / y_sum;
    for (int j = lane; j < k; j += 32) {
      float p = 0.0f;
      if (sid[j] >= 0) p = tail ? expf(fmaf(__ldg(top + j), inv_t, -lse_teacher)) : expf((__ldg(top + j) - y_max) * inv_t) * norm;
      mass += p;
      if (warp == 0) sp[j] = p;
    }
    mass = warp_sum(mass);
  }
  const float rest = tail ? fmaxf(1.0f - mass, 0.0f) : 0.0f;  // p_r

  cp_async_wait_all();
  __syncthreads();
  // Warp 0 takes the ids' logits out of the part. Slots that name one id find out by writing their numbers to its place:
  // the one that stays there speaks for all.
  bool twice = false;
  if (warp == 0) {
    auto each = [&](auto f) {
      for (int j = lane; j < k; j += 32) {
        const int id = sid[j];
        if (id >= e0 && id < e1) f(j, id - base);
      }
      __syncwarp();
    };
    auto number = [](int j) {
      if constexpr (sizeof(E) == 2) return static_cast<E>(j);
      else return __int_as_float(j);
    };
    each([&](int j, int at) { sx[j] = to_f32(held[at]); });
    each([&](int j, int at) { held[at] = number(j); });
    each([&](int j, int at) {
      int o;
      if constexpr (sizeof(E) == 2) o = held[at];
      else o = __float_as_int(held[at]);
      sown[j] = o;
      twice |= o != j;
    });
    each([&](int, int at) { held[at] = minus_inf<E>(); });
    twice = __any_sync(kAll, twice);
    if constexpr (kSums) {
      Sum top;
      for (int j = lane; j < k; j += 32) {
        const int id = sid[j];
        if (id < e0 || id >= e1 || sown[j] != j) continue;
        const float x[1] = {sx[j]};
        top.add(x, x[0], c);
      }
      top.merge_warp(c);
      if (lane == 0) {
        part.m_top = top.m;
        part.s_top = top.s;
      }
    }
  }
  __syncthreads();

  // Of the whole row: references and sums outside the ids and at them.
  float m_out, s_out, m, s;
  if constexpr (kSums) {
    Sum mine;
    for (int g = tid; g < g1 - g0; g += threads) {
      float x[N];
      unpack(tile[g], x);
      mine.add(x, max_of(x), c);
    }
    mine.merge_warp(c);
    if (lane == 0) sums[warp] = make_float2(mine.m, mine.s);
    __syncthreads();
    if (warp == 0) {
      mine = Sum{};
      if (lane < threads / 32) mine = Sum{sums[lane].x, sums[lane].y};
      mine.merge_warp(c);
      if (lane == 0) {
        part.m_out = mine.m;
        part.s_out = mine.s;
      }
      __syncwarp();
    }
    if (parts > 1) {
      cluster_arrive();
      cluster_wait();
    }
    if (warp == 0) {
      Sum outside, top;
      if (lane < parts) {
        outside.m = ld_cluster(&part.m_out, lane);
        outside.s = ld_cluster(&part.s_out, lane);
        top.m = ld_cluster(&part.m_top, lane);
        top.s = ld_cluster(&part.s_top, lane);
      }
      outside.merge_warp(c);
      top.merge_warp(c);
      if (lane == 0) whole = Part{outside.m, outside.s, top.m, top.s};
    }
    if (parts > 1) cluster_arrive();  // nobody ends while another reads its part
    __syncthreads();
    m_out = whole.m_out, s_out = whole.s_out;
    Sum all;
    all.m = m_out, all.s = s_out;
    all.merge(whole.m_top, whole.s_top, c);
    m = all.m, s = all.s;
  } else {
    m = __ldg(a.stats_in + 2 * t) * a.temperature;
    m_out = __ldg(a.stats_in + 2 * t + 1) * a.temperature;
    s = s_out = 1.0f;
  }
  const bool empty = m == -INFINITY;  // a row of -inf alone has no probabilities: q = 0
  if (empty) m = 0.0f, s = 1.0f;
  const bool none = m_out == -INFINITY;
  if (none) m_out = 0.0f, s_out = 1.0f;

  float factor;
  if constexpr (kPolicy) {
    const float lp = (sx[0] - m) - logf(s);
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
    // outside the ids: e^{(x - ref) / t} times `scale`
    const float ref = tail ? m_out : m;
    float scale = factor * inv_s;
    if (tail) {
      const float q_rest = s_out * ex2_approx((m_out - m) * c) * inv_s;
      scale = none ? 0.0f : factor * (q_rest - rest) / s_out;
    }
    auto value = [&](float x) { return ex2_approx((x - ref) * c) * scale; };
    if (e0 < e1) {
      const int shift = -base;  // of an element in `held`
      const bool same = lead_of(out) == lead;
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
#pragma unroll
            for (int u = 0; u < N; ++u) x[u] = value(x[u]);
            return pack(x);
          },
          [&](int e) { return from_f32(value(to_f32(held[e + shift])), E{}); });
    }
    __syncthreads();
    if (warp == 0) {
      for (int j = lane; j < k; j += 32) {
        const int id = sid[j];
        if (id < e0 || id >= e1 || sown[j] != j) continue;
        float p = sp[j];
        if (twice) {
          p = 0.0f;
          for (int i = 0; i < k; ++i) p += sid[i] == id ? sp[i] : 0.0f;
        }
        out[id] = from_f32(factor * (ex2_approx((sx[j] - m) * c) * inv_s - p), E{});
      }
    }
  }
  // The loss, by the last warp: sum_j p_j ((y_j - (x_j - m)) / t - (lse_teacher - ln s)), its few terms in 64 bits.
  if (kSums && !kPolicy && rank == 0 && warp == threads / 32 - 1) {
    double cross = 0.0, sum_p = 0.0;
    for (int j = lane; j < k; j += 32)
      if (sid[j] >= 0 && sp[j] > 0.0f) {
        const double p = sp[j], y = __ldg(a.top + t * k + j), x = sx[j];
        cross += p * (y - (x - static_cast<double>(m)));
        sum_p += p;
      }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      cross += __shfl_xor_sync(kAll, cross, o);
      sum_p += __shfl_xor_sync(kAll, sum_p, o);
    }
    if (lane == 0) {
      const double inv = 1.0 / static_cast<double>(a.temperature), ln_s = log(static_cast<double>(s));
      const double lse_y = tail ? static_cast<double>(lse_teacher) : static_cast<double>(y_max) * inv + log(static_cast<double>(y_sum));
      double loss = cross * inv - sum_p * (lse_y - ln_s), lse = static_cast<double>(m) * inv + ln_s, lse_out = lse;
      if (tail) {
        const double ln_out = none ? -INFINITY : log(static_cast<double>(s_out));
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
  if constexpr (kSums)
    if (parts > 1) cluster_wait();
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
