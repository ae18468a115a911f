// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// Sequence b brings n drafted tokens d_0 .. d_{n-1} and the target's rows of logits at their places and behind the last one.
// With p_i = softmax(target row i / t) and q_i = softmax(draft row i / t), drafts are taken in order while
//   u_i q_i(d_i) < p_i(d_i);
// at the first refusal the next token is argmax_v max(p_i(v) - q_i(v), 0) / e_v, behind the last draft argmax_v p_n(v) / e_v.
// For u uniform in [0, 1) and e exponential the tokens are distributed as if each had been drawn from p. Drafts without
// probabilities of their own (looked up in the prompt, say) are q_i = [v = d_i]. At t = 0 a draft is taken if it is the
// target's likeliest token (the lowest of equals), which is also the next token.
//
// Bound by memory: rows up to the first refusal are read once (the refused pair, and the row behind the last draft, a second
// time, from L2 mostly), the noise once. One cluster of CTAs a sequence, each with a contiguous part of the vocabulary; they
// join maxima and sums over distributed shared memory, and each takes the decisions for itself. Rows go in groups: one
// barrier of the cluster a group; rows behind a refusal in the same group are read in vain.
//
// Sums are fp32 with the hardware's base-2 exponential; the decisions and the probabilities that tokens are drawn from take
// expf of the logits' differences.
#include "logits.cuh"
#include "once_per_device.cuh"

namespace qrr {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kGroup = 16;  // places of a group, at most
constexpr int kInFlight = 4;
constexpr uint32_t kAll = 0xFFFFFFFFu;
enum class Form { kModel, kLookup, kGreedy };

// A row's sum, and the first place of its maximum (greedy).
struct RowSum {
  float m, s;
  int arg;
};

__device__ __forceinline__ uint64_t warp_max64(uint64_t v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const uint64_t w = __shfl_xor_sync(kAll, v, o);
    v = w > v ? w : v;
  }
  return v;
}

// Candidates by score, the lowest index of equals: a positive float orders as its bits do.
__device__ __forceinline__ uint64_t candidate(float score, int v) {
  return static_cast<uint64_t>(__float_as_uint(score)) << 32 | (kAll - static_cast<uint32_t>(v));
}

// Elements e .. e + kPer of a row from its granules if they are aligned, one by one if not.
template <class E>
__device__ __forceinline__ void load_block(const E* row, int e, float (&x)[kPer<E>]) {
  if ((reinterpret_cast<uintptr_t>(row + e) & 15u) == 0) {
    unpack(__ldg(reinterpret_cast<const uint4*>(row + e)), x);
  } else {
#pragma unroll
    for (int u = 0; u < kPer<E>; ++u) x[u] = to_f32(__ldg(row + e + u));
  }
}
template <int N>
__device__ __forceinline__ void load_noise(const float* row, int e, float (&x)[N]) {
  if ((reinterpret_cast<uintptr_t>(row + e) & 15u) == 0) {
#pragma unroll
    for (int u = 0; u < N; u += 4) {
      const float4 f = __ldcs(reinterpret_cast<const float4*>(row + e + u));
      x[u] = f.x, x[u + 1] = f.y, x[u + 2] = f.z, x[u + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int u = 0; u < N; ++u) x[u] = __ldcs(row + e + u);
  }
}

template <class E, Form F>
__global__ void __launch_bounds__(kThreads, 3) verify_drafts_kernel(const VerifyArgs a, const int parts, const int group) {
  constexpr int N = kPer<E>;
  constexpr bool kModel = F == Form::kModel, kGreedy = F == Form::kGreedy;
  constexpr int kRows = kModel ? 2 : 1;  // rows a place
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / parts, rank = blockIdx.x % parts, V = a.V;

  __shared__ RowSum warps[kGroup * kRows][kWarps];
  __shared__ RowSum mine[2][kGroup * kRows];  // by the groups' parity: others may still read the last one's
  __shared__ RowSum whole[kGroup * kRows];
  __shared__ uint64_t best_warps[kWarps][2], best[2];
  __shared__ int s_end, s_refused;

  int64_t first = static_cast<int64_t>(b) * (a.T / a.B), behind = first + a.T / a.B;
  if (a.cu) {
    first = __ldg(a.cu + b);
    behind = __ldg(a.cu + b + 1);
    if (first < 0 || behind < first || behind > a.T) {
      if (rank == 0 && tid == 0) flag(a.status, QRR_DEV_BAD_INDEX);
      return;
    }
  }
  // A negative draft is none: those before it are all there are.
  const int given = static_cast<int>(behind - first);
  if (tid == 0) s_end = given;
  __syncthreads();
  for (int i = tid; i < given; i += kThreads) {
    const int d = __ldg(a.drafts + first + i);
    if (d >= 0 && d < V) continue;
    if (d >= V) flag(a.status, QRR_DEV_BAD_INDEX);
    atomicMin(&s_end, i);
  }
  __syncthreads();
  const int n = s_end;
  const E* const target = static_cast<const E*>(a.target) + (first + b) * a.ld_target;
  const E* const draft = kModel ? static_cast<const E*>(a.draft) + first * a.ld_draft : nullptr;
  int32_t* const tokens = a.tokens + first + b;
  float* const logp = a.logp + first + b;
  const float inv_t = kGreedy ? 1.0f : 1.0f / a.temperature, c = kLog2e * inv_t;

  // this CTA's granules of a row: a range that does not depend on where the row starts
  const int per = (granules_of<E>(N - 1, V) + parts - 1) / parts;
  auto row_of = [&](int place, int which) { return which ? draft + place * a.ld_draft : target + place * a.ld_target; };

  int taken = 0, done = 0, parity = 0;
  bool refused = false;
  RowSum p_row{}, q_row{};  // of the row that the next token is drawn from
  while (true) {
    const int places = min(group, n + 1 - done);  // at least one
    const int rows = kModel ? places + min(places, n - done) : places;
    // rows of the group: targets first, then drafts
    auto group_row = [&](int r) { return r < places ? row_of(done + r, 0) : row_of(done + r - places, 1); };
    const int chunks = (per + kThreads * kInFlight - 1) / (kThreads * kInFlight);
    auto load = [&](const E* row, int chunk, uint4 (&g)[kInFlight]) {
      const int lead = lead_of(row), end = min((rank + 1) * per, granules_of<E>(lead, V));
      int i = rank * per + chunk * kThreads * kInFlight + tid;
#pragma unroll
      for (int u = 0; u < kInFlight; ++u, i += kThreads) {
        const int e = i * N - lead;
        const uint32_t none = N == 8 ? 0xFF80FF80u : 0xFF800000u;
        g[u] = make_uint4(none, none, none, none);
        if (i < end) {
          if (e >= 0 && e + N <= V) g[u] = __ldg(reinterpret_cast<const uint4*>(row + e));
          else g[u] = load_cut(row, e, V);
        }
      }
    };
    uint4 next[kInFlight];
    const E* row = group_row(0);
    load(row, 0, next);
    Sum sum;
    int where = -1;  // the granule of the maximum
    for (int r = 0, chunk = 0; r < rows;) {
      uint4 now[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) now[u] = next[u];
      const int here = chunk;
      const bool last = ++chunk == chunks;
      const E* const old = row;
      if (last) {
        chunk = 0;
        if (r + 1 < rows) row = group_row(r + 1);
      }
      if (!last || r + 1 < rows) load(row, chunk, next);
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        float x[N];
        unpack(now[u], x);
        const float top = max_of(x);
        if constexpr (kGreedy)
          if (top > sum.m) where = rank * per + (here * kInFlight + u) * kThreads + tid;
        sum.add_largest(x, top, c);
      }
      if (!last) continue;
      const float m = sum.m;
      sum.merge_warp(c);
      int arg = V;
      if constexpr (kGreedy) {
        if (where >= 0 && m == sum.m) {
          const int e = where * N - lead_of(old);
          for (int u = N - 1; u >= 0; --u)
            if (e + u >= 0 && e + u < V && to_f32(old[e + u]) == m) arg = e + u;
        }
        arg = __reduce_min_sync(kAll, arg);
        where = -1;
      }
      if (lane == 0) warps[r][warp] = RowSum{sum.m, sum.s, arg};
      sum = Sum{};
      ++r;
    }
    __syncthreads();
    auto join = [&](RowSum& into, const RowSum& x) {
      if constexpr (kGreedy) {
        if (x.m > into.m) into.arg = x.arg;
        else if (x.m == into.m) into.arg = min(into.arg, x.arg);
      }
      Sum both{into.m, into.s};
      both.merge(x.m, x.s, c);
      into.m = both.m, into.s = both.s;
    };
    if (tid < rows) {
      RowSum x = warps[tid][0];
      for (int w = 1; w < kWarps; ++w) join(x, warps[tid][w]);
      mine[parity][tid] = x;
    }
    if (parts > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    if (tid < rows) {
      RowSum x{-INFINITY, 0.0f, V};
      for (int o = 0; o < parts; ++o) {
        RowSum y;
        y.m = ld_cluster(&mine[parity][tid].m, o);
        y.s = ld_cluster(&mine[parity][tid].s, o);
        y.arg = __float_as_int(ld_cluster(reinterpret_cast<const float*>(&mine[parity][tid].arg), o));
        join(x, y);
      }
      if (!(fabsf(x.m) < INFINITY) || !(x.s < INFINITY)) {
        if (rank == 0) flag(a.status, QRR_DEV_NONFINITE);
        if (x.m == -INFINITY) x.m = 0.0f, x.s = 1.0f;  // a row of -inf alone: no probabilities
      }
      const Ref ref(x.m, c);  // from here on a sum of e^{(x - m) / t}
      if (!ref.far) x.s *= ex2_approx(fmaf(-x.m, c, ref.r));
      whole[tid] = x;
    }
    if (tid == 0) s_refused = kGroup;
    __syncthreads();
    // the drafts of the group, a thread each
    if (tid < places && done + tid < n) {
      const int i = done + tid, d = __ldg(a.drafts + first + i);
      const RowSum p = whole[tid];
      const float dp = to_f32(target[i * a.ld_target + d]) - p.m;
      bool ok;
      if constexpr (kGreedy) {
        ok = d == p.arg;
      } else if constexpr (kModel) {
        // u q < p as u (s_p / s_q) e^{((x_q - m_q) - (x_p - m_p)) / t} < 1
        const RowSum q = whole[places + tid];
        const float dq = to_f32(draft[i * a.ld_draft + d]) - q.m;
        ok = __ldg(a.uniforms + first + i) * (p.s / q.s) * expf((dq - dp) * inv_t) < 1.0f;
      } else {
        ok = __ldg(a.uniforms + first + i) * p.s < expf(dp * inv_t);
      }
      if (!ok) atomicMin(&s_refused, tid);
    }
    __syncthreads();
    const int accepted = min(s_refused, min(places, n - done));
    if (rank == 0 && tid < accepted) {
      const int d = __ldg(a.drafts + first + done + tid);
      tokens[done + tid] = d;
      logp[done + tid] = (to_f32(target[(done + tid) * a.ld_target + d]) - whole[tid].m) * inv_t - logf(whole[tid].s);
    }
    taken = done + accepted;
    if (accepted < places) {
      refused = taken < n;
      p_row = whole[accepted];
      if constexpr (kModel)
        if (refused) q_row = whole[places + accepted];
      break;
    }
    done += places;
    parity ^= 1;
    __syncthreads();  // `whole` and s_refused are written again
  }

  int token = -1;
  if constexpr (kGreedy) {
    token = p_row.arg < V ? p_row.arg : -1;
  } else {
    const E* const row = row_of(taken, 0);
    const E* const other = kModel && refused ? row_of(taken, 1) : nullptr;
    const float* const noise = a.noise + b * a.ld_noise;
    const int drafted = refused ? __ldg(a.drafts + first + taken) : -1;
    const int lead = lead_of(row), end = min((rank + 1) * per, granules_of<E>(lead, V));
    const float m = p_row.m, mq = q_row.m;
    const float inv_p = 1.0f / p_row.s, inv_q = kModel && refused ? 1.0f / q_row.s : 0.0f;
    float left = 0.0f, all = 0.0f;  // the best scores of what is left, and of p
    int left_at = 0, all_at = 0;
    auto consider = [&](float x, float y, float e, int v) {
      const float p = __fmul_rn(expf((x - m) * inv_t), inv_p);
      float r = p;
      if (refused) {
        // both products rounded: contracted to an FMA, the difference of equal rows would be a rounding error and not 0
        if constexpr (kModel) r = p - __fmul_rn(expf((y - mq) * inv_t), inv_q);
        else r = v == drafted ? 0.0f : p;
        if (p / e > all) all = p / e, all_at = v;
      }
      if (r / e > left) left = r / e, left_at = v;
    };
    for (int i = rank * per + tid; i < end; i += kThreads) {
      const int e = i * N - lead;
      if (e >= 0 && e + N <= V) {
        float x[N], y[N], z[N];
        load_block(row, e, x);
        load_noise(noise, e, z);
        if (kModel && refused) load_block(other, e, y);
#pragma unroll
        for (int u = 0; u < N; ++u) consider(x[u], y[u], z[u], e + u);
      } else {
        for (int v = max(e, 0); v < min(e + N, V); ++v)
          consider(to_f32(row[v]), kModel && refused ? to_f32(other[v]) : 0.0f, __ldg(noise + v), v);
      }
    }
    uint64_t c_left = left > 0.0f ? candidate(left, left_at) : 0, c_all = all > 0.0f ? candidate(all, all_at) : 0;
    c_left = warp_max64(c_left);
    c_all = warp_max64(c_all);
    if (lane == 0) best_warps[warp][0] = c_left, best_warps[warp][1] = c_all;
    __syncthreads();
    if (tid < 2) {
      uint64_t x = 0;
      for (int w = 0; w < kWarps; ++w) x = best_warps[w][tid] > x ? best_warps[w][tid] : x;
      best[tid] = x;
    }
    if (parts > 1) {
      cluster_arrive();
      cluster_wait();
    }
    if (rank == 0 && warp == 0) {
      __syncwarp();
      uint64_t x = 0, y = 0;
      if (lane < parts) x = ld_cluster(&best[0], lane), y = ld_cluster(&best[1], lane);
      x = warp_max64(x);
      y = warp_max64(y);
      if (x == 0) x = y;  // nothing is left of p: from p itself
      if (x) token = static_cast<int>(kAll - static_cast<uint32_t>(x));
    }
  }
  if (rank == 0) {
    if (tid == 0) {
      tokens[taken] = token;
      logp[taken] = token < 0 ? 0.0f : (to_f32(target[taken * a.ld_target + token]) - p_row.m) * inv_t - logf(p_row.s);
      a.accepted[b] = taken;
    }
    for (int i = taken + 1 + tid; i <= given; i += kThreads) {
      tokens[i] = -1;
      logp[i] = 0.0f;
    }
  }
  if (parts > 1) {  // nobody ends while another reads from it
    cluster_arrive();
    cluster_wait();
  }
}

template <class E, Form F>
cudaError_t launch(const VerifyArgs& a, cudaStream_t stream) {
  int dev = 0, sms = kSMs;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  static OncePerDevice wide;
  e = wide(dev, [] { return cudaFuncSetAttribute(verify_drafts_kernel<E, F>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); });
  if (e != cudaSuccess) return e;
  const int granules = granules_of<E>(kPer<E> - 1, a.V);
  int parts = 1;
  while (parts < 16 && static_cast<int64_t>(a.B) * parts < 2 * sms && granules > parts * kThreads) parts *= 2;
  const int group = static_cast<int64_t>(a.B) * parts < sms ? kGroup : 1;
  return launch_clusters(verify_drafts_kernel<E, F>, static_cast<unsigned>(a.B) * parts, parts, kThreads, 0, stream, a, parts, group);
}

template <class E>
cudaError_t launch(const VerifyArgs& a, cudaStream_t stream) {
  if (a.temperature == 0.0f) return launch<E, Form::kGreedy>(a, stream);
  return a.draft ? launch<E, Form::kModel>(a, stream) : launch<E, Form::kLookup>(a, stream);
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs& a, cudaStream_t stream) {
  if (a.B == 0) return cudaSuccess;
  return a.fp32 ? launch<float>(a, stream) : launch<Bf16>(a, stream);
}

}  // namespace qrr
