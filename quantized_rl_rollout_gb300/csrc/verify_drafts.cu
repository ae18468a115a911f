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
// time, from L2 mostly), the noise once. Which rows those are is known when the rows before are summed, and waiting for that
// would cost more than it saves: one launch sums the rows, the first places of all sequences first, and its CTAs pass over what
// lies behind a refusal that is known by then. So what is read in vain is about as much as is under way at a time. The last
// of the parts of a place to be summed decides it. A launch before it checks the drafts, one behind it draws the tokens.
//
// 64 sequences of 8 drafts over 128256 bf16 logits take 53 us, 38% of a copy's rate by the bytes that have to be read. Some 36
// of them sum rows: 171 MB at 4.6 TB/s where 104 MB have to be read, but a place at a time for the sequences that go on would
// take 9 tasks of 4 us one after another, as long. The rest draws: 33 MB of noise, and as much of rows again.
// Launches of their own for places 0 and 1, for 2 .. and for all took 65 to 75 us: a launch that reads a few rows takes as
// long as one that reads 64 MB. Taking tasks that are known to be needed before others changed nothing. One sequence
// takes 12 us, three launches that wait for one another.
//
// Sums are fp32 with the hardware's base-2 exponential. Drafts are decided, and tokens drawn, from probabilities by the exact
// one; where a token is drawn, bounds by the hardware's say which few can be the best.
#include <limits.h>

#include <algorithm>
#include <type_traits>

#include "logits.cuh"
#include "once_per_device.cuh"
#include "verify_order.cuh"

namespace qrr {

namespace {

constexpr int kSumWorkers = 256, kSumThreads = kSumWorkers + 32, kSumCtas = 4, kDrawThreads = 512;
constexpr int kSumParts = 32, kMaxParts = 16;  // at most, of a row where it is summed and where a token is drawn
enum class Form { kModel, kLookup, kGreedy };

// A part of a row: a reference and the sum there; its largest logit and where that is first (greedy).
struct alignas(16) RowSum {
  float m, s, largest;
  int arg;
};

// What is known of a sequence: drafts before the first that is none (negative, or behind the vocabulary); and the places that
// are needed, which a refusal makes fewer.
struct alignas(8) State {
  int usable, needed;
};

// The workspace: sums of a target row of each place of every sequence, then of each draft row; states; parts that are summed
// of each place; the sequence of each place (with offsets, and of places in sequences alone).
struct Workspace {
  RowSum* sums;
  State* states;
  int* summed;
  int* owners;
  __host__ __device__ Workspace(const VerifyArgs& a, int parts) {
    sums = static_cast<RowSum*>(a.workspace);
    states = reinterpret_cast<State*>(sums + (2 * a.T + a.B) * parts);
    summed = reinterpret_cast<int*>(states + a.B);
    owners = summed + (a.T + a.B);
  }
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

// Part `rank` of `parts` of a row's granules: its whole ones, and the row's cut ones if they are here (-1: not).
template <class E>
struct Span {
  const E* row;
  int V, lead, w0, w1, head, tail;
  __device__ __forceinline__ Span(const E* row_, int V_, int rank, int parts) : row(row_), V(V_), lead(lead_of(row_)) {
    const int per = (granules_of<E>(kPer<E> - 1, V) + parts - 1) / parts;  // wherever the row starts
    const int all = granules_of<E>(lead, V), g0 = min(rank * per, all), g1 = min(g0 + per, all);
    const bool at_head = g0 == 0 && g1 > 0 && lead > 0, at_tail = g1 == all && g1 > g0 && (lead + V) % kPer<E> != 0;
    w0 = at_head ? 1 : g0;
    w1 = max(at_tail ? g1 - 1 : g1, w0);
    head = at_head ? 0 : -1;
    tail = at_tail && !(at_head && all == 1) ? all - 1 : -1;
  }
  __device__ __forceinline__ const uint4* granules() const { return reinterpret_cast<const uint4*>(row - lead); }
  __device__ __forceinline__ uint4 cut(int i) const { return load_cut(row, i * kPer<E> - lead, V); }
};

// The rows and drafts of a sequence.
template <class E>
struct Sequence {
  int64_t first;  // draft
  int given;      // drafts
  bool valid;     // its offsets are
  const E *target, *draft;
  __device__ __forceinline__ Sequence(const VerifyArgs& a, int b) : first(0), given(0), valid(true) {
    int64_t behind;
    if (a.cu) {
      first = __ldg(a.cu + b);
      behind = __ldg(a.cu + b + 1);
      valid = first >= 0 && behind >= first && behind <= a.T;
    } else {
      first = static_cast<int64_t>(b) * (a.T / a.B);
      behind = first + a.T / a.B;
    }
    given = valid ? static_cast<int>(behind - first) : 0;
    target = static_cast<const E*>(a.target) + (first + b) * a.ld_target;
    draft = static_cast<const E*>(a.draft) + first * a.ld_draft;
  }
};

// Of a row of -inf alone, which has no probabilities: 0 of each logit.
__device__ __forceinline__ RowSum sane(RowSum x) {
  if (x.m == -INFINITY) x.m = 0.0f, x.s = 1.0f;
  return x;
}

// The sum of a row from its parts, by a warp (the same in every lane).
template <Form F>
__device__ __forceinline__ RowSum merge_parts(RowSum x, Scale c, int V) {
  Sum sum{x.m, x.s};
  sum.merge_warp(c);
  if constexpr (F == Form::kGreedy) {
    const float top = warp_max(x.largest);
    x.arg = __reduce_min_sync(kAll, x.largest == top ? x.arg : V);
    x.largest = top;
  }
  x.m = sum.m, x.s = sum.s;
  return x;
}
__device__ __forceinline__ RowSum part_of_row(const RowSum* parts_of, int parts, int V) {  // a lane each
  const int lane = threadIdx.x & 31;
  RowSum x{-INFINITY, 0.0f, -INFINITY, V};
  if (lane < parts) {
    const float4 f = __ldcg(reinterpret_cast<const float4*>(parts_of + lane));
    x = RowSum{f.x, f.y, f.z, __float_as_int(f.w)};
  }
  return x;
}

// The base-2 logarithm of p / q where a reference is far: what a logit has above it is taken first, as the numbers
// themselves have no digits for the difference.
__device__ __noinline__ float far_apart(RowSum p, RowSum q, float dp, float dq, Scale c) {
  const Ref at(p.m, c), at_q(q.m, c);
  return ((dp - at.m) - (dq - at_q.m)) * c + (at.offset(c) - at_q.offset(c)) - (log2f(p.s) - log2f(q.s));
}

// Whether a draft is taken, from the sums of its place and its logits.
template <Form F>
__device__ __forceinline__ bool taken_by(RowSum p, RowSum q, int drafted, float u, float dp, float dq, Scale c) {
  if constexpr (F == Form::kGreedy) return drafted == p.arg;
  p = sane(p);
  const Ref at(p.m, c);
  // 0 q < p as p > 0, though p / q may be below fp32's range. (NaN: refused.)
  auto above = [&](float l, float p_by_q) { return u > 0.0f ? u < p_by_q : dp > -INFINITY && l == l; };
  if constexpr (F == Form::kLookup) {
    const float l = ln_share(dp, at, p.s, Log2(at, p.s), c);
    return above(l, expf(l));
  }
  // u q < p as u < 2^{c (x_p - x_q) - (r_p - r_q) - (log2 s_p - log2 s_q)}
  q = sane(q);
  const Ref at_q(q.m, c);
  float l;
  if (at.far || at_q.far) {
    l = far_apart(p, q, dp, dq, c);
  } else {
    const Log2 lp(at, p.s), lq(at_q, q.s);
    l = c.exponent(dp - dq, lp.whole - lq.whole) - (lp.part - lq.part);
  }
  return above(l, exp2f(l));
}

// Checks offsets and drafts, a warp a sequence, and sets up the workspace.
template <class E>
__global__ void __launch_bounds__(256) verify_begin_kernel(const VerifyArgs a, const int parts) {
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, b = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  if (b >= a.B) return;
  const Sequence<E> s(a, b);
  const Workspace to(a, parts);
  int usable = s.given;
  for (int i = lane; i < s.given; i += 32) {
    const int d = __ldg(a.drafts + s.first + i);
    if (d < 0 || d >= a.V) usable = min(usable, i);
    to.summed[s.first + b + i] = 0;
    if (a.cu) to.owners[s.first + b + i] = b;
  }
  usable = __reduce_min_sync(kAll, usable);
  if (lane != 0) return;
  if (a.cu && s.valid) to.owners[s.first + b + s.given] = b;
  to.states[b] = State{usable, s.valid ? usable + 1 : 0};
  if (!s.valid || (usable < s.given && __ldg(a.drafts + s.first + usable) >= a.V)) flag(a.status, QRR_DEV_BAD_INDEX);
}

// A warp's sum of a span once more, at its largest logits (called with copies, so that what the callers hold stays in registers).
template <class E>
__device__ __noinline__ Sum sum_again(const Span<E> span, int tid, Scale c) {
  Sum sum;
  auto add = [&](uint4 g) {
    float x[kPer<E>];
    unpack(g, x);
    sum.add_largest(x, max_of(x), c);
  };
  for (int i = span.w0 + tid; i < span.w1; i += kSumWorkers) add(__ldg(span.granules() + i));
  if (tid == 0 && span.head >= 0) add(span.cut(0));
  if (tid == kSumWorkers - 1 && span.tail >= 0) add(span.cut(span.tail));
  sum.merge_warp(c);
  return sum;
}

// Sums of rows. Task (i * kRows + which) * parts + rank is a part of a row, i the place in the order (PlaceOrder), which: the
// target's (0) or the draft's (1). A CTA takes the tasks blockIdx.x, blockIdx.x + gridDim.x, .. that are needed: eight warps
// sum a task's granules while one more joins the sums of the task before, decides that place if it is its last part, and
// looks for the task behind. Four CTAs an SM leave a thread 56 registers; 24 to 52 bytes are spilled.
template <class E, Form F>
__global__ void __launch_bounds__(kSumThreads, kSumCtas) verify_sums_kernel(const VerifyArgs a, const int parts) {
  constexpr int N = kPer<E>;
  constexpr bool kModel = F == Form::kModel, kGreedy = F == Form::kGreedy;
  constexpr int kRows = kModel ? 2 : 1, kWarps = kSumWorkers / 32, kInFlight = 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = a.V;
  const Scale c = a.scale;
  const Workspace at(a, parts);
  struct Task {
    const E* row;  // null: no more
    int rank;
  };
  __shared__ Task tasks[2];
  __shared__ RowSum sums[2][kWarps];
  __shared__ int most;

  griddep_launch_dependents();
  if (tid == 0) most = 0;
  __syncthreads();
  griddep_wait();  // (in every block: the next launch relies on it)
  int longest = 0;
  for (int b = tid; b < a.B; b += kSumThreads) longest = max(longest, __ldcg(&at.states[b].usable) + 1);
  atomicMax(&most, longest);
  __syncthreads();

  if (warp < kWarps) {
    __syncthreads();  // the first task
    for (int k = 0;; ++k) {
      const Task task = tasks[k & 1];
      if (!task.row) return;
      const Span<E> span(task.row, V, task.rank, parts);
      const uint4* const granules = span.granules() + span.w0;
      const int whole = span.w1 - span.w0;
      uint4 g[kInFlight];
      auto fetch = [&](int first) {
#pragma unroll
        for (int u = 0; u < kInFlight; ++u)
          if (first + u * kSumWorkers < whole) g[u] = __ldg(granules + first + u * kSumWorkers);
      };
      fetch(tid);
      float sample = -INFINITY;  // a warp's reference: the largest of its first granules
      if (tid < whole) {
        float x[N];
        unpack(g[0], x);
        sample = max_of(x);
      }
      const Ref ref(warp_max(sample), c);
      FixedSum<E> fixed;
      fixed.start(ref, c);
      float largest = -INFINITY;
      int where = -1;  // the granule of the largest
      auto use = [&](int i, uint4 v) {
        if constexpr (kGreedy) {
          float x[N];
          unpack(v, x);
          const float top = max_of(x);
          if (top > largest) largest = top, where = i;
        }
        fixed.add(v);
      };
      if (tid == 0 && span.head >= 0) use(0, span.cut(0));
      for (int first = tid;;) {
#pragma unroll
        for (int u = 0; u < kInFlight; ++u)
          if (first + u * kSumWorkers < whole) use(span.w0 + first + u * kSumWorkers, g[u]);
        first += kInFlight * kSumWorkers;
        if (first - tid >= whole) break;
        fetch(first);
      }
      if (tid == kSumWorkers - 1 && span.tail >= 0) use(span.tail, span.cut(span.tail));
      RowSum x{ref.m, warp_sum(ref.far ? INFINITY : fixed.total()), largest, V};
      // A sum near the ends of fp32's range is taken again, at the warp's largest logit. (It may have no values at all.)
      if (!(x.s > 0x1p-60f && x.s < 0x1p64f)) {
        const Sum again = sum_again(span, tid, c);
        x.m = again.m, x.s = again.s;
      }
      if constexpr (kGreedy) {
        x.largest = warp_max(largest);
        int arg = V;
        if (where >= 0 && largest == x.largest) {
          const int e = where * N - span.lead;
          for (int w = N - 1; w >= 0; --w)
            if (e + w >= 0 && e + w < V && to_f32(task.row[e + w]) == largest) arg = e + w;
        }
        x.arg = __reduce_min_sync(kAll, arg);
      }
      if (lane == 0) sums[k & 1][warp] = x;
      __syncthreads();
    }
  }

  // The last warp.
  struct Where {
    int place, b, which, rank, usable;
    int64_t first;
  };
  struct Candidate {
    Where at;
    bool needed;
  };
  const int log_parts = __ffs(parts) - 1;
  const PlaceOrder order(most, a.B, a.T + a.B);
  const int64_t total = order.total * kRows * parts;
  int64_t next = blockIdx.x;  // the first task that is not looked at
  auto ask = [&] {            // a lane each
    Candidate x;
    const int64_t task = next + static_cast<int64_t>(lane) * gridDim.x, row = task >> log_parts, i = row / kRows;
    x.at.rank = static_cast<int>(task & (parts - 1)), x.at.which = static_cast<int>(row % kRows);
    x.at.place = total <= INT_MAX ? static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(a.B)) : static_cast<int>(i / a.B);
    x.at.b = static_cast<int>(i - static_cast<int64_t>(x.at.place) * a.B);
    x.at.first = 0, x.at.usable = 0;
    x.needed = task < total;
    if (i >= order.by_place && x.needed) {  // by row: rows outside the sequences have no owner, or whatever stood there
      x.at.b = __ldcg(at.owners + (i - order.by_place));
      x.needed = x.at.b >= 0 && x.at.b < a.B;
      if (x.needed) {
        const int64_t place = i - order.by_place - x.at.b - __ldg(a.cu + x.at.b);
        x.needed = place >= order.level && place <= a.T;
        x.at.place = static_cast<int>(place);
      }
    }
    if (x.needed) {
      const int2 state = __ldcg(reinterpret_cast<const int2*>(at.states + x.at.b));
      x.at.first = a.cu ? __ldg(a.cu + x.at.b) : x.at.b * (a.T / a.B);
      x.at.usable = state.x;
      x.needed = x.at.place < state.y && !(x.at.which == 1 && x.at.place >= state.x);
    }
    return x;
  };
  // The next task; whether there is one. It is looked for behind the join of the task before (64 sequences: 53 us; before it, 55).
  auto choose = [&](Where& w, int slot) {
    for (;;) {
      const Candidate x = ask();
      const uint32_t needed = __ballot_sync(kAll, x.needed);
      if (needed) {
        const int from = __ffs(needed) - 1;
        if (lane == from) {
          const Where& y = x.at;
          tasks[slot].row = y.which ? static_cast<const E*>(a.draft) + (y.first + y.place) * a.ld_draft
                                    : static_cast<const E*>(a.target) + (y.first + y.b + y.place) * a.ld_target;
          tasks[slot].rank = y.rank;
        }
        w.place = __shfl_sync(kAll, x.at.place, from), w.b = __shfl_sync(kAll, x.at.b, from);
        w.which = __shfl_sync(kAll, x.at.which, from), w.rank = __shfl_sync(kAll, x.at.rank, from);
        w.usable = __shfl_sync(kAll, x.at.usable, from), w.first = __shfl_sync(kAll, x.at.first, from);
        next += static_cast<int64_t>(from + 1) * gridDim.x;
        return true;
      }
      next += 32 * static_cast<int64_t>(gridDim.x);
      if (next >= total) break;
    }
    if (lane == 0) tasks[slot].row = nullptr;
    return false;
  };
  auto finish = [&](const Where& w, const RowSum* of_warps) {
    const int64_t row = w.first + w.b + w.place, draft = w.first + w.place;
    const bool decided = w.place < w.usable;  // by a draft
    int drafted = 0;
    float u = 0.0f;
    if (decided) {
      drafted = __ldg(a.drafts + draft);
      if (!kGreedy) u = __ldg(a.uniforms + draft);
    }
    RowSum x{-INFINITY, 0.0f, -INFINITY, V};
    if (lane < kWarps) x = of_warps[lane];
    x = merge_parts<F>(x, c, V);
    int before = 0;
    if (lane == 0) {
      const int64_t i = w.which ? a.T + a.B + draft : row;
      __stcg(reinterpret_cast<float4*>(at.sums + i * parts + w.rank), make_float4(x.m, x.s, x.largest, __int_as_float(x.arg)));
      if (decided) asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(at.summed + row) : "memory");
    }
    before = __shfl_sync(kAll, before, 0);
    if (!decided || before != kRows * parts - 1) return;
    __syncwarp();
    // All that is loaded, and then the two joins: others wait for what is decided here.
    RowSum p = part_of_row(at.sums + row * parts, parts, V), q{};
    float dp = 0.0f, dq = 0.0f;
    if (!kGreedy) dp = to_f32(__ldg(static_cast<const E*>(a.target) + row * a.ld_target + drafted));
    if constexpr (kModel) {
      q = part_of_row(at.sums + (a.T + a.B + draft) * parts, parts, V);
      dq = to_f32(__ldg(static_cast<const E*>(a.draft) + draft * a.ld_draft + drafted));
    }
    p = merge_parts<F>(p, c, V);
    if constexpr (kModel) q = merge_parts<F>(q, c, V);
    if (!taken_by<F>(p, q, drafted, u, dp, dq, c) && lane == 0) atomicMin(&at.states[w.b].needed, w.place + 1);
  };
  Where now{}, then{}, last{};
  bool any = choose(now, 0);
  __syncthreads();
  for (int k = 0;; ++k) {  // task k is being summed
    if (k > 0) finish(last, sums[(k - 1) & 1]);
    if (!any) return;
    any = choose(then, (k + 1) & 1);
    last = now, now = then;
    __syncthreads();
  }
}

// Draws the next token and writes what comes out: a cluster of CTAs a sequence, each with a part of the vocabulary.
template <class E, Form F>
__global__ void __launch_bounds__(kDrawThreads, 2) verify_draw_kernel(const VerifyArgs a, const int sum_parts, const int parts) {
  constexpr int N = kPer<E>;
  constexpr bool kModel = F == Form::kModel, kGreedy = F == Form::kGreedy;
  constexpr int kThreads = kDrawThreads, kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / parts, rank = blockIdx.x % parts, V = a.V;
  const Scale c = a.scale;
  const Workspace from(a, sum_parts);
  __shared__ RowSum rows[2];
  __shared__ uint64_t best_warps[2][kWarps], best[2][kMaxParts];
  __shared__ float scores[kWarps];

  if (parts > 1) cluster_arrive();  // this CTA runs
  const Sequence<E> s(a, b);
  griddep_wait();
  if (parts > 1) cluster_wait();  // every CTA runs
  if (!s.valid) return;
  const int2 state = __ldcg(reinterpret_cast<const int2*>(from.states + b));
  const int n = state.x, taken = state.y - 1;
  int32_t* const tokens = a.tokens + s.first + b;
  float* const logp = a.logp + s.first + b;
  // The places up to the refusal, a warp each (other CTAs: that one alone).
  for (int i = rank == 0 ? warp : taken + warp; i <= taken; i += kWarps) {
    const int drafted = i < taken ? __ldg(a.drafts + s.first + i) : 0;
    RowSum p = part_of_row(from.sums + (s.first + b + i) * sum_parts, sum_parts, V), q{-INFINITY, 0.0f, 0.0f, 0};
    if (kModel && i < n) q = part_of_row(from.sums + (a.T + a.B + s.first + i) * sum_parts, sum_parts, V);
    const float x = to_f32(__ldg(s.target + i * a.ld_target + drafted));
    p = merge_parts<F>(p, c, V);
    if (kModel && i < n) q = merge_parts<F>(q, c, V);
    else q = RowSum{0.0f, 1.0f, 0.0f, 0};
    if (lane != 0) continue;
    auto bad = [](const RowSum& r) { return !(fabsf(r.m) < INFINITY) || !(r.s < INFINITY); };
    if (bad(p) || bad(q)) flag(a.status, QRR_DEV_NONFINITE);
    if (i == taken) {
      rows[0] = sane(p), rows[1] = sane(q);
    } else {
      const RowSum whole = sane(p);
      const Ref at(whole.m, c);
      tokens[i] = drafted;
      logp[i] = ln_share(x, at, whole.s, Log2(at, whole.s), c);
    }
  }
  __syncthreads();
  const bool refused = taken < n;
  const RowSum p_row = rows[0], q_row = rows[1];
  const Ref p_ref(p_row.m, c), q_ref(q_row.m, c);
  int token = -1;
  if constexpr (kGreedy) {
    token = p_row.arg >= 0 && p_row.arg < V ? p_row.arg : -1;
  } else {
    const E* const row = s.target + taken * a.ld_target;
    const E* const other = kModel && refused ? s.draft + taken * a.ld_draft : nullptr;
    const float* const noise = a.noise + b * a.ld_noise;
    const int drafted = refused ? __ldg(a.drafts + s.first + taken) : -1;
    const Span<E> span(row, V, rank, parts);
    const int lead = span.lead;
    // The score itself. Both products are rounded: contracted to an FMA, the difference of equal rows would be a rounding
    // error and not 0.
    const bool minus = kModel && refused;
    auto scale = [&](const RowSum& r, const Ref& at) { return 1.0f / (at.far ? r.s : r.s * ex2_approx(c.exponent(-at.m, -at.r))); };
    const float inv_p = scale(p_row, p_ref), inv_q = minus ? scale(q_row, q_ref) : 0.0f;
    auto score = [&](float x, float y, float e, int v, bool whole_p) {
      float r = __fmul_rn(expf((x - p_ref.m) * c.inv_t), inv_p);
      if (minus && !whole_p) r -= __fmul_rn(expf((y - q_ref.m) * c.inv_t), inv_q);
      if (v == drafted && !kModel && !whole_p) r = 0.0f;
      return r / e;
    };
    // f(token) of this thread's part of the span: for looks that are rare, so by element, with no arrays that loops index.
    auto each = [&](auto f) {
      auto granule = [&](int i) {
#pragma unroll 1
        for (int v = max(i * N - lead, 0); v < min(i * N - lead + N, V); ++v) f(v);
      };
      if (tid == 0 && span.head >= 0) granule(0);
      for (int i = span.w0 + tid; i < span.w1; i += kThreads) granule(i);
      if (tid == kThreads - 1 && span.tail >= 0) granule(span.tail);
    };
    // An upper bound of max(p - q, 0) / e by the hardware's exponentials and reciprocal, within kSlack of p and q. A thread
    // keeps the best granule by it, and how good the second is.
    constexpr float kSlack = 0x1p-16f;
    const float p_up = (1.0f + kSlack) / p_row.s, q_down = minus ? (1.0f - kSlack) / q_row.s : 0.0f;
    // Of a looked-up draft nothing is left.
    const int gone = !kModel && refused ? (drafted + lead) / N : -1, gone_at = (drafted + lead) % N;
    float upper = 0.0f, second = 0.0f;
    int at = -1;
    auto bound = [&](int i, float(&x)[N], const float(&y)[N], const float(&z)[N]) {
      if (!kModel && i == gone) {
#pragma unroll
        for (int u = 0; u < N; ++u)
          if (u == gone_at) x[u] = -INFINITY;
      }
      float best = 0.0f;
#pragma unroll
      for (int u = 0; u < N; ++u) {
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(z[u]));
        float r = p_ref(x[u], c) * p_up;
        if (minus) r = fmaf(-q_ref(y[u], c), q_down, r);
        best = fmaxf(best, r * inv);
      }
      if (best > upper) second = upper, upper = best, at = i;
      else second = fmaxf(second, best);
    };
    // Whole granules, kBatch at a time with all their loads first. Rows and noise that start alike are read by 16 bytes all.
    constexpr int kBatch = 2;
    auto bounds = [&](auto alike) {
      constexpr bool kAlike = decltype(alike)::value;
      for (int i = span.w0 + tid; i < span.w1; i += kBatch * kThreads) {
        uint4 xs[kBatch], ys[kBatch];
        E y_each[kBatch][N];
        float z[kBatch][N];
#pragma unroll
        for (int w = 0; w < kBatch; ++w) {
          const int g = min(i + w * kThreads, span.w1 - 1), e = g * N - lead;
          xs[w] = __ldg(span.granules() + g);
          ys[w] = make_uint4(0, 0, 0, 0);
          if constexpr (kAlike) {
#pragma unroll
            for (int u = 0; u < N; u += 4) {
              const float4 f = __ldcs(reinterpret_cast<const float4*>(noise + e + u));
              z[w][u] = f.x, z[w][u + 1] = f.y, z[w][u + 2] = f.z, z[w][u + 3] = f.w;
            }
            if (minus) ys[w] = __ldg(reinterpret_cast<const uint4*>(other + e));
          } else {
#pragma unroll
            for (int u = 0; u < N; ++u) {
              z[w][u] = __ldg(noise + e + u);
              y_each[w][u] = minus ? __ldg(other + e + u) : E{};
            }
          }
        }
#pragma unroll
        for (int w = 0; w < kBatch; ++w) {
          if (i + w * kThreads >= span.w1) break;
          float x[N], y[N];
          unpack(xs[w], x);
          if constexpr (kAlike) {
            unpack(ys[w], y);
          } else {
#pragma unroll
            for (int u = 0; u < N; ++u) y[u] = to_f32(y_each[w][u]);
          }
          bound(i + w * kThreads, x, y, z[w]);
        }
      }
    };
    const int e0 = span.w0 * N - lead;
    const bool alike = (reinterpret_cast<uintptr_t>(noise + e0) & 15u) == 0 &&
                       (!minus || (reinterpret_cast<uintptr_t>(other + e0) & 15u) == 0);
    if (alike) bounds(std::true_type{});
    else bounds(std::false_type{});
    // The cut granules: -inf beside the row, with noise 1.
    auto bound_cut = [&](int i) {
      float x[N], y[N], z[N];
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const int v = i * N - lead + u;
        const bool in = v >= 0 && v < V;
        x[u] = in ? to_f32(row[v]) : -INFINITY;
        y[u] = in && minus ? to_f32(other[v]) : -INFINITY;
        z[u] = in ? noise[v] : 1.0f;
      }
      bound(i, x, y, z);
    };
    if (tid == 0 && span.head >= 0) bound_cut(0);
    if (tid == kThreads - 1 && span.tail >= 0) bound_cut(span.tail);
    // The best granule's score is what others have to reach by their bounds.
    float best_score = 0.0f;
    int best_at = 0;
    auto take = [&](float s, int v) {
      if (s > best_score || (s == best_score && s > 0.0f && v < best_at)) best_score = s, best_at = v;
    };
    auto look = [&](bool mine) {  // at the granules of these threads: by the warp, an element a lane
      for (uint32_t left = __ballot_sync(kAll, mine); left != 0; left &= left - 1) {
        const int v = __shfl_sync(kAll, at, __ffs(left) - 1) * N - lead + lane;
        if (lane < N && v >= 0 && v < V) take(score(to_f32(row[v]), minus ? to_f32(other[v]) : 0.0f, noise[v], v, false), v);
      }
    };
    // At the warp's best by the bounds first, then at those that may be better than the best of these.
    const float warp_upper = warp_max(upper);
    const uint32_t best_lanes = __ballot_sync(kAll, upper > 0.0f && upper == warp_upper);
    const bool first = best_lanes != 0 && lane == __ffs(best_lanes) - 1;
    look(first);
    const float warp_score = warp_max(best_score);
    if (lane == 0) scores[warp] = warp_score;
    __syncthreads();
    const float reached = warp_max(scores[min(lane, kWarps - 1)]);
    const bool several = at >= 0 && second >= reached && second > 0.0f;
    look(at >= 0 && upper >= reached && !first && !several);
    if (several) each([&](int v) { take(score(to_f32(row[v]), minus ? to_f32(other[v]) : 0.0f, noise[v], v, false), v); });
    uint64_t c_left = best_score > 0.0f ? candidate(best_score, best_at) : 0;
    // The best of all parts, in every thread.
    auto best_of_all = [&](uint64_t mine, int round) {
      mine = warp_max64(mine);
      if (lane == 0) best_warps[round][warp] = mine;
      __syncthreads();
      if (warp == 0) {
        const uint64_t x = warp_max64(best_warps[round][min(lane, kWarps - 1)]);
        if (lane < parts) st_cluster(&best[round][rank], lane, x);
      }
      if (parts > 1) {
        cluster_arrive();
        cluster_wait();
      } else {
        __syncthreads();
      }
      return warp_max64(best[round][min(lane, parts - 1)]);
    };
    uint64_t found = best_of_all(c_left, 0);
    if (found == 0 && refused) {  // nothing is left of p: from p itself
      best_score = 0.0f;
      each([&](int v) { take(score(to_f32(row[v]), 0.0f, noise[v], v, true), v); });
      found = best_of_all(best_score > 0.0f ? candidate(best_score, best_at) : 0, 1);
    }
    if (found) token = static_cast<int>(kAll - static_cast<uint32_t>(found));
  }
  if (rank == 0) {
    if (tid == 0) {
      tokens[taken] = token;
      logp[taken] = token < 0 ? 0.0f
                              : ln_share(to_f32(s.target[taken * a.ld_target + token]), p_ref, p_row.s, Log2(p_ref, p_row.s), c);
      a.accepted[b] = taken;
    }
    for (int i = taken + 1 + tid; i <= s.given; i += kThreads) {
      tokens[i] = -1;
      logp[i] = 0.0f;
    }
  }
}

// Parts of a row that is summed, of 32 KB: as much as the threads of a CTA have under way at once. (Four CTAs an SM: 56.8 us for
// 64 sequences of 8 drafts, three 58.9.)
int sum_parts(int64_t V, int fp32) {
  const int64_t granules = (V + (fp32 ? 3 : 7)) / (fp32 ? 4 : 8) + 1;
  int parts = 1;
  while (parts < kSumParts && granules > parts * static_cast<int64_t>(8 * kSumWorkers)) parts *= 2;
  return parts;
}

template <class... K, class... A>
cudaError_t launch_after(bool after, void (*kernel)(K...), unsigned grid, int cluster, int threads, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = after ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class E, Form F>
cudaError_t launch(const VerifyArgs& a, cudaStream_t stream) {
  constexpr int kRows = F == Form::kModel ? 2 : 1;
  int dev = 0, sms = kSMs;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  static OncePerDevice wide;
  e = wide(dev, [] { return cudaFuncSetAttribute(verify_draw_kernel<E, F>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); });
  if (e != cudaSuccess) return e;
  const int parts = sum_parts(a.V, a.fp32);
  e = launch_after(false, verify_begin_kernel<E>, static_cast<unsigned>((a.B + 7) / 8), 1, 256, stream, a, parts);
  if (e != cudaSuccess) return e;
  const int64_t tasks = (kRows * a.T + a.B) * parts;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tasks, static_cast<int64_t>(sms) * kSumCtas));
  e = launch_after(true, verify_sums_kernel<E, F>, grid, 1, kSumThreads, stream, a, parts);
  if (e != cudaSuccess) return e;
  // Enough CTAs for the SMs draw the tokens, a granule a thread at least. (Enough for two an SM: 62 us where this took 56 for 64
  // sequences, 57 for 52 with 200: what a CTA does beside its granules costs more.)
  const int granules = granules_of<E>(kPer<E> - 1, a.V);
  int draw_parts = 1;
  while (F != Form::kGreedy && draw_parts < kMaxParts && static_cast<int64_t>(a.B) * draw_parts < sms && granules > draw_parts * kDrawThreads)
    draw_parts *= 2;
  return launch_after(true, verify_draw_kernel<E, F>, static_cast<unsigned>(a.B) * draw_parts, draw_parts, kDrawThreads, stream, a, parts,
                      draw_parts);
}

template <class E>
cudaError_t launch(const VerifyArgs& a, cudaStream_t stream) {
  if (a.temperature == 0.0) return launch<E, Form::kGreedy>(a, stream);
  return a.draft ? launch<E, Form::kModel>(a, stream) : launch<E, Form::kLookup>(a, stream);
}

}  // namespace

size_t verify_drafts_ws_bytes(int64_t T, int64_t B, int64_t V, int fp32) {
  return static_cast<size_t>(2 * T + B) * sum_parts(V, fp32) * sizeof(RowSum) + static_cast<size_t>(B) * sizeof(State) +
         2 * static_cast<size_t>(T + B) * sizeof(int);
}

cudaError_t launch_verify_drafts(VerifyArgs a, cudaStream_t stream) {
  if (a.B == 0) return cudaSuccess;
  a.scale = scale_of(a.temperature == 0.0 ? 1.0 : a.temperature);
  return a.fp32 ? launch<float>(a, stream) : launch<Bf16>(a, stream);
}

}  // namespace qrr
