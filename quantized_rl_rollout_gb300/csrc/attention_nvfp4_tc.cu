// Attention over the paged NVFP4 key/value cache, many query rows a sequence
// (prompts, new turns): the formulas of attention_nvfp4.cu on the 5th-generation
// tensor cores.
//
// An item is 256 rows of a sequence and a KV head (row = new token x G + query
// head of the group), as two tiles of 128; its keys and values come in tiles of
// 128 tokens.  The key tiles of all items form one sequence that is cut in
// equal ranges, one a CTA (one CTA an SM), as in the other kernel; pieces of
// items that cross ranges go to the workspace and are joined afterwards.
//
// A CTA's warps:
//   0..3, 4..7  softmax of row tile 0 and 1: a thread a row.  Loads its query
//               row as f16 (a power of two a row) into shared memory, then for
//               every key tile turns the scores in tensor memory into weights
//               (f16, over the scores' own columns), and at the end scales and
//               stores the row.
//   8..11       codes and scales -> f16 key and value tiles in shared memory
//               (code x block scale is exact), two stages each, 128-byte
//               swizzled.
//   12          issues the MMAs: S_i = Q_i K^T (M128 N128), O_i += P_i V
//               (P from tensor memory, V MN-major).  Order per key tile:
//               PV_0, S_0 of the next, PV_1, S_1 of the next, so one tile's
//               softmax runs under the other's MMAs.
//   13          fetches codes and scales by bulk copies, a run of tokens in one
//               page each, into a ring of three raw tiles (keys and values in
//               turn), running ahead over the ends of items.
// Tensor memory: S_0, S_1, O_0, O_1 of 128 columns each.
//
// A row's weights are formed with the running reference in one pass over its
// scores; only when a score exceeds it by kRoom (and on a row's first tile) the
// pass is repeated with a new one (a whole number) and what the row has so far
// is scaled.
//
// A key tile of 256 rows takes 3800 cycles, of which the MMAs are 2048 (64 an
// M128 N128 K16): a group's chain of scores (480 to reach the softmax), softmax (2000),
// weights to the issuer (300) and its two MMAs (1024) is what bounds, the other
// group's runs beside it.  An item's start and end take 10000 more: query rows 5000,
// output 4500.  19 x 64 tokens over 8128, 4 query heads a head of 128: 1085 TFLOP/s; a
// prompt of 4096 tokens 880 (156 us, 8 of start and 13 of join among them), of 16384
// 1230; 4 x 300..700 tokens over 6000..10000 (5 query heads) 1050..1150.  Measured
// and not taken: scores in two 64-column buffers (as fast: the MMAs read the
// queries twice as often); the first half of a tile's weights handed over early,
// the next codes in registers while one tile is converted, query rows copied by
// two warps of their own (prompt 4 to 9 % longer); 16 softmax warps, two a row
// (24 %); a tile's maximum before its weights (20 %: the scores are read twice).
#include "attention_nvfp4.cuh"
#include "tc.cuh"

namespace qrr {

using namespace attn4;
using namespace attn4::many;

namespace {

constexpr int kThreads = 14 * 32;
constexpr int kMinTiles = 4;  // key tiles of a range
constexpr int kSeqs = 1024;   // sequences whose counts are kept in shared memory
constexpr uint32_t kTmemCols = 512;

template <int D>
struct Smem {
  static constexpr int kTile = 128 * D * 2;  // bytes of a query, key or value tile
  uint8_t q[2][kTile], k[2][kTile], v[2][kTile];
  // codes and scales of the next three key or value tiles
  uint8_t raw[3][64 * D];
  uint8_t raw_s[3][8 * D];
  uint64_t raw_full[3], raw_empty[3];
  uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2], done;
  uint32_t tmem;
  int abort;
  int32_t seq_widths[kSeqs];  // -1: above 32 bits
  int64_t part[kThreads / 32];
};

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// The wait for this thread's tensor-memory loads, with the loaded registers as
// operands so that no use of them moves above it.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// What one KV head of sequence b counts for over all its row tiles, by a warp.
__device__ __forceinline__ int64_t seq_width(const Params& p, int b, int lane) {
  const int64_t sum = lane_width(p.byG, seq_of(p, b), lane);
  // a lane's sum is below 2^41 (2^17 row tiles of 2^23 key tiles): 26 bits and the rest
  const uint32_t lo = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(sum) & 0x3FFFFFFu);
  const uint32_t hi = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(sum >> 26));
  return (static_cast<int64_t>(hi) << 26) + lo;
}

// The walk over a range's pieces of items; every thread of the CTA makes it.
struct Walk {
  Seq s;
  int b, h, qt, qts, tiles;  // current item and its key tiles
  int t0, t1;                // the piece's key tiles
  int counts;                // what it takes of the range
  int64_t left;              // of the range, from t0 on
  __device__ __forceinline__ void piece(const Params& p) {
    tiles = key_tiles(p.byG, s, qt);
    counts = static_cast<int>(min(static_cast<int64_t>(tiles + kItemCost - t0), left));
    t1 = min(t0 + counts, tiles);
  }
  // false: the range ends with what its only item counts for beyond its tiles
  __device__ __forceinline__ bool begin(const Params& p, int b_, int64_t off, int64_t left_) {
    b = b_;
    left = left_;
    s = seq_of(p, b);
    qts = row_tiles(p.byG, s);
    const int lane = threadIdx.x & 31;
    const int64_t per = seq_width(p, b, lane);  // of one head
    h = static_cast<int>(off / per);
    int64_t rest = off - h * per;
    for (qt = 0;; qt += 32) {  // 32 row tiles at a time
      const int own = qt + lane < qts ? width(p.byG, s, qt + lane) : 0;
      int incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t in = __ballot_sync(0xFFFFFFFFu, rest >= incl - own && rest < incl);
      if (in) {
        const int k = __ffs(static_cast<int>(in)) - 1;
        rest -= __shfl_sync(0xFFFFFFFFu, incl - own, k);
        qt += k;
        break;
      }
      rest -= __shfl_sync(0xFFFFFFFFu, incl, 31);
      if (qt + 32 >= qts) {  // not reached: off lies in the sequence
        qt = max(qts - 1, 0);
        rest = 0;
        break;
      }
    }
    t0 = static_cast<int>(rest);
    piece(p);
    return t0 < tiles || next(p);
  }
  __device__ __forceinline__ bool next(const Params& p) {
    left -= counts;
    if (left <= 0) return false;
    t0 = 0;
    if (++qt == qts) {
      qt = 0;
      if (++h == p.c.Hkv) {
        h = 0;
        do {
          if (++b >= p.c.B) return false;
          s = seq_of(p, b);
          qts = row_tiles(p.byG, s);
        } while (qts == 0);
      }
    }
    piece(p);
    return true;
  }
};

// ---- codes -> f16 tiles ------------------------------------------------------

// A lane's share of a raw tile, and its conversion.  Row r of a tile lies at
// 128 r in each of its D / 64 column halves of 16 KB, its 16-byte pieces at
// their index exclusive-or r % 8.  A thread takes a chunk of 32 values of one
// row in each of D / 32 passes.
template <int D>
struct Codes {
  static constexpr int kPasses = D / 32, kRowsPass = 128 / kPasses;
  uint4 w[kPasses];
  uint32_t s[kPasses];  // the chunk's two block scales
  // rows from `live` on have no token: their scales count as zero (what lies
  // there may be anything)
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int live, int t) {
    const int c = t % kPasses;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = i * kRowsPass + t / kPasses;
      w[i] = *reinterpret_cast<const uint4*>(codes + r * (D / 2) + 16 * c);
      s[i] = *reinterpret_cast<const uint16_t*>(scales + r * (D / 16) + 2 * c);
      if (r >= live) s[i] = 0u;
    }
  }
  __device__ __forceinline__ void convert(uint8_t* tile, int t) const {
    const int c = t % kPasses, r0 = t / kPasses;
    // the two column halves have the same banks: lanes of the second one take
    // their words in another order
    const bool swap = c >= 2;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = i * kRowsPass + r0;
      const uint32_t s2 = e4m3x2_to_f16x2(s[i]);
      const uint32_t sc[2] = {__byte_perm(s2, s2, swap ? 0x3232 : 0x1010), __byte_perm(s2, s2, swap ? 0x1010 : 0x3232)};
      const uint32_t ww[4] = {swap ? w[i].z : w[i].x, swap ? w[i].w : w[i].y, swap ? w[i].x : w[i].z, swap ? w[i].y : w[i].w};
      uint8_t* row = tile + (c >> 1) * (128 * 128) + r * 128;
      const int x = (4 * (c & 1)) ^ (swap ? 2 : 0) ^ (r & 7);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t f[4];
        f16x2x4_from_e2m1x8(ww[k], f);
        const uint32_t y = sc[k >> 1];
        *reinterpret_cast<uint4*>(row + ((x ^ k) << 4)) = make_uint4(hmul2(f[0], y), hmul2(f[1], y), hmul2(f[2], y), hmul2(f[3], y));
      }
    }
  }
};

// ---- softmax -------------------------------------------------------------------

// 32 scores of a row -> weights 2^(s f - m): f16 pairs, their fp32 sums, the
// largest score.
__device__ __forceinline__ void weights(const uint32_t (&r)[32], uint64_t f2, uint64_t nm2, float& top, uint64_t& sum,
                                        uint32_t (&out)[16]) {
  float mx[2] = {-INFINITY, -INFINITY};
  uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float a = __uint_as_float(r[2 * i]), b = __uint_as_float(r[2 * i + 1]);
    mx[i & 1] = max3(mx[i & 1], a, b);
    uint64_t x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
    asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(x) : "l"(f2), "l"(nm2));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
    a = ex2(a);
    b = ex2(b);
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(acc[i & 1]) : "l"(x));
    out[i] = f16x2(a, b);
  }
  top = fmaxf(mx[0], mx[1]);
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(sum) : "l"(acc[0]), "l"(acc[1]));
}

__device__ __forceinline__ uint64_t twice(float x) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
  return r;
}

// 64 bytes of a row.  A store instruction takes a cycle a lane and row here (each
// lane's row lies elsewhere), so as few as there can be: 32 bytes a lane where the
// rows are so aligned.
__device__ __forceinline__ void store16(uint16_t* to, const uint32_t (&y)[16], bool wide) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < 16; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + 2 * i), "r"(y[i]), "r"(y[i + 1]),
                   "r"(y[i + 2]), "r"(y[i + 3]), "r"(y[i + 4]), "r"(y[i + 5]), "r"(y[i + 6]), "r"(y[i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<uint4*>(to)[i] = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
  }
}

// Two bf16 values times a power of two, as f16.
__device__ __forceinline__ uint32_t scaled_f16x2(uint32_t w, uint64_t sc) {
  uint64_t x;
  float a, b;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(bf16_lo(w)), "f"(bf16_hi(w)));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(sc));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
  return f16x2(a, b);
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_nvfp4_tc_kernel(const Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<D>& sh = *reinterpret_cast<Smem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  volatile int* abort = &sh.abort;

  griddep_launch_dependents();
  // ---- this CTA's range of the key tiles
  const int B = p.c.B;
  int64_t mine = 0;
  for (int b = warp; b < B; b += kThreads / 32) {
    const int64_t n = seq_width(p, b, lane);
    if (lane == 0 && b < kSeqs) sh.seq_widths[b] = n <= INT32_MAX ? static_cast<int>(n) : -1;
    mine += n;
  }
  if (lane == 0) sh.part[warp] = mine;
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      mbar_init(&sh.raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 4);
      mbar_init(&sh.k_full[i], 4);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_full[i], 4);
      mbar_init(&sh.v_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.o_full[i], 1);
    }
    mbar_init(&sh.done, 1);
    sh.abort = 0;
    fence_barrier_init();
  }
  if (warp == 12) tmem_alloc(&sh.tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  int64_t total = 0;
  for (int w = 0; w < kThreads / 32; ++w) total += sh.part[w];
  total *= p.c.Hkv;
  const int64_t per = max(static_cast<int64_t>(kMinTiles), (total + gridDim.x - 1) / gridDim.x);
  const int64_t begin = blockIdx.x * per, end = min(begin + per, total);
  Walk w;
  bool work = begin < end;
  if (work) {
    // the sequence that the range begins in; every warp looks for itself
    int64_t off = begin;
    int found = -1;
    for (int b0 = 0; b0 < B && found < 0; b0 += 32) {
      const bool in_b = b0 + lane < B, kept = b0 + 32 <= kSeqs;
      int64_t n = kept && in_b ? sh.seq_widths[b0 + lane] : 0;
      for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, kept ? n < 0 : in_b); todo; todo &= todo - 1) {
        const int i = __ffs(static_cast<int>(todo)) - 1;
        const int64_t x = seq_width(p, b0 + i, lane);
        if (lane == i) n = x;
      }
      const int64_t own = n * p.c.Hkv;
      int64_t incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t in = __ballot_sync(0xFFFFFFFFu, off >= incl - own && off < incl);
      if (in) {
        found = __ffs(static_cast<int>(in)) - 1;
        off -= __shfl_sync(0xFFFFFFFFu, incl - own, found);
        found += b0;
      } else {
        off -= __shfl_sync(0xFFFFFFFFu, incl, 31);
      }
    }
    work = w.begin(p, found, off, end - begin);
  }
  if (!work) {
    if (tid == 0) {
      p.rec[blockIdx.x].pieces = 0;
      if (blockIdx.x == 0) griddep_wait();
    }
    if (warp == 12) tmem_dealloc(tmem, kTmemCols);
    return;
  }

  if (warp < 8) {
    // ---------------- softmax ----------------
    const int tile = warp >> 2, r = tid & 127;
    const uint32_t ts = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 128 * tile;
    const uint32_t to = ts + 256;
    // the warp's 32 rows of the query tile, by 16-byte pieces: lanes `sub` and
    // `piece` of a copy of kAtOnce rows
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
    uint8_t* const stage = sh.q[tile];
    auto at = [&](int rr, int pc) { return stage + (pc >> 3) * (128 * 128) + rr * 128 + (((pc & 7) ^ (rr & 7)) << 4); };
    // The query rows of a piece come in two steps: copied as they are, kLanes
    // lanes a row (as soon as no MMA reads the ones before), then turned into f16
    // in place, a thread a row.  (Loops that run once a piece are kept rolled:
    // straight code would wait for its own instructions.)
    auto copy_rows = [&](const Walk& x) {
      const int piece = lane % kLanes, sub = lane / kLanes;
      const int row = x.qt * kRows + 128 * tile + r, rows = x.s.n * p.G;
      const bool in = row < rows;
      const int token = in ? x.s.first + p.byG.div(row) : -1, head = in ? x.h * p.G + p.byG.mod(row) : 0;
#pragma unroll 4
      for (int i = 0; i < kLanes; ++i) {
        const int from = i * kAtOnce + sub;  // the copied row's own lane
        const int tq = __shfl_sync(0xFFFFFFFFu, token, from), hq = __shfl_sync(0xFFFFFFFFu, head, from);
        const uint16_t* src = p.q + max(tq, 0) * p.ld_q + hq * D + piece * 8;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(at(32 * (warp & 3) + from, piece))),
                     "l"(src), "r"(tq >= 0 ? 16 : 0)
                     : "memory");
      }
    };
    // returns the factor of the row's scores
    auto convert_rows = [&](const Walk& x) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      uint32_t mx = 0u;
#pragma unroll 8
      for (int i = 0; i < kLanes; ++i) mx = max(mx, absmax_bits8(*reinterpret_cast<const uint4*>(at(r, i))));
      if (mx >= 0x7F80u) flag(p.status, QRR_DEV_NONFINITE);
      const int e = max(query_exp(mx), -127);  // one factor 2^-e (a row below 2^-113 comes out smaller)
      const uint64_t sc = twice(__uint_as_float(static_cast<uint32_t>(127 - e) << 23));
#pragma unroll 4
      for (int i = 0; i < kLanes; ++i) {
        uint4* y = reinterpret_cast<uint4*>(at(r, i));
        const uint4 v = *y;
        *y = make_uint4(scaled_f16x2(v.x, sc), scaled_f16x2(v.y, sc), scaled_f16x2(v.z, sc), scaled_f16x2(v.w, sc));
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full[tile]);
      // at least the smallest normal value: a masked score times it stays -inf
      return fmaxf(p.scale * kLog2e * (p.c.kg ? __ldg(p.c.kg + x.h) : 1.0f) * ldexpf(1.0f, e), 1.17549435e-38f);
    };
    auto active = [&](const Walk& x) { return x.qt * kRows + 128 * tile < x.s.n * p.G; };
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    Record rec{};
    uint32_t s_phase = 0, o_phase = 0;
    bool ok = true, more = true;
    float f = 1.0f;
    if (active(w)) {
      copy_rows(w);
      f = convert_rows(w);
    }
    while (more) {
      Walk nx = w;
      more = nx.next(p);
      float next_f = 1.0f;
      if (active(w)) {
        const int row = w.qt * kRows + 128 * tile + r, rows = w.s.n * p.G;
        const bool in = row < rows;
        const uint64_t f2 = twice(f);
        // rows behind the last one are never read: they need no mask
        const int lim = in ? min(w.s.pos + p.byG.div(row), w.s.last) : kAllSeen;
        const int lim_warp = __reduce_min_sync(0xFFFFFFFFu, lim);
        float m = kNone, l = 0.0f;
        for (int j = w.t0; j < w.t1 && ok; ++j) {
          if (!mbar_wait(&sh.s_full[tile], s_phase, abort, p.status)) {
            ok = false;
            break;
          }
          s_phase ^= 1;
          tc_fence_after();
          // the last scores are formed: no MMA reads these query rows any more
          if (j + 1 == w.t1 && more && active(nx)) copy_rows(nx);
          const int seen = seen_of(lim, j);  // of this tile's tokens
          const bool mask = kTok * j + kTok - 1 > lim_warp;
          // 32 columns at a time; weights 32 c .. 32 c + 31 go to the columns
          // 16 c .. 16 c + 15, whose scores have been loaded by then
          auto chunk = [&](uint32_t (&x)[32], int c) {
            if (mask)
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = i < seen - 32 * c ? x[i] : 0xFF800000u;
            uint32_t y[16];
            float top;
            uint64_t sum;
            while (true) {
              weights(x, f2, twice(-m), top, sum, y);
              const bool move = top * f > m + kRoom;
              if (!__any_sync(0xFFFFFFFFu, move)) break;
              // the weights of the chunks before are read back below: a load of tensor
              // memory is not ordered behind a store but by this wait
              tmem_st_wait();
              // A new reference: scale what the row has so far, and form the chunk's weights
              // again.  References are whole numbers, so the factor is a power of two and
              // a stored weight is rounded again only below f16's normal range (by little
              // more than 2^-25, 2^-32 of the row's largest weight).  f16 has powers of
              // two down to 2^-24: smaller factors come as a product.
              const float m1 = move ? floorf(top * f) - kLift : m, by = m - m1;
              const float a = by > -127.0f ? __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(by)) << 23) : 0.0f;
              m = m1;
              l *= a;
              const float a_hi = fmaxf(a, 0x1p-24f), a_lo = a < 0x1p-24f ? a * 0x1p24f : 1.0f;
              const uint32_t hi2 = f16x2(a_hi, a_hi), lo2 = f16x2(a_lo, a_lo);
#pragma unroll 1
              for (int k = 0; k < c; ++k) {
                uint32_t z[16];
                tmem_ld16(ts + 16 * k, z);
                tmem_ld_wait16(z);
#pragma unroll
                for (int i = 0; i < 16; ++i) z[i] = hmul2(hmul2(z[i], hi2), lo2);
                tmem_st16(ts + 16 * k, z);
              }
              if (j > w.t0)
#pragma unroll 1
                for (int k = 0; k < D / 16; ++k) {
                  uint32_t z[16];
                  tmem_ld16(to + 16 * k, z);
                  tmem_ld_wait16(z);
#pragma unroll
                  for (int i = 0; i < 16; ++i) z[i] = __float_as_uint(__uint_as_float(z[i]) * a);
                  tmem_st16(to + 16 * k, z);
                }
              tmem_st_wait();
            }
            float s0, s1;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(s0), "=f"(s1) : "l"(sum));
            l += s0 + s1;
            tmem_st16(ts + 16 * c, y);
          };
          uint32_t xa[32], xb[32];
          tmem_ld32(ts, xa);
          tmem_ld_wait32(xa);
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {
            tmem_ld32(ts + 32 * c + 32, xb);
            chunk(xa, c);
            tmem_ld_wait32(xb);
            tmem_ld32(ts + 64, xa);  // (the last time for nothing)
            chunk(xb, c + 1);
            tmem_ld_wait32(xa);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_full[tile]);
        }
        if (!ok) break;
        if (more && active(nx)) next_f = convert_rows(nx);
        // ---- the row's result
        if (!mbar_wait(&sh.o_full[tile], o_phase, abort, p.status)) break;
        o_phase ^= 1;
        tc_fence_after();
        const bool whole = w.t0 == 0 && w.t1 == w.tiles;
        const float vg = p.c.vg ? __ldg(p.c.vg + w.h) : 1.0f;
        const float inv = row_factor(vg, l);
        const int64_t orow = in ? out_row(p, w.s.first, w.h, row) : 0;
        const int64_t piece = 2 * blockIdx.x + (w.t0 > 0 ? 0 : 1);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[32];
          tmem_ld32(to + 32 * c, x);
          tmem_ld_wait32(x);
          if (whole) {
            uint32_t y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const __nv_bfloat162 v2 = __floats2bfloat162_rn(__uint_as_float(x[2 * i]) * inv, __uint_as_float(x[2 * i + 1]) * inv);
              y[i] = *reinterpret_cast<const uint32_t*>(&v2);
            }
            if (in) store16(p.out + orow * D + 32 * c, y, wide);
          } else if (in) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<uint4*>(p.po)[(piece * (D / 4) + 8 * c + i) * kRows + 128 * tile + r] =
                  make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
        }
        if (in && whole && p.lse) p.lse[orow] = row_lse(m, l);
        if (in && !whole) p.pm[piece * kRows + 128 * tile + r] = m, p.pl[piece * kRows + 128 * tile + r] = l;
        __syncwarp();
        tc_fence_before();
      } else if (more && active(nx)) {
        copy_rows(nx);
        next_f = convert_rows(nx);
      }
      if (tid == 0 && w.t0 == 0 && w.t1 < w.tiles) {
        rec.pieces = 1 + static_cast<int>((w.tiles - w.t1 + per - 1) / per);
        rec.range = blockIdx.x, rec.rt = w.qt, rec.h = w.h, rec.first = w.s.first, rec.n = w.s.n;
      }
      w = nx;
      f = next_f;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (tid == 0) p.rec[blockIdx.x] = rec;
  } else if (warp < 12) {
    // ---------------- codes -> key and value tiles ----------------
    const int t = tid - 256;
    int use = 0, slot = 0, turn = 0;
    bool ok = true;
    auto half = [&](uint8_t* tile, uint64_t* empty, uint64_t* full, int live) {
      if (!mbar_wait(&sh.raw_full[slot], turn & 1, abort, p.status)) return false;
      Codes<D> x;
      x.load(sh.raw[slot], sh.raw_s[slot], live, t);
      // The next copy into the slot is a write of the asynchronous proxy: only this
      // fence orders the reads above before it (the arrive alone does not; without
      // the fence a read can come after the wait below, and finds the next tile).
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.raw_empty[slot]);
      if (use >= 2 && !mbar_wait(empty, ((use >> 1) - 1) & 1, abort, p.status)) return false;
      x.convert(tile, t);
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
      if (++slot == 3) slot = 0, ++turn;
      return true;
    };
    do {
      const int last = last_seen(p.byG, w.s, w.qt);
      for (int j = w.t0; j < w.t1 && ok; ++j, ++use) {
        const int st = use & 1, live = seen_of(last, j);
        ok = half(sh.k[st], &sh.k_empty[st], &sh.k_full[st], live) && half(sh.v[st], &sh.v_empty[st], &sh.v_full[st], live);
      }
    } while (ok && w.next(p));
  } else if (warp == 13) {
    // ---------------- codes and scales into the ring ----------------
    const int run = min(1 << p.c.page_shift, kTok);  // tokens of a copy: of one page
    int slot = 0, n = 0;
    bool ok = true;
    do {
      const int last = last_seen(p.byG, w.s, w.qt);
      const int32_t* table = p.c.table + static_cast<int64_t>(w.b) * p.c.max_pages;
      for (int j = w.t0; j < w.t1 && ok; ++j) {
        const int tok = kTok * j + lane * run;
        int rows = lane * run < kTok ? min(max(last + 1 - tok, 0), run) : 0;
        int64_t row = 0;
        if (rows > 0) {
          const int pg = __ldg(table + (tok >> p.c.page_shift));
          if (pg >= 0 && pg < p.c.num_pages) {
            row = kv_row(p.c, pg, w.h, tok & ((1 << p.c.page_shift) - 1));
          } else {
            flag(p.status, QRR_DEV_BAD_INDEX);
            rows = 0;
          }
        }
        rows = (rows + 3) & ~3;  // whole 16 bytes of scales; within the page
        const uint32_t bytes = __reduce_add_sync(0xFFFFFFFFu, rows * (D / 2 + D / 16));
        for (int v = 0; v < 2; ++v, ++n) {
          if (n >= 3 && !mbar_wait(&sh.raw_empty[slot], (n / 3 - 1) & 1, abort, p.status)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&sh.raw_full[slot], bytes);
          __syncwarp();
          if (rows > 0) {
            bulk_load(sh.raw[slot] + lane * run * (D / 2), (v ? p.c.vc : p.c.kc) + row * (D / 2), rows * (D / 2), &sh.raw_full[slot]);
            bulk_load(sh.raw_s[slot] + lane * run * (D / 16), (v ? p.c.vs : p.c.ks) + row * (D / 16), rows * (D / 16), &sh.raw_full[slot]);
          }
          if (++slot == 3) slot = 0;
        }
      }
    } while (ok && w.next(p));
    // every issued copy has landed before the CTA exits
    volatile int no_abort = 0;
    for (int i = max(0, n - 3); i < n; ++i) mbar_wait(&sh.raw_full[i % 3], (i / 3) & 1, &no_abort, p.status);
  } else {
    // ---------------- MMA issuer ----------------
    if (elect_one()) {
      constexpr uint32_t id_s = make_idesc(kFmtF16, kFmtF16, 128, kTok);
      constexpr uint32_t id_o = make_idesc_major(kFmtF16, kFmtF16, 128, D, false, true);
      int use = 0, use0 = 0;
      uint32_t p_phase[2] = {0, 0}, q_phase[2] = {0, 0};
      bool ok = true;
      do {
        const int tiles = w.qt * kRows + 128 < w.s.n * p.G ? 2 : 1;  // row tiles with rows
        const int n = w.t1 - w.t0;
        use0 = use;
        auto scores = [&](int i, int st) {
          const uint32_t a = smem_u32(sh.q[i]), b = smem_u32(sh.k[st]);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k >> 2) * (128 * 128) + (k & 3) * 32;
            mma_bf16_ss(tmem + 128 * i, sw128_desc(a + off), sw128_desc(b + off), id_s, k > 0);
          }
          mma_commit(&sh.s_full[i]);
        };
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          if (!ok || !mbar_wait(bar, parity, abort, p.status)) {
            ok = false;
            return false;
          }
          tc_fence_after();
          return true;
        };
        for (int i = 0; i < tiles; ++i) {
          if (!wait(&sh.q_full[i], q_phase[i])) break;
          q_phase[i] ^= 1;
          if (i == 0 && !wait(&sh.k_full[use & 1], (use >> 1) & 1)) break;
          scores(i, use & 1);
        }
        if (ok) mma_commit(&sh.k_empty[use & 1]);
        for (int j = 0; j < n && ok; ++j, ++use) {
          const int st = use & 1;
          for (int i = 0; i < tiles; ++i) {
            if (!wait(&sh.p_full[i], p_phase[i])) break;
            p_phase[i] ^= 1;
            if (i == 0 && !wait(&sh.v_full[st], (use >> 1) & 1)) break;
            uint64_t b[8];
            const uint32_t v = smem_u32(sh.v[st]);
#pragma unroll
            for (int k = 0; k < 8; ++k) b[k] = sw128_mn_desc(v + k * 2048, 128 * 128);
            mma8_ts(tmem + 256 + 128 * i, tmem + 128 * i, b, id_o, j > 0);
            if (i + 1 == tiles) mma_commit(&sh.v_empty[st]);
            if (j + 1 == n) mma_commit(&sh.o_full[i]);
            else {
              const int su = use + 1;
              if (i == 0 && !wait(&sh.k_full[su & 1], (su >> 1) & 1)) break;
              scores(i, su & 1);
              if (i + 1 == tiles) mma_commit(&sh.k_empty[su & 1]);
            }
          }
        }
        use = use0 + n;
      } while (ok && w.next(p));
      mma_commit(&sh.done);
      volatile int no_abort = 0;
      mbar_wait(&sh.done, 0, &no_abort, p.status);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  // this grid ends after the one that it may run beside (see the launch)
  if (blockIdx.x == 0 && tid == 0) griddep_wait();
}

namespace {

// Joins this kernel's items: many rows, most often of two pieces.  A piece's output
// is [D / 4][row][4], so that the rows' threads write side by side.  Here eight
// rows a warp, four lanes a row, a lane every fourth four values; two pieces'
// loads at a time, sums in the order of the pieces.
template <int D>
__global__ void __launch_bounds__(256) join_many_kernel(const Params p) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, part = lane >> 3, first = (blockIdx.x % (kRows / 64)) * 64 + (threadIdx.x >> 5) * 8;
  const Record rec = p.rec[blockIdx.x / (kRows / 64)];
  const int r = first + (lane & 7), row = rec.rt * kRows + r;
  if (rec.pieces == 0 || rec.rt * kRows + first >= rec.n * p.G) return;  // (the same for the warp)
  const float vg = p.c.vg ? __ldg(p.c.vg + rec.h) : 1.0f;
  auto piece = [&](int i) { return piece_row(rec, i, 1); };
  float m = kNone, l = 0.0f, o[D / 16][4] = {};
  for (int i0 = 0; i0 < rec.pieces; i0 += 4) {
    // the row's lanes take a piece's (m, l) each
    const int n = min(4, rec.pieces - i0);
    float mi = kNone, li = 0.0f;
    if (part < n) {
      mi = p.pm[piece(i0 + part) * kRows + r];
      li = p.pl[piece(i0 + part) * kRows + r];
    }
    float a = 0.0f;
#pragma unroll 1
    for (int i = 0; i < n; i += 2) {
      float4 x[2][D / 16];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          x[u][k] = reinterpret_cast<const float4*>(p.po)[(piece(i0 + min(i + u, n - 1)) * (D / 4) + 4 * k + part) * kRows + r];
      if (i == 0) {
        float top = fmaxf(mi, __shfl_xor_sync(0xFFFFFFFFu, mi, 8));
        top = fmaxf(m, fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16)));
        const float old = ex2(m - top);
        m = top;
        a = ex2(mi - top);
        float sum = a * li;
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
        l = l * old + sum;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int d = 0; d < 4; ++d) o[k][d] *= old;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float ai = i + u < n ? __shfl_sync(0xFFFFFFFFu, a, 8 * (i + u) + (lane & 7)) : 0.0f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          o[k][0] += ai * x[u][k].x, o[k][1] += ai * x[u][k].y, o[k][2] += ai * x[u][k].z, o[k][3] += ai * x[u][k].w;
      }
    }
  }
  if (row >= rec.n * p.G) return;
  const float inv = row_factor(vg, l);
  const int64_t orow = out_row(p, rec.first, rec.h, row);
#pragma unroll
  for (int k = 0; k < D / 16; ++k) *reinterpret_cast<uint2*>(p.out + orow * D + 16 * k + 4 * part) = bf16x4(o[k], inv);
  if (p.lse && part == 0) p.lse[orow] = row_lse(m, l);
}

template <int D>
cudaError_t launch(const AttnNvfp4Args& a, uint8_t* ws, bool beside, cudaStream_t stream) {
  constexpr int smem = static_cast<int>(sizeof(Smem<D>)) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory");
  int dev = 0, sms = kSMs;
  cudaError_t e = device_of(dev, sms);
  if (e != cudaSuccess) return e;
  static OncePerDevice limit;
  e = limit(dev, [] { return cudaFuncSetAttribute(attn_nvfp4_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  const int grid = sms < kMaxSms ? sms : kMaxSms;
  const Params p = make_params(a, ws, grid, kRows, grid);
  // behind the other kernel's launches it may run beside them: what it reads was
  // there before those, what it writes they do not touch
  if (beside) {
    e = launch_dependent(attn_nvfp4_tc_kernel<D>, dim3(grid), kThreads, smem, stream, p);
    if (e != cudaSuccess) return e;
  } else {
    attn_nvfp4_tc_kernel<D><<<grid, kThreads, smem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(join_many_kernel<D>, dim3(grid * (kRows / 64)), 256, 0, stream, p);
}

}  // namespace

size_t attention_nvfp4_tc_ws_bytes(int D) { return ws_bytes(D, kMaxSms, kRows, kMaxSms); }

cudaError_t launch_attention_nvfp4_tc(const AttnNvfp4Args& a, uint8_t* ws, bool beside, cudaStream_t stream) {
  return a.c.D == 128 ? launch<128>(a, ws, beside, stream) : launch<64>(a, ws, beside, stream);
}

}  // namespace qrr
