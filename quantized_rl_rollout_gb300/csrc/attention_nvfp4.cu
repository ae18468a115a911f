// Attention over the paged NVFP4 key/value cache, few query rows a sequence.
//
//   o[r] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q[r] . k_j),
//   lse[r] = log sum_j p_j,  over the positions j <= pos[b] + i
//
// for the rows r = (i, query head of the group) of a sequence b and a KV head:
// the G = Hq / Hkv query heads of each of the sequence's new tokens share every
// key and value that is read.  A row that sees nothing gives zeros, lse -inf.
//
// Work is cut stream-K: the 32-token tiles of all (sequence, KV head) items, one
// after another, in equal ranges, one a warp, so ragged lengths balance by
// themselves (an item counts kItemCost tiles more than it has, about what its
// start and end cost).  A warp whose range holds a whole item writes its
// result; the pieces of an item that crosses ranges go to the workspace (at
// most two a warp) and a second kernel joins them, in the items' order, so
// results do not depend on timing.
//
// A tile's codes and scales come by asynchronous copies into the warp's own ring
// of kStages tiles, two tiles ahead and on into the next item, and from there
// to the lanes that feed them to the tensor core (m16n8k16, f16 operands, fp32
// sums); no warp waits for another.  With 16 keys (16 tokens x D) as the A operand
// a score tile is [16 tokens x 8 rows]; its exponentials, as f16 and transposed by
// one matrix-move per 8 tokens, are the B operand of O^T += V^T P^T.  The products code x block scale are exact in f16 (at most
// 6 significant bits, 2^-10 .. 2688).  The query enters as f16 after a power
// of two a row that brings its largest value into [2^14, 2^15), exact for every
// value within 2^-29 of that; the head's global scales multiply the scores and
// the output.
// Softmax statistics are fp32, sums taken before p is rounded to f16.  A row's
// running reference m starts 7 below the first tile's largest score (base 2)
// and is only moved when some score exceeds it by 15, so p = 2^(s - m) stays
// within f16, the row's largest p is at least 2^7, and a p keeps f16's full 11
// bits down to 2^-21 of that (an absolute 2^-32 of it below).
//
// Bound by memory, at the ends by latency.  64 sequences of 2048..4096 tokens, 8
// heads of 128, 4 query heads each: 47 us for 199 MB (4.2 TB/s; 29 us at the copy
// rate).  Between its ends the kernel streams 6.3 TB/s; 4 us pass before the first
// loads (the ranges have to be found), the warps' ends lie 8 us apart, and the join
// and the launches take 8.  Rows share the conversion of codes: per token and head
// 8 and 16 rows cost about the same, 32 twice that (registers: 8 warps an SM).
#include <algorithm>

#include "attention_nvfp4.cuh"
#include "tc.cuh"

namespace qrr {

using namespace attn4;

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// CTAs an SM, by registers: with 4 the 128 of a lane are too few for D = 128 (64
// sequences of 2048..4096 tokens: 46 us with 3, 50 with 4; D = 64: 42 and 41);
// 16 rows with 3 spill (32 sequences of 1..9 new tokens: 78 us, 69 with 2)
constexpr int ctas_per_sm(int d, int nt) { return nt >= 2 ? 2 : d == 128 ? 3 : 4; }
constexpr int kTok = 32;      // tokens of a tile
constexpr int kMinTiles = 4;  // tiles of a range
constexpr int kItemCost = 1;
constexpr int kStages = 3;    // tiles of a warp's ring

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// `W` 32-bit words, a halfword and a byte from shared memory.
template <int W>
struct Words {
  uint32_t w[W];
  __device__ __forceinline__ void load(uint32_t at) {
    if constexpr (W == 4)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
    else if constexpr (W == 2) asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
    else asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
  }
};
__device__ __forceinline__ uint32_t load_u16(uint32_t at) {
  uint16_t x;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ uint32_t load_u8(uint32_t at) {
  uint32_t x;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}

// (a & m) | (b & ~m)
__device__ __forceinline__ uint32_t choose(uint32_t a, uint32_t b, uint32_t m) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(r) : "r"(a), "r"(b), "r"(m));
  return r;
}

// A tile in a warp's ring: two halves of 16 rows each of key codes, value codes,
// key scales, value scales.  Keys' rows 4..7 and 12..15 of a half change places,
// and (D = 128) values' rows 2, 3, 6, 7, ... have their halves swapped, so that
// the lanes of a read find their bytes in different banks.
template <int D>
struct Raw {
  uint8_t k[2][8 * D], v[2][8 * D], ks[2][D], vs[2][D];
};

// A half tile's operands in a lane's registers.  Lane (g, c) = (lane / 4,
// lane % 4) holds, of tokens tau and tau + 8 with tau = g / 2 + 4 (g % 2), the
// keys' values [D / 4 c, D / 4 (c + 1)), and of tokens c, c + 4, c + 8, c + 12
// the values' [D / 8 g, D / 8 (g + 1)): the order of tokens and of values that
// the two MMAs sum over is free, so each lane takes contiguous bytes.
template <int D>
struct Places {  // of a lane's bytes in the ring's first tile
  uint32_t k, ks, v, vs;
  __device__ __forceinline__ Places(const Raw<D>* ring, int lane) {
    const int g = lane >> 2, c = lane & 3, tau = (g >> 1) + 4 * (g & 1), at = tau ^ (D == 128 ? tau >> 2 : 2 * (tau >> 2));
    k = smem_u32(ring->k) + at * (D / 2) + c * (D / 8);
    ks = smem_u32(ring->ks) + tau * (D / 16) + c * (D / 64);
    v = smem_u32(ring->v) + c * (D / 2) + ((g * (D / 16)) ^ (D == 128 ? 16 * (c & 2) : 0));
    vs = smem_u32(ring->vs) + c * (D / 16) + (D == 128 ? g : g >> 1);
  }
};

template <int D>
struct Keys {
  Words<D / 32> k[2];
  uint32_t s[2];
  __device__ __forceinline__ void load(uint32_t at, uint32_t at_s, int half) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      k[i].load(at + half * 8 * D + 8 * i * (D / 2));
      if constexpr (D == 128) s[i] = load_u16(at_s + half * D + 8 * i * (D / 16));
      else s[i] = load_u8(at_s + half * D + 8 * i * (D / 16));
    }
  }
};

template <int D>
struct Values {
  Words<D / 64> v[4];
  uint32_t s[4];
  __device__ __forceinline__ void load(uint32_t at, uint32_t at_s, int half) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j].load(at + half * 8 * D + 4 * j * (D / 2));
      s[j] = load_u8(at_s + half * D + 4 * j * (D / 16));
    }
  }
};

struct Item : Seq {
  int b, h;   // sequence, KV head
  int tiles;  // that its last row sees
  int width;  // that it counts for (none: it has more rows than this kernel takes, or sees nothing)
};

// Sequence b's items.  `pad`: whole ranges of kMinTiles each.
__device__ __forceinline__ void seq_item(const Params& p, int b, bool pad, Item& it) {
  static_cast<Seq&>(it) = seq_of(p, b);
  it.b = b;
  it.tiles = (it.last + kTok) / kTok;
  const int64_t rows = static_cast<int64_t>(it.n) * p.G;
  const bool here = rows > 0 && rows <= kFewRows && it.last >= 0;
  it.width = !here ? 0 : pad ? (it.tiles + kMinTiles - 1) / kMinTiles * kMinTiles : it.tiles + kItemCost;
}

// The walk over the items of a range: tiles [t0, stop) of one at a time, and
// [t0, t1) as they count.
struct Walk : Item {
  int t0, t1, stop;
  int64_t left;  // of the range, from t0 on
  __device__ __forceinline__ void cut() {
    t1 = static_cast<int>(min(static_cast<int64_t>(width), t0 + left));
    stop = min(t1, tiles);
  }
  // whether the piece has tiles (an item's end may count for more than it has)
  __device__ __forceinline__ bool empty() const { return t0 >= tiles; }
  __device__ __forceinline__ void begin(const Params& p, int b_, int64_t off, bool pad, int64_t left_) {
    seq_item(p, b_, pad, *this);
    h = static_cast<int>(off / width);
    t0 = static_cast<int>(off - static_cast<int64_t>(h) * width);
    left = left_;
    cut();
  }
  __device__ __forceinline__ bool next(const Params& p, bool pad) {
    left -= t1 - t0;
    if (left <= 0) return false;
    t0 = 0;
    if (++h == p.c.Hkv) {
      int at = b;
      do seq_item(p, ++at, pad, *this);
      while (width == 0 && at + 1 < p.c.B);
      h = 0;
    }
    cut();
    return true;
  }
};

// The copies of a range's tiles into the warp's ring, kStages - 1 ahead of their
// use.  Inside a page the addresses only advance; the table's next entry is read
// a page ahead.  (Pages of 16 tokens: two to a tile.)
template <int D>
struct Feed {
  Walk w;
  const uint8_t *kp, *vp, *sp;  // the lane's bytes of the next tile (scales: keys' in the lower half of the warp)
  int64_t to_half, to_half_s;   // from the codes and scales of the tile's first half to its second's
  const int32_t* entry;         // the table's entry behind the tile's page
  uint32_t to, to_v, to_s;      // places in the ring's first tile
  int t, next_pg, next_half;
  bool more;
  // the page (two pages of 16) of the tile that `entry` belongs to
  __device__ __forceinline__ void read_page(const Params& p, int tile) {
    if (tile >= w.stop) return;
    next_pg = __ldg(entry);
    if (p.c.page_shift < 5 && kTok * tile + 16 <= w.last) next_half = __ldg(entry + 1);
  }
  // addresses of tile t, in the page that was read
  __device__ __forceinline__ void enter_page(const Params& p, int lane) {
    uint32_t now = static_cast<uint32_t>(next_pg), half = static_cast<uint32_t>(next_half);
    const int sh = p.c.page_shift, mask = sh >= 5 ? (1 << (sh - 5)) - 1 : 0;
    entry += sh >= 5 ? 1 : 2;
    read_page(p, (t | mask) + 1);
    const uint32_t pages = static_cast<uint32_t>(p.c.num_pages);
    if (now >= pages || (sh < 5 && half >= pages)) {
      flag(p.status, QRR_DEV_BAD_INDEX);
      now = half = 0u;
    }
    const uint32_t row = ((now * p.c.Hkv + w.h) << sh) + static_cast<uint32_t>(t & mask) * kTok;
    if (sh < 5) {
      const int64_t rows = (static_cast<int64_t>(half) - now) * p.c.Hkv * 16;
      to_half = rows * (D / 2);
      to_half_s = rows * (D / 16);
    }
    kp = p.c.kc + lane * 16 + static_cast<uint64_t>(row) * (D / 2);
    vp = p.c.vc + lane * 16 + static_cast<uint64_t>(row) * (D / 2);
    sp = (lane < 16 ? p.c.ks : p.c.vs) + (lane & 15) * (D / 16) + static_cast<uint64_t>(row) * (D / 16);
  }
  // the first tile at or after t, over the ends of items
  __device__ __forceinline__ void settle(const Params& p, bool pad, int lane) {
    while (more && t >= w.stop) {
      more = w.next(p, pad);
      t = w.t0;
    }
    if (more) {
      entry = p.c.table + static_cast<int64_t>(w.b) * p.c.max_pages + ((kTok * t) >> p.c.page_shift);
      next_half = 0;
      read_page(p, t);
      enter_page(p, lane);
    }
  }
  __device__ __forceinline__ void begin(const Params& p, const Walk& from, const Raw<D>* ring, int lane, bool pad) {
    constexpr int kChunks = D / 32;  // of 16 bytes a row
    const int r = lane / kChunks, c = lane % kChunks;
    to = smem_u32(ring) + (r ^ ((D == 128 ? 1 : 2) * (r >> 2 & 1))) * (D / 2) + c * 16;
    to_v = smem_u32(ring->v) + r * (D / 2) + ((c * 16) ^ (D == 128 ? 16 * (r & 2) : 0));
    to_s = smem_u32(lane < 16 ? ring->ks : ring->vs) + (lane & 15) * (D / 16);
    w = from;
    t = w.t0;
    to_half = 8 * D;
    to_half_s = D;
    more = true;
    settle(p, pad, lane);
  }
  // the next tile into the ring's tile `so` bytes from its first
  __device__ __forceinline__ void issue(const Params& p, bool pad, uint32_t so, int lane) {
    if (more) {
      const uint32_t a = to + so, b = to_v + so, c = to_s + so;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t *k = h ? kp + to_half : kp, *v = h ? vp + to_half : vp, *s = h ? sp + to_half_s : sp;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(a + (8 * D * h + 512 * i)), "l"(k + 512 * i) : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(b + (8 * D * h + 512 * i)), "l"(v + 512 * i) : "memory");
        }
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(c + D * h), "l"(s), "n"(D / 16) : "memory");
      }
      ++t;
      kp += 16 * D;
      vp += 16 * D;
      sp += 2 * D;
      if (t >= w.stop) settle(p, pad, lane);
      else if (((kTok * t) & ((1 << p.c.page_shift) - 1) & -kTok) == 0 || p.c.page_shift < 5) enter_page(p, lane);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
};

// A warp's rows and running state; NT groups of 8 rows.  Lane (g, c) feeds the
// query of row g of a group to the MMAs and holds the results of rows 2 c and
// 2 c + 1.  The query is in registers, that of four groups in shared memory.
template <int NT>
constexpr bool kQInSmem = NT > 2;
template <int D, int NT>
struct State {
  uint4 q[kQInSmem<NT> ? 1 : NT][D / 32];
  uint32_t qs;  // shared memory: the lane's 16 bytes of [NT][D / 32][32 lanes]
  float f[NT][2];    // score factor of the lane's two rows (log2 units)
  int lim[NT][2];    // their last visible position, before the piece's end
  float m[NT][2], l[NT][2];
  float o[NT][D / 16][4];
};

template <int D, int NT>
__device__ __forceinline__ void load_rows(const Params& p, const Item& it, int end, int lane, State<D, NT>& s) {
  const int g = lane >> 2, c = lane & 3;
  const float kg = p.c.kg ? __ldg(p.c.kg + it.h) : 1.0f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 8 * nt + g;
    const bool in = r < it.n * p.G;
    uint32_t w[D / 8] = {};
    uint32_t mx = 0u;
    if (in) {
      const uint16_t* src = p.q + (it.first + p.byG.div(r)) * p.ld_q + static_cast<int64_t>(it.h * p.G + p.byG.mod(r)) * D + c * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(src) + i);
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        mx = max(mx, absmax_bits8(x));
      }
    }
    mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
    if (mx >= 0x7F80u) flag(p.status, QRR_DEV_NONFINITE);
    const int e = query_exp(mx);
    const Pow2Scaler sc(e);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      uint32_t y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = f16x2(sc(bf16_lo(w[4 * j + i])), sc(bf16_hi(w[4 * j + i])));
      if constexpr (kQInSmem<NT>)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(s.qs + 512 * (nt * (D / 32) + j)), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
      else s.q[nt][j] = make_uint4(y[0], y[1], y[2], y[3]);
    }
    // at least the smallest normal value: a masked score times it stays -inf
    const float f = fmaxf(p.scale * kLog2e * kg * ldexpf(1.0f, e), 1.17549435e-38f);
    const int lim = in ? min(min(it.pos + p.byG.div(r), it.last), end - 1) : -1;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      s.f[nt][x] = __shfl_sync(0xFFFFFFFFu, f, 4 * (2 * c + x));
      s.lim[nt][x] = __shfl_sync(0xFFFFFFFFu, lim, 4 * (2 * c + x));
      s.m[nt][x] = kNone;
      s.l[nt][x] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) s.o[nt][j][i] = 0.0f;
  }
}

// One tile, of whose tokens `live` exist (kTok or more: all).  `all`: every row
// sees every token of it.
template <int D, int NT>
__device__ __forceinline__ void step(const Places<D>& at, uint32_t so, int t, int live, bool all, int lane, State<D, NT>& s) {
  const int g = lane >> 2, c = lane & 3;
  // four groups: a half tile at a time, for its registers
  constexpr int H = NT > 2 ? 1 : 2;
#pragma unroll 1
  for (int h0 = 0; h0 < 2; h0 += H) {
    float e[H][NT][4];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      Keys<D> x;
      x.load(at.k + so, at.ks + so, h0 + h);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) e[h][nt][i] = 0.0f;
      const uint32_t s0 = e4m3x2_to_f16x2(x.s[0]), s1 = e4m3x2_to_f16x2(x.s[1]);
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const uint32_t sel = w < 2 ? 0x1010u : 0x3232u;  // D = 64: both words in the lane's one block
        const uint32_t f0 = __byte_perm(s0, s0, sel), f1 = __byte_perm(s1, s1, sel);
        uint32_t a[4], b[4];
        f16x2x4_from_e2m1x8(x.k[0].w[w], a);
        f16x2x4_from_e2m1x8(x.k[1].w[w], b);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = hmul2(a[i], f0), b[i] = hmul2(b[i], f1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint4 y;
          if constexpr (kQInSmem<NT>)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w) : "r"(s.qs + 512 * (nt * (D / 32) + w)));
          else y = s.q[nt][w];
          mma16816(e[h][nt], a[0], b[0], a[1], b[1], y.x, y.y);
          mma16816(e[h][nt], a[2], b[2], a[3], b[3], y.z, y.w);
        }
      }
    }
    // lane's scores: rows 2 c, 2 c + 1 of each group; tokens tau, tau + 8 of each
    // half
    const int tok = kTok * t + 16 * h0 + (g >> 1) + 4 * (g & 1);
    if (!all)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (tok + 16 * h + 8 * (i >> 1) > s.lim[nt][i & 1]) e[h][nt][i] = -INFINITY;
    float top[NT][2], most = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        top[nt][i] = H == 2 ? fmaxf(max3(e[0][nt][i], e[0][nt][i + 2], e[H - 1][nt][i]), e[H - 1][nt][i + 2]) : fmaxf(e[0][nt][i], e[0][nt][i + 2]);
      most = max3(most, fmaf(top[nt][0], s.f[nt][0], -s.m[nt][0]), fmaf(top[nt][1], s.f[nt][1], -s.m[nt][1]));
    }
    if (__any_sync(0xFFFFFFFFu, most > kRoom)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v = top[nt][i];
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
          const float m = fmaxf(v * s.f[nt][i] - kLift, s.m[nt][i]), a = ex2(s.m[nt][i] - m);
          s.m[nt][i] = m;
          s.l[nt][i] *= a;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) s.o[nt][j][i] *= a, s.o[nt][j][i + 2] *= a;
        }
    }
    uint32_t p[H][NT][2];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) e[h][nt][i] = ex2(fmaf(e[h][nt][i], s.f[nt][i & 1], -s.m[nt][i & 1]));
        s.l[nt][0] += e[h][nt][0] + e[h][nt][2];
        s.l[nt][1] += e[h][nt][1] + e[h][nt][3];
        p[h][nt][0] = movmatrix(f16x2(e[h][nt][0], e[h][nt][1]));
        p[h][nt][1] = movmatrix(f16x2(e[h][nt][2], e[h][nt][3]));
      }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      Values<D> x;
      x.load(at.v + so, at.vs + so, h0 + h);
      // the two pairs' scales; those of tokens that do not exist count as zero (what
      // lies there may be anything, a NaN among it)
      uint32_t v01 = __byte_perm(x.s[0], x.s[1], 0x7740), v23 = __byte_perm(x.s[2], x.s[3], 0x7740);
      if (live < kTok) {
        const int n = live - 16 * (h0 + h) - c;
        v01 &= (n > 0 ? 0xFFu : 0u) | (n > 4 ? 0xFF00u : 0u);
        v23 &= (n > 8 ? 0xFFu : 0u) | (n > 12 ? 0xFF00u : 0u);
      }
      const uint32_t f0 = e4m3x2_to_f16x2(v01), f1 = e4m3x2_to_f16x2(v23);
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {
        // bytes of (first, second) token's codes of one value: even values, odd values
        uint32_t a[4], b[4], d[4], u[4];
        f16x2x4_from_e2m1x8(choose(x.v[0].w[w], x.v[1].w[w] << 4, 0x0F0F0F0Fu), a);
        f16x2x4_from_e2m1x8(choose(x.v[0].w[w] >> 4, x.v[1].w[w], 0x0F0F0F0Fu), b);
        f16x2x4_from_e2m1x8(choose(x.v[2].w[w], x.v[3].w[w] << 4, 0x0F0F0F0Fu), d);
        f16x2x4_from_e2m1x8(choose(x.v[2].w[w] >> 4, x.v[3].w[w], 0x0F0F0F0Fu), u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = hmul2(a[i], f0), b[i] = hmul2(b[i], f0), d[i] = hmul2(d[i], f1), u[i] = hmul2(u[i], f1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(s.o[nt][4 * w + i], a[i], b[i], d[i], u[i], p[h][nt][0], p[h][nt][1]);
        }
      }
    }
  }
}

// A piece of an item: its tiles, and the rows' results or a piece of them.  RT:
// rows of a piece in the workspace.
template <int D, int NT, int RT>
__device__ __forceinline__ void piece(const Params& p, const Walk& it, Feed<D>& feed, const Places<D>& at, bool pad, int range,
                                      int64_t per, uint32_t qs, uint32_t& so, uint32_t& free, int lane) {
  const int c = lane & 3, g = lane >> 2;
  State<D, NT> s;
  s.qs = qs;
  load_rows<D, NT>(p, it, kTok * it.stop, lane, s);
  // tiles before this one are seen whole by every row (rows behind the last one
  // are never read: no mask for them)
  const int whole = (min(it.pos, it.last) + 1) / kTok;
#pragma unroll 1
  for (int t = it.t0; t < it.stop; ++t) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();  // the tile is there for all lanes, and the one before it read by all
    feed.issue(p, pad, free, lane);
    step<D, NT>(at, so, t, it.last + 1 - kTok * t, t < whole, lane, s);
    free = so;
    so = so == (kStages - 1) * sizeof(Raw<D>) ? 0 : so + static_cast<uint32_t>(sizeof(Raw<D>));
  }
  // ---- the rows' results, or a piece of them
  if (it.empty()) return;
  const bool cut0 = it.t0 > 0, cut1 = it.t1 < it.tiles;
  const int64_t piece = static_cast<int64_t>(2 * range + (cut0 ? 0 : 1)) * RT;
  const float vg = p.c.vg ? __ldg(p.c.vg + it.h) : 1.0f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 8 * nt + 2 * c + i;
      float l = s.l[nt][i];
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
      if (r >= it.n * p.G) continue;
      if (!cut0 && !cut1) {
        const float inv = row_factor(vg, l);
        const int64_t orow = out_row(p, it.first, it.h, r);
        uint32_t w[D / 16];
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(s.o[nt][j][i] * inv, s.o[nt][j][i + 2] * inv);
          w[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
          reinterpret_cast<uint4*>(p.out + orow * D + D / 8 * g)[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        if (p.lse && g == 0) p.lse[orow] = row_lse(s.m[nt][i], l);
      } else {
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          reinterpret_cast<float4*>(p.po + (piece + r) * D + D / 8 * g)[j] =
              make_float4(s.o[nt][2 * j][i], s.o[nt][2 * j][i + 2], s.o[nt][2 * j + 1][i], s.o[nt][2 * j + 1][i + 2]);
        if (g == 0) p.pm[piece + r] = s.m[nt][i], p.pl[piece + r] = l;
      }
    }
  if (!cut0 && lane == 0)
    p.rec[static_cast<int64_t>(it.b) * p.c.Hkv + it.h] =
        Record{cut1 ? 1 + static_cast<int>((it.tiles - it.t1 + per - 1) / per) : 0, range, 0, it.h, it.first, it.n};
}

}  // namespace

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, NT)) attn_nvfp4_kernel(const Params p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Raw<D>* const ring = reinterpret_cast<Raw<D>*>(smem_raw) + kStages * (threadIdx.x >> 5);  // the warp's
  __shared__ int64_t sums[2][kWarps], at_off[kWarps];
  __shared__ int at_b[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();

  // sequences without work here; of one that sees nothing a CTA writes the rows
  const int B = p.c.B;
  for (int b = blockIdx.x; b < B; b += gridDim.x) {
    Item q;
    seq_item(p, b, false, q);
    if (q.width > 0) continue;
    for (int i = tid; i < p.c.Hkv; i += kThreads) p.rec[static_cast<int64_t>(b) * p.c.Hkv + i].pieces = 0;
    if (static_cast<int64_t>(q.n) * p.G > kFewRows) continue;
    const int64_t row = static_cast<int64_t>(q.first) * p.Hq;
    for (int i = tid; i < q.n * p.Hq * (D / 8); i += kThreads) reinterpret_cast<uint4*>(p.out + row * D)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse)
      for (int i = tid; i < q.n * p.Hq; i += kThreads) p.lse[row + i] = -INFINITY;
  }

  // ---- the warps' ranges of the tile sequence
  const int ranges = gridDim.x * kWarps, strip = (B + kThreads - 1) / kThreads;
  const int b0 = min(tid * strip, B), b1 = min(b0 + strip, B);
  int64_t sum = 0, padded = 0;
  for (int b = b0; b < b1; ++b) {
    Item it;
    seq_item(p, b, false, it);
    sum += it.width;
    if (it.width > 0) padded += (it.tiles + kMinTiles - 1) / kMinTiles * kMinTiles;
  }
  sum *= p.c.Hkv;
  padded *= p.c.Hkv;
  int64_t total = padded;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  if (lane == 0) sums[0][warp] = total;
  __syncthreads();
  total = 0;
  for (int w = 0; w < kWarps; ++w) total += sums[0][w];
  // little work: every item in whole ranges, so that none is cut where it need
  // not be
  const bool pad = total <= static_cast<int64_t>(ranges) * kMinTiles;
  const int64_t own = pad ? padded : sum;
  int64_t incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sums[1][warp] = incl;
  __syncthreads();
  total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) incl += sums[1][w];
    total += sums[1][w];
  }
  const int64_t per = pad ? kMinTiles : (total + ranges - 1) / ranges;
  for (int w = 0; w < kWarps; ++w) {
    const int64_t begin = (static_cast<int64_t>(blockIdx.x) * kWarps + w) * per;
    if (begin >= incl - own && begin < incl) {
      int64_t off = begin - (incl - own);
      for (int b = b0; b < b1; ++b) {
        Item it;
        seq_item(p, b, pad, it);
        const int64_t all = static_cast<int64_t>(it.width) * p.c.Hkv;
        if (off < all) {
          at_b[w] = b;
          at_off[w] = off;
          break;
        }
        off -= all;
      }
    }
  }
  __syncthreads();
  const int range = blockIdx.x * kWarps + warp;
  const int64_t left = min(per, total - range * per);
  if (left <= 0) return;

  Walk it;
  it.begin(p, at_b[warp], at_off[warp], pad, left);
  Feed<D> feed;
  feed.begin(p, it, ring, lane, pad);
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) feed.issue(p, pad, i * static_cast<uint32_t>(sizeof(Raw<D>)), lane);
  const Places<D> at(ring, lane);
  const uint32_t qs = smem_u32(smem_raw) + sizeof(Raw<D>) * kStages * kWarps + (warp * NT * (D / 32) * 32 + lane) * 16;
  // the ring's tile in use, and the one before it: that is filled next
  uint32_t so = 0, free = (kStages - 1) * static_cast<uint32_t>(sizeof(Raw<D>));
  do {
    if (NT <= 2 || it.n * p.G > 16) piece<D, NT, 8 * NT>(p, it, feed, at, pad, range, per, qs, so, free, lane);
    else piece<D, 2, 8 * NT>(p, it, feed, at, pad, range, per, qs, so, free, lane);
  } while (it.next(p, pad));
  asm volatile("cp.async.wait_all;" ::: "memory");
}

namespace {

// Joins items of a few pieces each: a warp a row.  The lanes take the pieces'
// (m, l), 32 at a time; sums over them are formed in the order of the pieces'
// lanes, the outputs' in the order of the pieces.  RT: rows of a piece.
template <int D, int RT>
__global__ void __launch_bounds__(256) join_rows_kernel(const Params p) {
  constexpr int V = D / 32;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
  const Record rec = p.rec[blockIdx.x];
  const int row = rec.rt * RT + r;
  if (rec.pieces == 0 || row >= rec.n * p.G) return;
  const float vg = p.c.vg ? __ldg(p.c.vg + rec.h) : 1.0f;
  float m = kNone, l = 0.0f, o[V] = {};
  for (int i0 = 0; i0 < rec.pieces; i0 += 32) {
    const int n = min(32, rec.pieces - i0);
    float mi = kNone, li = 0.0f, old;
    if (lane < n) {
      mi = p.pm[piece_row(rec, i0 + lane, RT) + r];
      li = p.pl[piece_row(rec, i0 + lane, RT) + r];
    }
    const float a = piece_weight(mi, li, m, l, old);
#pragma unroll
    for (int d = 0; d < V; ++d) o[d] *= old;
    // `many` pieces' outputs from the i-th on; eight loads under way at a time
    // where there are as many
    auto add = [&](auto many, int i) {
      constexpr int kMany = decltype(many)::value;
      float v[kMany][V];
#pragma unroll
      for (int u = 0; u < kMany; ++u) {
        const float* src = p.po + (piece_row(rec, i0 + min(i + u, n - 1), RT) + r) * D + V * lane;
        if constexpr (V == 4) {
          const float4 x = *reinterpret_cast<const float4*>(src);
          v[u][0] = x.x, v[u][1] = x.y, v[u][2] = x.z, v[u][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(src);
          v[u][0] = x.x, v[u][1] = x.y;
        }
      }
#pragma unroll
      for (int u = 0; u < kMany; ++u) {
        const float ai = __shfl_sync(0xFFFFFFFFu, a, (i + u) & 31);  // 0 behind the last piece
#pragma unroll
        for (int d = 0; d < V; ++d) o[d] += ai * v[u][d];
      }
    };
    int i = 0;
    for (; i + 8 <= n; i += 8) add(std::integral_constant<int, 8>{}, i);
    for (; i < n; i += 2) add(std::integral_constant<int, 2>{}, i);
  }
  const float inv = row_factor(vg, l);
  const int64_t orow = out_row(p, rec.first, rec.h, row);
  uint32_t y[V / 2];
#pragma unroll
  for (int d = 0; d < V / 2; ++d) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * d] * inv, o[2 * d + 1] * inv);
    y[d] = *reinterpret_cast<const uint32_t*>(&b);
  }
  if constexpr (V == 4) *reinterpret_cast<uint2*>(p.out + orow * D + V * lane) = make_uint2(y[0], y[1]);
  else *reinterpret_cast<uint32_t*>(p.out + orow * D + V * lane) = y[0];
  if (p.lse && lane == 0) p.lse[orow] = row_lse(m, l);
}

// Joins items of many pieces each (long sequences, few of them): a warp takes a quarter of a row's
// values (row blockIdx.y of items 2 blockIdx.x and the next); groups of D / 16 lanes
// take the pieces in turn, so a batch of 32 pieces' loads is under way at once.
// Every sum has a fixed order.
template <int D, int RT>
__global__ void __launch_bounds__(256) join_pieces_kernel(const Params p) {
  constexpr int kLanes = D / 16, kGroups = 32 / kLanes;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp & 3, grp = lane / kLanes, row = blockIdx.y;
  const int64_t item = 2 * static_cast<int64_t>(blockIdx.x) + (warp >> 2);
  if (item >= static_cast<int64_t>(p.c.B) * p.c.Hkv) return;
  const Record rec = p.rec[item];
  if (rec.pieces == 0 || row >= rec.n * p.G) return;
  const float vg = p.c.vg ? __ldg(p.c.vg + rec.h) : 1.0f;
  const float* const po = p.po + part * (D / 4) + 4 * (lane % kLanes);
  float m = kNone, l = 0.0f, o[4] = {};
  for (int i0 = 0; i0 < rec.pieces; i0 += 32) {
    const int n = min(32, rec.pieces - i0);
    float mi = kNone, li = 0.0f, old;
    if (lane < n) {
      mi = p.pm[piece_row(rec, i0 + lane, RT) + row];
      li = p.pl[piece_row(rec, i0 + lane, RT) + row];
    }
    // kGroups x `many` pieces
    auto add = [&](auto many) {
      constexpr int kMany = decltype(many)::value;
      float4 x[kMany];
#pragma unroll
      for (int u = 0; u < kMany; ++u)
        x[u] = *reinterpret_cast<const float4*>(po + (piece_row(rec, i0 + min(kGroups * u + grp, n - 1), RT) + row) * D);
      const float a = piece_weight(mi, li, m, l, old);
#pragma unroll
      for (int d = 0; d < 4; ++d) o[d] *= old;
#pragma unroll
      for (int u = 0; u < kMany; ++u) {
        const float ai = __shfl_sync(0xFFFFFFFFu, a, kGroups * u + grp);  // 0 behind the last piece
        o[0] += ai * x[u].x, o[1] += ai * x[u].y, o[2] += ai * x[u].z, o[3] += ai * x[u].w;
      }
    };
    if (n <= kGroups) add(std::integral_constant<int, 1>{});
    else add(std::integral_constant<int, kLanes>{});
  }
#pragma unroll
  for (int y = kLanes; y < 32; y <<= 1)
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] += __shfl_xor_sync(0xFFFFFFFFu, o[d], y);
  const int64_t orow = out_row(p, rec.first, rec.h, row);
  if (grp == 0)
    *reinterpret_cast<uint2*>(p.out + orow * D + part * (D / 4) + 4 * lane) = bf16x4(o, row_factor(vg, l));
  if (p.lse && part == 0 && lane == 0) p.lse[orow] = row_lse(m, l);
}

template <int D, int NT>
cudaError_t launch(const AttnNvfp4Args& a, int dev, int grid, cudaStream_t stream) {
  constexpr int RT = 8 * NT;
  const int ranges = grid * kWarps, rows = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(a.max_new) * (a.Hq / a.c.Hkv), RT));
  const int64_t items = static_cast<int64_t>(a.c.B) * a.c.Hkv;
  const Params p = make_params(a, a.ws, ranges, RT, items);
  constexpr int smem = (static_cast<int>(sizeof(Raw<D>)) * kStages + (kQInSmem<NT> ? NT * D * 16 : 0)) * kWarps;
  static OncePerDevice limit;
  cudaError_t e = limit(dev, [] { return cudaFuncSetAttribute(attn_nvfp4_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  attn_nvfp4_kernel<D, NT><<<grid, kThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  // no sequence may have rows (the kernel has told those that do), or a cache whose
  // longest sequence fits a range, and a range for every item: nothing is cut
  if (e != cudaSuccess || rows == 0 || (a.c.capacity() <= kMinTiles * kTok && items <= ranges)) return e;
  // Eight pieces an item on average, or more: 8 sequences of 20000..33000 tokens
  // join in 6 us by pieces, in 12 by rows; 64 of 2048..4096 (4 pieces) in 7.7 and 5.8.
  if (ranges >= 8 * items)
    return launch_dependent(join_pieces_kernel<D, RT>, dim3(static_cast<unsigned>((items + 1) / 2), rows), 256, 0, stream, p);
  return launch_dependent(join_rows_kernel<D, RT>, dim3(static_cast<unsigned>(items), NT), 256, 0, stream, p);
}

// Whether some sequence may have few rows, or many (see kFewRows).
bool any_few(int G) { return G <= kFewRows; }
bool any_many(int64_t max_new, int G) { return max_new * G > kFewRows; }

// Groups of 8 rows that this kernel is launched for.
int row_groups(int64_t max_new, int G) { return max_new * G <= 8 ? 1 : max_new * G <= 16 ? 2 : 4; }

size_t few_ws_bytes(int D, int64_t items, int64_t max_new, int G) {
  const int nt = row_groups(max_new, G);
  return any_few(G) ? ws_bytes(D, kMaxSms * ctas_per_sm(D, nt) * kWarps, 8 * nt, items) : 0;
}

}  // namespace

size_t attention_nvfp4_ws_bytes(int D, int B, int Hq, int Hkv, int64_t max_new) {
  const int G = Hq / Hkv;
  return few_ws_bytes(D, static_cast<int64_t>(B) * Hkv, max_new, G) + (any_many(max_new, G) ? attention_nvfp4_tc_ws_bytes(D) : 0);
}

cudaError_t launch_attention_nvfp4(const AttnNvfp4Args& a, cudaStream_t stream) {
  if (a.r.T == 0 || a.Hq == 0 || a.c.B == 0) return cudaSuccess;
  int dev = 0, sms = kSMs;
  cudaError_t e = device_of(dev, sms);
  if (e != cudaSuccess) return e;
  const int G = a.Hq / a.c.Hkv;
  if (any_few(G)) {
    const int nt = row_groups(a.max_new, G), grid = (sms < kMaxSms ? sms : kMaxSms) * ctas_per_sm(a.c.D, nt);
    e = a.c.D == 128 ? (nt == 1   ? launch<128, 1>(a, dev, grid, stream)
                        : nt == 2 ? launch<128, 2>(a, dev, grid, stream)
                                  : launch<128, 4>(a, dev, grid, stream))
                     : (nt == 1   ? launch<64, 1>(a, dev, grid, stream)
                        : nt == 2 ? launch<64, 2>(a, dev, grid, stream)
                                  : launch<64, 4>(a, dev, grid, stream));
    if (e != cudaSuccess) return e;
  }
  if (!any_many(a.max_new, G)) return cudaSuccess;
  uint8_t* const ws = a.ws + few_ws_bytes(a.c.D, static_cast<int64_t>(a.c.B) * a.c.Hkv, a.max_new, G);
  return launch_attention_nvfp4_tc(a, ws, any_few(G), stream);
}

}  // namespace qrr
