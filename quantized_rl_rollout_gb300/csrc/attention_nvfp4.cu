// Attention over the paged NVFP4 key/value cache, few query rows a sequence.
//
//   o[r] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q[r] . k_j),
//   lse[r] = log sum_j p_j,  over the positions j <= pos[b] + i
//
// for the rows r = (i, query head of the group) of a sequence b and a KV head:
// the G = Hq / Hkv query heads of each of the sequence's new tokens share every
// key and value that is read.  A row that sees nothing gives zeros, lse -inf.
//
// Work is cut stream-K: the 16-token tiles of all (sequence, row tile, KV head)
// items, one after another, in equal ranges, one a CTA, so ragged lengths
// balance by themselves.  A CTA whose range holds a whole item writes its
// result; the pieces of an item that crosses ranges go to the workspace (at
// most two a CTA) and a second kernel joins them, in the items' order, so
// results do not depend on timing.
//
// Inside a CTA the warps take tiles in turn, each on its own: a tile's codes
// and scales come from global memory straight into the registers of the lanes
// that feed them to the tensor core (m16n8k16, f16 operands, fp32 sums), so
// there is no shared memory and no barrier in the loop.  With K (16 tokens x
// D) as the A operand the score tile is [16 tokens x 8 rows]; its exponentials,
// as f16 and transposed by one matrix-move per 8 tokens, are the B operand of
// O^T += V^T P^T.  The products code x block scale are exact in f16 (at most
// 6 significant bits, 2^-10 .. 2688).  The query enters as f16 after a power
// of two a row that brings its largest value into [2^14, 2^15), exact for every
// value within 2^-29 of that; the head's global scales multiply the scores and
// the output.
// Softmax statistics are fp32, sums taken before p is rounded to f16.  A row's
// running reference m starts 7 below the first tile's largest score (base 2)
// and is only moved when some score exceeds it by 15, so p = 2^(s - m) stays
// within f16, the row's largest p is at least 2^7, and a p keeps f16's full 11
// bits down to 2^-21 of that (an absolute 2^-32 of it below).
#include "attention_nvfp4.cuh"
#include "tc.cuh"

namespace qrr {

using namespace attn4;

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kCtasPerSm = 4;
constexpr int kMinTiles = 8;  // tiles of a range: two a warp

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

template <int W>
struct Words {
  uint32_t w[W];
};

template <int W>
__device__ __forceinline__ Words<W> load_words(const uint8_t* p) {
  Words<W> r;
  if constexpr (W == 4) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
    r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
  } else if constexpr (W == 2) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    r.w[0] = x.x, r.w[1] = x.y;
  } else {
    r.w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
  return r;
}

// One tile's operands in a lane's registers.  Lane (g, c) = (lane / 4,
// lane % 4) holds, of tokens tau and tau + 8 with tau = g / 2 + 4 (g % 2), the
// keys' values [D / 4 c, D / 4 (c + 1)), and of tokens c, c + 4, c + 8, c + 12
// the values' [D / 8 g, D / 8 (g + 1)): the order of tokens and of values that
// the two MMAs sum over is free, so each lane takes contiguous bytes.
template <int D>
struct Tile {
  Words<D / 32> k[2];
  Words<D / 64> v[4];
  uint32_t ks[2], vs[4];
  int live;  // tokens of the tile that exist (0..16)
};

struct Item : Seq {
  int b, rt, h;  // sequence, row tile, KV head
  int tiles;     // tiles of the item (at least 1)
};

// Sequence b's row tiles (none if it has more rows than this kernel takes).
template <int RT>
__device__ __forceinline__ void seq_item(const Params& p, int b, Item& it, int& rts) {
  static_cast<Seq&>(it) = seq_of(p, b);
  it.tiles = max(1, (it.last + 16) >> 4);
  const int64_t rows = static_cast<int64_t>(it.n) * p.G;
  rts = rows > kFewRows ? 0 : static_cast<int>((rows + RT - 1) / RT);
}

template <int D>
__device__ __forceinline__ void load_tile(const Params& p, const int32_t* table, int h, int t, int last, int lane,
                                          Tile<D>& x) {
  const int g = lane >> 2, c = lane & 3;
  const int tok = 16 * t;
  int pg = __ldg(table + (tok >> p.c.page_shift));
  x.live = min(16, last + 1 - tok);
  if (pg < 0 || pg >= p.c.num_pages) {
    flag(p.status, QRR_DEV_BAD_INDEX);
    x.live = 0;
  }
  if (x.live <= 0) {
    x = Tile<D>{};
    return;
  }
  const int64_t row = kv_row(p.c, pg, h, tok & ((1 << p.c.page_shift) - 1));
  const int tau = (g >> 1) + 4 * (g & 1);
  const uint8_t* kc = p.c.kc + (row + tau) * (D / 2) + c * (D / 8);
  const uint8_t* ks = p.c.ks + (row + tau) * (D / 16) + c * (D / 64);
  const uint8_t* vc = p.c.vc + (row + c) * (D / 2) + g * (D / 16);
  const uint8_t* vs = p.c.vs + (row + c) * (D / 16) + (D == 128 ? g : g >> 1);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x.k[i] = load_words<D / 32>(kc + i * 8 * (D / 2));
    if constexpr (D == 128) x.ks[i] = __ldg(reinterpret_cast<const uint16_t*>(ks + i * 8 * (D / 16)));
    else x.ks[i] = __ldg(ks + i * 8 * (D / 16));
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x.v[j] = load_words<D / 64>(vc + j * 4 * (D / 2));
    x.vs[j] = __ldg(vs + j * 4 * (D / 16));
  }
}

// A warp's rows and running state; NT groups of 8 rows.  Lane (g, c) feeds the
// query of row g of a group to the MMAs and holds the results of rows 2 c and
// 2 c + 1.
template <int D, int NT>
struct State {
  uint32_t q[NT][D / 16][2];
  float f[NT][2];    // score factor of the lane's two rows (log2 units)
  int lim[NT][2];    // their last visible position
  float m[NT][2], l[NT][2];
  float o[NT][D / 16][4];
};

template <int D, int NT>
__device__ __forceinline__ void load_rows(const Params& p, const Item& it, int lane, State<D, NT>& s) {
  const int g = lane >> 2, c = lane & 3;
  const float kg = p.c.kg ? __ldg(p.c.kg + it.h) : 1.0f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = it.rt * 8 * NT + 8 * nt + g;
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
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) s.q[nt][j][i] = f16x2(sc(bf16_lo(w[2 * j + i])), sc(bf16_hi(w[2 * j + i])));
    const float f = p.scale * kLog2e * kg * ldexpf(1.0f, e);
    const int lim = in ? min(it.pos + p.byG.div(r), it.last) : -1;
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

// One tile of 16 tokens.  `all`: every row sees every token of it.
template <int D, int NT>
__device__ __forceinline__ void step(const Tile<D>& x, int t, bool all, int lane, State<D, NT>& s) {
  const int g = lane >> 2, c = lane & 3;
  float sc[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[nt][i] = 0.0f;
  {
    const uint32_t s0 = e4m3x2_to_f16x2(x.ks[0]), s1 = e4m3x2_to_f16x2(x.ks[1]);
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
        mma16816(sc[nt], a[0], b[0], a[1], b[1], s.q[nt][2 * w][0], s.q[nt][2 * w][1]);
        mma16816(sc[nt], a[2], b[2], a[3], b[3], s.q[nt][2 * w + 1][0], s.q[nt][2 * w + 1][1]);
      }
    }
  }
  // lane's scores: rows 2 c, 2 c + 1 of each group; tokens tau, tau + 8
  const int tok = 16 * t + (g >> 1) + 4 * (g & 1);
  bool over = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sc[nt][i] *= s.f[nt][i & 1];
      if (!all && (i < 2 ? tok : tok + 8) > s.lim[nt][i & 1]) sc[nt][i] = -INFINITY;
      over |= sc[nt][i] > s.m[nt][i & 1] + kRoom;
    }
  if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = fmaxf(sc[nt][i], sc[nt][i + 2]);
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
        const float m = fmaxf(v - kLift, s.m[nt][i]), a = ex2(s.m[nt][i] - m);
        s.m[nt][i] = m;
        s.l[nt][i] *= a;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) s.o[nt][j][i] *= a, s.o[nt][j][i + 2] *= a;
      }
  }
  uint32_t p[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = ex2(sc[nt][i] - s.m[nt][i & 1]);
    s.l[nt][0] += e[0] + e[2];
    s.l[nt][1] += e[1] + e[3];
    p[nt][0] = movmatrix(f16x2(e[0], e[1]));
    p[nt][1] = movmatrix(f16x2(e[2], e[3]));
  }
  uint32_t vs[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) vs[j] = c + 4 * j < x.live ? x.vs[j] : 0u;  // what no token wrote may hold a NaN
  const uint32_t f0 = e4m3x2_to_f16x2(vs[0] | vs[1] << 8), f1 = e4m3x2_to_f16x2(vs[2] | vs[3] << 8);
#pragma unroll
  for (int w = 0; w < D / 64; ++w) {
    // bytes of (first, second) token's codes of one value: even values, odd values
    uint32_t a[4], b[4], d[4], e[4];
    f16x2x4_from_e2m1x8((x.v[0].w[w] & 0x0F0F0F0Fu) | (x.v[1].w[w] << 4 & 0xF0F0F0F0u), a);
    f16x2x4_from_e2m1x8((x.v[0].w[w] >> 4 & 0x0F0F0F0Fu) | (x.v[1].w[w] & 0xF0F0F0F0u), b);
    f16x2x4_from_e2m1x8((x.v[2].w[w] & 0x0F0F0F0Fu) | (x.v[3].w[w] << 4 & 0xF0F0F0F0u), d);
    f16x2x4_from_e2m1x8((x.v[2].w[w] >> 4 & 0x0F0F0F0Fu) | (x.v[3].w[w] & 0xF0F0F0F0u), e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = hmul2(a[i], f0), b[i] = hmul2(b[i], f0), d[i] = hmul2(d[i], f1), e[i] = hmul2(e[i], f1);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma16816(s.o[nt][4 * w + i], a[i], b[i], d[i], e[i], p[nt][0], p[nt][1]);
    }
  }
}

}  // namespace

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? kCtasPerSm : 2) attn_nvfp4_kernel(const Params p) {
  constexpr int RT = 8 * NT;
  __shared__ float so[kWarps][RT][D + 4];
  __shared__ float sm[kWarps][RT], sl[kWarps][RT];
  __shared__ int64_t scan[2][kWarps];
  __shared__ int64_t at_off;
  __shared__ int at_b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- this CTA's range of the tile sequence
  const int B = p.c.B, strip = (B + kThreads - 1) / kThreads;
  const int b0 = min(tid * strip, B), b1 = min(b0 + strip, B);
  int64_t sum = 0, padded = 0;
  for (int b = b0; b < b1; ++b) {
    Item it;
    int rts;
    seq_item<RT>(p, b, it, rts);
    const int64_t items = static_cast<int64_t>(rts) * p.c.Hkv;
    sum += items * it.tiles;
    padded += items * ((it.tiles + kMinTiles - 1) / kMinTiles * kMinTiles);
  }
  int64_t total_padded = padded;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) total_padded += __shfl_xor_sync(0xFFFFFFFFu, total_padded, o);
  if (lane == 0) scan[0][warp] = total_padded;
  __syncthreads();
  total_padded = 0;
  for (int w = 0; w < kWarps; ++w) total_padded += scan[0][w];
  // little work: every item padded to whole ranges of kMinTiles, so that none
  // is cut where it need not be
  const bool pad = total_padded <= static_cast<int64_t>(gridDim.x) * kMinTiles;
  const int64_t own = pad ? padded : sum;
  int64_t incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan[1][warp] = incl;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) incl += scan[1][w];
    total += scan[1][w];
  }
  const int64_t per = pad ? kMinTiles : (total + gridDim.x - 1) / gridDim.x;
  const int64_t begin = blockIdx.x * per, end = min(begin + per, total);
  Record rec{};
  if (begin >= end) {
    if (tid == 0) p.rec[blockIdx.x] = rec;
    return;
  }
  auto width = [&](const Item& it) { return pad ? (it.tiles + kMinTiles - 1) / kMinTiles * kMinTiles : it.tiles; };
  if (begin >= incl - own && begin < incl) {
    int64_t off = begin - (incl - own);
    for (int b = b0; b < b1; ++b) {
      Item it;
      int rts;
      seq_item<RT>(p, b, it, rts);
      const int64_t w = static_cast<int64_t>(rts) * p.c.Hkv * width(it);
      if (off < w) {
        at_b = b;
        at_off = off;
        break;
      }
      off -= w;
    }
  }
  __syncthreads();

  Item it;
  it.b = at_b;
  int rts;
  seq_item<RT>(p, it.b, it, rts);
  int64_t idx = at_off / width(it);  // item of the sequence: row tile, head
  int t0 = static_cast<int>(at_off % width(it));
  State<D, NT> s;
  for (int64_t left = end - begin; left > 0;) {
    it.rt = static_cast<int>(idx / p.c.Hkv);
    it.h = static_cast<int>(idx % p.c.Hkv);
    const int w = width(it), t1 = static_cast<int>(min(static_cast<int64_t>(w), t0 + left));
    load_rows<D, NT>(p, it, lane, s);
    // what the rows of this tile see at most, and at least (rows behind the
    // last one are never read again: they need no mask)
    const int r_end = min((it.rt + 1) * RT, it.n * p.G);
    const int see = min(it.pos + p.byG.div(r_end - 1), it.last);
    const int sure = min(it.pos + p.byG.div(it.rt * RT), it.last);
    const int stop = min(t1, (see + 16) >> 4);
    const int32_t* table = p.c.table + static_cast<int64_t>(it.b) * p.c.max_pages;
    Tile<D> x, y;
    int t = t0 + warp;
    if (t < stop) load_tile<D>(p, table, it.h, t, see, lane, x);
    while (t < stop) {
      if (t + kWarps < stop) load_tile<D>(p, table, it.h, t + kWarps, see, lane, y);
      step<D, NT>(x, t, x.live == 16 && 16 * t + 15 <= sure, lane, s);
      x = y;
      t += kWarps;
    }
    // ---- join the warps
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * nt + 2 * c + i;
        float l = s.l[nt][i];
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
        if (g == 0) {
          sm[warp][r] = s.m[nt][i];
          sl[warp][r] = l;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
          *reinterpret_cast<float2*>(&so[warp][r][D / 8 * g + 2 * j]) = make_float2(s.o[nt][j][i], s.o[nt][j][i + 2]);
      }
    __syncthreads();
    const bool cut0 = t0 > 0, cut1 = t1 < w;
    const int piece = 2 * blockIdx.x + (cut0 ? 0 : 1);
    const float vg = p.c.vg ? __ldg(p.c.vg + it.h) : 1.0f;
    for (int e = tid; e < RT * (D / 4); e += kThreads) {
      const int r = e / (D / 4), d = 4 * (e % (D / 4));
      const int row = it.rt * RT + r;
      if (row >= it.n * p.G) break;
      float m = kNone;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) m = fmaxf(m, sm[k][r]);
      float l = 0.0f, o[4] = {};
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float a = ex2(sm[k][r] - m);
        l += a * sl[k][r];
        const float4 v = *reinterpret_cast<const float4*>(&so[k][r][d]);
        o[0] += a * v.x, o[1] += a * v.y, o[2] += a * v.z, o[3] += a * v.w;
      }
      if (!cut0 && !cut1) {
        const float inv = l > 0.0f ? __fdividef(vg, l) : 0.0f;
        const int64_t orow = out_row(p, it.first, it.h, row);
        const __nv_bfloat162 u = __floats2bfloat162_rn(o[0] * inv, o[1] * inv), v = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
        *reinterpret_cast<uint2*>(p.out + orow * D + d) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
        if (p.lse && d == 0) p.lse[orow] = l > 0.0f ? (m + lg2(l)) * kLn2 : -INFINITY;
      } else {
        const int64_t pr = static_cast<int64_t>(piece) * RT + r;
        *reinterpret_cast<float4*>(p.po + pr * D + d) = make_float4(o[0], o[1], o[2], o[3]);
        if (d == 0) p.pm[pr] = m, p.pl[pr] = l;
      }
    }
    if (cut0) rec.cont = 1, rec.cont_more = cut1;
    else if (cut1) rec.start = 1, rec.rt = it.rt, rec.h = it.h, rec.first = it.first, rec.n = it.n;
    __syncthreads();
    left -= t1 - t0;
    t0 = 0;
    if (left > 0 && ++idx == static_cast<int64_t>(rts) * p.c.Hkv) {
      idx = 0;
      do seq_item<RT>(p, ++it.b, it, rts);
      while (rts == 0 && it.b + 1 < B);
    }
  }
  if (tid == 0) p.rec[blockIdx.x] = rec;
}

namespace {

template <int D, int NT>
cudaError_t launch(const AttnNvfp4Args& a, int grid, cudaStream_t stream) {
  constexpr int RT = 8 * NT;
  const Params p = make_params(a, a.ws, grid, RT);
  attn_nvfp4_kernel<D, NT><<<grid, kThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  join_kernel<D, RT><<<dim3(grid, NT), 256, 0, stream>>>(p, grid);
  return cudaGetLastError();
}

// Whether some sequence may have few rows, or many (see kFewRows).
bool any_few(int G) { return G <= kFewRows; }
bool any_many(int64_t max_new, int G) { return max_new * G > kFewRows; }

size_t few_ws_bytes(int D) { return ws_bytes(D, kMaxSms * kCtasPerSm, kFewRows); }

}  // namespace

size_t attention_nvfp4_ws_bytes(int D, int64_t, int, int Hq, int Hkv, int64_t max_new) {
  const int G = Hq / Hkv;
  return few_ws_bytes(D) + (any_many(max_new, G) ? attention_nvfp4_tc_ws_bytes(D) : 0);
}

cudaError_t launch_attention_nvfp4(const AttnNvfp4Args& a, cudaStream_t stream) {
  if (a.r.T == 0 || a.Hq == 0 || a.c.B == 0) return cudaSuccess;
  int dev = 0, sms = kSMs;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int G = a.Hq / a.c.Hkv;
  if (any_few(G)) {
    const bool one = static_cast<int64_t>(a.max_new) * G <= 8;
    const int grid = (sms < kMaxSms ? sms : kMaxSms) * (one ? kCtasPerSm : 2);
    const cudaError_t e = a.c.D == 128 ? (one ? launch<128, 1>(a, grid, stream) : launch<128, 2>(a, grid, stream))
                                       : (one ? launch<64, 1>(a, grid, stream) : launch<64, 2>(a, grid, stream));
    if (e != cudaSuccess) return e;
  }
  return any_many(a.max_new, G) ? launch_attention_nvfp4_tc(a, a.ws + few_ws_bytes(a.c.D), stream) : cudaSuccess;
}

}  // namespace qrr
