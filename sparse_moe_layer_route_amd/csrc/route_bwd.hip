// Gradient of the router: from the gradients of the slot weights (moe_route's
// topk_w) and, added to them, of the logits, to the logits, the hidden states
// and the router's weights.
//   unnormalised weights w_j = p_{e_j}, p = softmax(l):
//     c = sum_v G_v p_v,          dl_v = p_v (G_v - c)
//   renormalised, q_v = exp(l_v - m) / sum_u n_u exp(l_u - m):
//     c = sum_v G_v q_v,          dl_v = q_v (G_v - n_v c)
//   with G_v the sum of dtopk_w over the slots of expert v and n_v their number
//   (0 or 1 for moe_route's ids; an expert named twice counts twice).
//   dx = dx_add + dl W_r,  dW_r = dl^T x.
//
// Launches: up to 64 tokens one (route_few_kernel); else the logits' gradient
// (route_dlogits_kernel), both products in one grid (route_products_kernel), and,
// when dW is cut into ranges of tokens, the sum of the ranges.  The products read
// x once and write dx once, which bounds them (E <= 64: 4 E flops for four bytes
// of bf16).
//
// bf16 layers run v_mfma_f32_16x16x32_bf16 on x and W as they are; dl is fp32
// and goes in as bf16 parts whose sum it is: three for dW (fp32 out, what is
// left out is 2^-24 of dl), two for dx (2^-16, against an output step of
// 2^-8).  The parts are written by the first launch as whole operand
// fragments.  Both operands want eight consecutive k (tokens for dW, experts
// for dx) in a lane, while x and W are contiguous along H: a lane loads eight
// columns of eight rows (16 bytes each; 16 lanes cover two 128-byte lines) and
// interleaves them in registers into the fragments of as many column tiles.
// fp32 layers run v_mfma_f32_16x16x4_f32, whose operands are single values.
//
// bf16, 16384 x 3584, 64 experts (246 MB, 45.5 us at the rate of a large copy):
// 73 us, of which 8 the logits' gradient, 61 the products, 5 the sum of the
// ranges.  With a launch each dW's products take 35 us (117 MB of x read at 3.4
// TB/s), dx's 27 (as much written at 4.3): side by side they gain nothing.  That is
// no bound of the memory, which does both at 5.4 in a copy, but of the waits in
// the two loops (see route_dw and route_dx).
#include <algorithm>
#include <type_traits>

#include "common.h"

namespace moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int RBWD_THREADS = 512;  // of the logits' gradient
constexpr int PROD_THREADS = 256;  // of the products
constexpr int PROD_WAVES = PROD_THREADS / MOE_WAVE;
constexpr int RBWD_STEP = 32;   // tokens of one dW step (the K of one bf16 MFMA)
// Column tiles of 16 a wave owns (H % 64 == 0: the last wave of a bf16 row may
// own 64 columns past the end, which it neither keeps nor stores).
template <typename T> constexpr int rbwd_nc() { return sizeof(T) == 2 ? 8 : 4; }
constexpr int DW_GROUP = PROD_WAVES;  // steps a bf16 dW block takes at once: each wave loads one
constexpr int RBWD_DW_PARTS = 3, RBWD_DX_PARTS = 2;

// Shapes of one call.  mt: 16-expert tiles, ks: 32-expert k steps of dx.
struct RouteBwdPlan {
  int mt, ks, steps, ncg;
  int per, splits;         // steps of a token range of dW, ranges
  int dx_tiles;            // 16-token tiles of one dx wave
  bool apart;              // dW and dx in launches of their own
  size_t fx, fw, part, total;  // workspace offsets: dx and dW fragments (fp32 layers: padded
                               // dlogits at fx), dW partials
  size_t up_to;                // bytes enough for any smaller T too
};

// Blocks of the products that an XCD holds at once: two a CU.
constexpr int RBWD_XCD_BLOCKS = 64;
// One dW block a CU: more ranges cost more partials than they gain (bf16 dW of
// 16384 x 3584: 45 us with 9 ranges, 48 with 18).
constexpr int RBWD_DW_BLOCKS = 256;
// fp32 products are bound by the matrix units.  From this many on dW and dx have a
// launch each (8192 x 3584, 64 experts: 96 us for the call, 119 in one launch; 2048
// x 2048, 64 experts: 25.6, 26.8, 40 experts: 23.1, 22.4).
constexpr int64_t RBWD_APART = 1 << 28;

static RouteBwdPlan route_bwd_plan(const moe_dims_t& d, int T) {
  RouteBwdPlan p{};
  p.mt = (d.n_experts + 15) / 16;
  p.ks = (p.mt + 1) / 2;
  p.steps = (T + RBWD_STEP - 1) / RBWD_STEP;
  const int cols = d.dtype == MOE_BF16 ? 16 * rbwd_nc<bf16>() : 16 * rbwd_nc<float>();
  p.ncg = (d.hidden + cols - 1) / cols;
  // Ranges of whole groups of steps (fp32: two steps for each set of its block's
  // waves at least), and one range where there are two groups: it spares the launch
  // that adds the ranges (256 x 2048, 64 experts: 9.4 us, 10.2 with two; 902 x 64, 27
  // experts: 9.0 with ranges of one group, 10.4 with two).
  const int most = std::max(1, RBWD_DW_BLOCKS / p.ncg);
  const int unit = d.dtype == MOE_BF16 ? DW_GROUP : p.mt > 1 ? PROD_WAVES : 2 * PROD_WAVES;
  const int even = (p.steps + most - 1) / most;
  const bool one = d.dtype == MOE_BF16 && p.steps <= 2 * DW_GROUP;
  p.per = one ? p.steps : (even + unit - 1) / unit * unit;
  p.splits = (p.steps + p.per - 1) / p.per;
  const int tiles = 2 * p.steps;
  p.apart = d.dtype == MOE_F32 && (int64_t)T * d.hidden * (16 * p.mt) >= RBWD_APART;
  // A dx wave takes as many token tiles as leave all blocks a place beside dW's, half
  // the places at least: one more an XCD waits for a place to the end (bf16, 16384 x
  // 3584, 64 experts: 74 us for the call with 252 blocks beside 252 of dW, 83 with 259;
  // 4096 x 1536, 40 experts: 19.6 with 258 beside 192, 20.5 with 192, 21.4 with 384).
  const int dw_places = (p.splits * p.ncg + 7) / 8;
  const int places =
      p.apart ? RBWD_XCD_BLOCKS / 2 : std::max(RBWD_XCD_BLOCKS / 2, RBWD_XCD_BLOCKS - dw_places);
  const int ranges = std::max(1, 8 * places * PROD_WAVES / p.ncg);
  p.dx_tiles = (tiles + ranges - 1) / ranges;
  size_t o = 0;
  auto take = [&](size_t n) {
    const size_t at = o;
    o = (o + n + 255) & ~(size_t)255;
    return at;
  };
  if (d.dtype == MOE_BF16) {
    p.fx = take((size_t)tiles * p.ks * RBWD_DX_PARTS * 1024);
    p.fw = take((size_t)p.steps * p.mt * RBWD_DW_PARTS * 1024);
  } else {
    p.fx = take((size_t)p.steps * RBWD_STEP * p.mt * 16 * 4);
  }
  // fewer tokens may have more ranges, up to one a unit of steps
  const size_t partial = (size_t)d.n_experts * d.hidden * 4;
  const int units = one ? 1 : std::min(most, (p.steps + unit - 1) / unit);
  p.up_to = o + (units > 1 ? units * partial : 0);
  if (p.splits > 1) p.part = take(p.splits * partial);
  p.total = o;
  return p;
}

// Reductions and broadcasts within rows of 16 lanes (one token each).
template <int CTRL> __device__ __forceinline__ float row_move(float v) {
  const int x = __float_as_int(v);
  return __int_as_float(dpp_move<CTRL, 0xf, false>(x, x));
}
__device__ __forceinline__ float row_sum(float v) {
  v += row_move<0xB1>(v);   // quad_perm 1,0,3,2
  v += row_move<0x4E>(v);   // quad_perm 2,3,0,1
  v += row_move<0x141>(v);  // row_half_mirror
  return v + row_move<0x140>(v);  // row_mirror
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, row_move<0xB1>(v));
  v = fmaxf(v, row_move<0x4E>(v));
  v = fmaxf(v, row_move<0x141>(v));
  return fmaxf(v, row_move<0x140>(v));
}

struct DlogitsArgs {
  int T, E, k, renorm;
  const int32_t* ids;
  const float *logits, *dtopk_w;
  const float* add;  // may be dlogits itself
  float* dlogits;
};
typedef float rbwd_tile_t[RBWD_STEP][MOE_MAX_EXPERTS + 1];

// dl of token t by 16 lanes: lane l holds experts l + 16 q (q < Q, E <= 16 Q) and
// slot l's id and gradient.  Tokens past T get the last one's.  No branch on a lane's expert or
// slot: selects only, so that all loads of a token go out together (64 x 64: 8.7
// us with branches, 3.9 without, a launch and a chain of short steps).
template <int Q>
__device__ __forceinline__ void token_dlogits(const DlogitsArgs& a, int t, float (&dl)[Q]) {
  const int l = threadIdx.x & 15, E = a.E, k = a.k;
  const bool renorm = a.renorm;
  const int64_t tc = min(t, a.T - 1);
#pragma unroll
  for (int q = 0; q < Q; ++q) dl[q] = a.add ? a.add[tc * E + min(l + 16 * q, E - 1)] : 0.f;
  if (a.dtopk_w) {
    float v[Q], G[Q], n[Q];
    bool part[Q];
    const int64_t o = tc * k + min(l, k - 1);
    const int id = l < k ? a.ids[o] : -1;  // slots past k match no expert
    const float g = a.dtopk_w[o];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      v[q] = a.logits[tc * E + min(l + 16 * q, E - 1)];
      G[q] = n[q] = 0.f;
    }
    // slot J's id and gradient come from lane J of the token's row
    auto slot = [&](auto J) {
      constexpr int j = decltype(J)::value;
      const int e = dpp_move<0x150 + j, 0xf, false>(id, id) - l;  // row_newbcast
      const float gj = row_move<0x150 + j>(g);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        G[q] += e == 16 * q ? gj : 0.f;
        n[q] += e == 16 * q ? 1.f : 0.f;
      }
    };
    slot(std::integral_constant<int, 0>{});
    slot(std::integral_constant<int, 1>{});
    slot(std::integral_constant<int, 2>{});
    slot(std::integral_constant<int, 3>{});
    slot(std::integral_constant<int, 4>{});
    slot(std::integral_constant<int, 5>{});
    slot(std::integral_constant<int, 6>{});
    slot(std::integral_constant<int, 7>{});
    float m = -__builtin_inff(), s = 0.f, c = 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      part[q] = l + 16 * q < E && (!renorm || n[q] > 0.f);
      m = fmaxf(m, part[q] ? v[q] : -__builtin_inff());
    }
    m = row_max(m);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      v[q] = part[q] ? expf(v[q] - m) : 0.f;
      s += renorm ? n[q] * v[q] : v[q];
    }
    s = row_sum(s);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      v[q] = part[q] ? v[q] / s : 0.f;
      c += part[q] && n[q] > 0.f ? G[q] * v[q] : 0.f;
    }
    c = row_sum(c);
#pragma unroll
    for (int q = 0; q < Q; ++q)
      dl[q] += part[q] ? v[q] * (G[q] - (renorm ? n[q] : 1.f) * c) : 0.f;
  }
}
// Token t's row of dlogits (store), of a tile of 32 tokens and of pad (or null).
template <int Q>
__device__ __forceinline__ void put_dlogits(const DlogitsArgs& a, int t, const float (&dl)[Q],
                                            bool store, rbwd_tile_t& tile, int mt, float* pad) {
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int e = (threadIdx.x & 15) + 16 * q;
    const bool on = e < a.E && t < a.T;
    if (on && store) a.dlogits[(int64_t)t * a.E + e] = dl[q];
    if (pad && q < mt) pad[(int64_t)t * (16 * mt) + e] = on ? dl[q] : 0.f;
    tile[t % RBWD_STEP][e] = on ? dl[q] : 0.f;
  }
}
// A finite value past the largest bf16 would round to infinity: that largest, and
// the next parts hold the rest.
__device__ __forceinline__ float bf16_finite(float v) {
  constexpr float MOST = 0x1.FEp127f;
  return fabsf(v) > MOST && fabsf(v) < __builtin_inff() ? copysignf(MOST, v) : v;
}
// The fragments of a tile, fx and fw each where not null:
//   fx [16-token tile][k step][part][lane]: token lane % 16, experts
//     32 s + 8 (lane / 16) .. +7 (zero past T and E),
//   fw [expert tile][part][lane]: expert lane % 16, tokens 8 (lane / 16) .. +7.
// The parts of a value are it rounded to bf16, what is left rounded, and so on
// (a value that is not finite leaves NaN).
template <int KS>
__device__ __forceinline__ void pack_dlogits(const rbwd_tile_t& tile, int mt, uint4* fx,
                                             uint4* fw) {
  // one thread per fragment slot, all of its parts
  const int nx = fx ? 2 * KS * 64 : 0, nw = fw ? mt * 64 : 0;
  for (int i = threadIdx.x; i < nx + nw; i += RBWD_THREADS) {
    const bool to_x = i < nx;
    const int l16 = i & 15, g8 = 8 * ((i >> 4) & 3), f = (to_x ? i : i - nx) >> 6;
    const int half = f / KS, st = f % KS;
    const float* src = to_x ? &tile[16 * half + l16][32 * st + g8] : &tile[g8][16 * f + l16];
    const int step = to_x ? 1 : MOE_MAX_EXPERTS + 1;
    float v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = src[c * step];
    const int parts = to_x ? RBWD_DX_PARTS : RBWD_DW_PARTS;
    uint4* dst = to_x ? fx + f * RBWD_DX_PARTS * 64 : fw + f * RBWD_DW_PARTS * 64;
#pragma unroll
    for (int p = 0; p < RBWD_DW_PARTS; ++p) {
      uint32_t w[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        w[c] = p == 0 ? f2_to_bf16x2(bf16_finite(v[2 * c]), bf16_finite(v[2 * c + 1]))
                      : f2_to_bf16x2(v[2 * c], v[2 * c + 1]);
        v[2 * c] -= bf16_lo(w[c]);
        v[2 * c + 1] -= bf16_hi(w[c]);
      }
      if (p < parts) dst[p * 64 + (i & 63)] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// One block per 32 tokens.  pad (fp32 layers, else null): dlogits again as [32
// steps][16 mt], zero past T and E.  fx / fw (bf16 layers, else null): the
// fragments of all steps in turn.  16384 x 64: 7.9 us, of 8 MB read and 14 written.
template <int KS>
__global__ void __launch_bounds__(RBWD_THREADS)
route_dlogits_kernel(DlogitsArgs a, int mt, float* __restrict__ pad,
                     uint4* __restrict__ fx, uint4* __restrict__ fw) {
  static_assert(RBWD_THREADS == 16 * RBWD_STEP, "16 lanes a token");
  __shared__ rbwd_tile_t tile;
  const int t = blockIdx.x * RBWD_STEP + (threadIdx.x >> 4);
  float dl[2 * KS];  // the fragments of dx take whole k steps of 32 experts
  token_dlogits(a, t, dl);
  put_dlogits(a, t, dl, true, tile, mt, pad);
  if (!fx && !fw) return;
  __syncthreads();
  pack_dlogits<KS>(tile, mt,
                   fx ? fx + (int64_t)blockIdx.x * 2 * KS * RBWD_DX_PARTS * 64 : nullptr,
                   fw ? fw + (int64_t)blockIdx.x * mt * RBWD_DW_PARTS * 64 : nullptr);
}

// Eight columns of eight rows -> fragment c: column c, the eight rows in k
// order.
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ bf16x8_t column_frag(const uint4 (&v)[8], int c) {
  const uint32_t sel = (c & 1) ? 0x07060302u : 0x05040100u;
  const int w = c >> 1;
  uint4 o;
  o.x = __builtin_amdgcn_perm(word_of(v[1], w), word_of(v[0], w), sel);
  o.y = __builtin_amdgcn_perm(word_of(v[3], w), word_of(v[2], w), sel);
  o.z = __builtin_amdgcn_perm(word_of(v[5], w), word_of(v[4], w), sel);
  o.w = __builtin_amdgcn_perm(word_of(v[7], w), word_of(v[6], w), sel);
  return __builtin_bit_cast(bf16x8_t, o);
}

// Rows r0 + 8 (lane / 16) .. +7, eight columns each, of a matrix whose row 0 is
// at p: `off` is the lane's byte offset, 8 (lane / 16) rows and its column.  The
// rest of the address is the same for the wave and stays in scalar registers.
__device__ __forceinline__ void load_rows8(const bf16* __restrict__ p, int64_t r0, int H, uint32_t off,
                                           uint4 (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p + (r0 + i) * H) + off);
}
// The same where rows from n_rows on are zero.
__device__ __forceinline__ void load_rows8_below(const bf16* __restrict__ p, int64_t r0, int n_rows,
                                                 int H, uint32_t off, uint4 (&v)[8]) {
  const int left = n_rows - (int)r0 - 8 * (lane_id() >> 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (i < left)
      v[i] = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p + (r0 + i) * H) + off);
  }
}
__device__ __forceinline__ uint32_t rows8_off(int H, int col) {
  return (uint32_t)(8 * (lane_id() >> 4) * H + col) * 2u;
}

struct RouteBwdArgs {
  int T, H, E, ncg, steps, per, splits, dx_tiles, dw_blocks;
  const float* pad;  // fp32 layers: dlogits [32 steps][16 MT]
  const uint4 *fx, *fw;
  float *part, *dw;
  int accumulate;
};

// How the four waves of an fp32 dW block share a range of tokens: MH halves of the
// expert tiles (MW each) by WAYS interleaved sets of steps.
template <int MT> struct DwShape {
  static constexpr int MH = MT > 1 ? 2 : 1, MW = (MT + MH - 1) / MH, WAYS = PROD_WAVES / MH;
};

template <int MT>
__device__ __forceinline__ void dw_steps(const RouteBwdArgs& a, const float* __restrict__ x, int col,
                                         int m0, int r0, int way, int s1,
                                         f32x4_t (&acc)[DwShape<MT>::MW][4]) {
  constexpr int MW = DwShape<MT>::MW, WAYS = DwShape<MT>::WAYS;
  const int lane = lane_id(), n = lane & 15, g = lane >> 4;
  // the lane's byte offsets; the rest of an address is the same for the wave
  const uint32_t x_off = (uint32_t)(g * a.H + col) * 4u, p_off = (uint32_t)(g * 16 * MT + n) * 4u;
  struct Half {
    float4 v[4];
    float d[4][MW];
  } h0, h1;
  auto load = [&](Half& h, int s, int half) {
    const int t = s * RBWD_STEP + 16 * half;
    const char* px = reinterpret_cast<const char*>(x + (int64_t)t * a.H);
    const char* pp = reinterpret_cast<const char*>(a.pad + (int64_t)t * (16 * MT));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      h.v[q] = *reinterpret_cast<const float4*>(px + (int64_t)q * 16 * a.H + x_off);
#pragma unroll
      for (int m = 0; m < MW; ++m)  // past the last tile the first one's, dropped at the end
        h.d[q][m] = *reinterpret_cast<const float*>(
            pp + (4 * q * MT + (m0 + m < MT ? m0 + m : 0)) * 64 + p_off);
    }
  };
  auto mfma = [&](const Half& h) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int m = 0; m < MW; ++m) {
        acc[m][0] = __builtin_amdgcn_mfma_f32_16x16x4f32(h.d[q][m], h.v[q].x, acc[m][0], 0, 0, 0);
        acc[m][1] = __builtin_amdgcn_mfma_f32_16x16x4f32(h.d[q][m], h.v[q].y, acc[m][1], 0, 0, 0);
        acc[m][2] = __builtin_amdgcn_mfma_f32_16x16x4f32(h.d[q][m], h.v[q].z, acc[m][2], 0, 0, 0);
        acc[m][3] = __builtin_amdgcn_mfma_f32_16x16x4f32(h.d[q][m], h.v[q].w, acc[m][3], 0, 0, 0);
      }
  };
  const int whole = a.T / RBWD_STEP;  // steps with all their rows
  const int e = min(s1, whole), s0 = r0 + way;
  if (s0 < e) {
    // half steps in turn, each asked for before the one before it is multiplied
    load(h0, s0, 0);
    for (int s = s0; s < e; s += WAYS) {
      load(h1, s, 1);
      __builtin_amdgcn_sched_barrier(0);
      mfma(h0);
      load(h0, min(s + WAYS, e - 1), 0);
      __builtin_amdgcn_sched_barrier(0);
      mfma(h1);
    }
  }
  if (whole < s1 && whole >= s0 && (whole - s0) % WAYS == 0) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int t = whole * RBWD_STEP + 16 * half + 4 * q + g;
        h0.v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < a.T) h0.v[q] = *reinterpret_cast<const float4*>(x + (int64_t)t * a.H + col);
#pragma unroll
        for (int m = 0; m < MW; ++m)
          h0.d[q][m] = a.pad[(int64_t)t * (16 * MT) + 16 * (m0 + m < MT ? m0 + m : 0) + n];
      }
      mfma(h0);
    }
  }
}

constexpr int DW_STEP_FLOATS = 8 * 64 * 4;  // of LDS: the fragments of a step's x
template <typename T, int MT>
constexpr int dw_lds_floats() {
  using S = DwShape<MT>;
  if (sizeof(T) == 2) return DW_GROUP * DW_STEP_FLOATS;
  return (S::WAYS - 1) * S::MH * 16 * S::MW * 16 * rbwd_nc<T>();
}

// dW of 128 columns over one range of tokens, bf16: the block's waves load a step
// of x each, interleave it into fragments and leave them in LDS for all four, which
// own an expert tile each (of fewer than three tiles a part of the columns), so no
// row is read or interleaved twice and a wave holds 32 accumulators.  Rows are asked
// for two groups of steps ahead and a step's fragments of dlogits as soon as the group
// before is through with theirs, which is after the rows of the group behind it: loads
// retire in order, so a group's first product waits for those rows too, and of the
// two groups asked for one is in flight.  The last step, if it is not whole, runs by itself, so
// that the loop has one way to load its rows.  1024 x 2048, 64 experts: 12.7 us for the
// call, 14.3 with the waves of a pair each loading and interleaving what both need;
// 16384 x 3584: 74.7, 74.0.  A second buffer, which spares one of the two barriers a
// group, gains nothing (12.7, 75) and halves the blocks that a CU has LDS for.
// WAVES: of the block; those from PROD_WAVES on only take part in its barriers.
template <int MT, int WAVES>
__device__ __forceinline__ void route_dw(const RouteBwdArgs& a, int item,
                                         const bf16* __restrict__ x, float* lds) {
  constexpr int TILES = MT == 3 ? 4 : MT, NC = 8 * TILES / PROD_WAVES;
  const int split = item / a.ncg, cg = item - split * a.ncg;
  const int lane = lane_id(), n = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool on = WAVES == PROD_WAVES || wv < PROD_WAVES;
  const int m = wv % TILES, c0 = wv / TILES * NC;
  const int s0 = split * a.per, s1 = min(a.steps, s0 + a.per);
  const int whole = a.T / RBWD_STEP, e = min(s1, whole);  // steps with all their rows
  const int groups = (e - s0 + DW_GROUP - 1) / DW_GROUP;
  uint4* frags = reinterpret_cast<uint4*>(lds);
  // lanes past H read the row's last columns; their results are dropped below
  const uint32_t off = rows8_off(a.H, min(cg * 128 + 8 * n, a.H - 8));
  // loads past the end ask for the last step again, unused
  auto rows = [&](int gi, uint4 (&v)[8]) {
    load_rows8(x, (int64_t)min(s0 + gi * DW_GROUP + wv, e - 1) * RBWD_STEP, a.H, off, v);
  };
  uint4 d[DW_GROUP][RBWD_DW_PARTS];
  auto parts = [&](int s, int q) {
    const uint4* at = a.fw + ((int64_t)s * MT + min(m, MT - 1)) * RBWD_DW_PARTS * 64;
    const char* src = reinterpret_cast<const char*>(at);
#pragma unroll
    for (int p = 0; p < RBWD_DW_PARTS; ++p)
      d[q][p] = *reinterpret_cast<const uint4*>(src + p * 1024 + lane * 16u);
  };
  f32x4_t acc[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) acc[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto put = [&](uint4* buf, const uint4 (&v)[8]) {
#pragma unroll
    for (int c = 0; c < 8; ++c) buf[c * 64 + lane] = __builtin_bit_cast(uint4, column_frag(v, c));
  };
  auto mfma = [&](const uint4* buf, int q) {
    bf16x8_t b[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) b[c] = __builtin_bit_cast(bf16x8_t, buf[(c0 + c) * 64 + lane]);
#pragma unroll
    for (int p = RBWD_DW_PARTS - 1; p >= 0; --p)  // smallest part first
#pragma unroll
      for (int c = 0; c < NC; ++c)
        acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, d[q][p]), b[c],
                                                         acc[c], 0, 0, 0);
  };
  uint4 v0[8], v1[8];
  auto group = [&](int gi, uint4 (&v)[8]) {
    const int s = s0 + gi * DW_GROUP;
    if (gi > 0) __syncthreads();  // all are through with the group before
    if (on && s + wv < e) put(frags + wv * 512, v);
    if (on) rows(gi + 2, v);
    // the scheduler would move the loads down to their uses
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < DW_GROUP; ++q) {
      if (s + q < e && m < MT && on) mfma(frags + q * 512, q);
      if (on) parts(min(s + DW_GROUP + q, e - 1), q);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (groups > 0) {
    if (on) {
      rows(0, v0);
#pragma unroll
      for (int q = 0; q < DW_GROUP; ++q) parts(min(s0 + q, e - 1), q);
      rows(1, v1);
    }
    for (int gi = 0; gi < groups; gi += 2) {
      group(gi, v0);
      if (gi + 1 < groups) group(gi + 1, v1);
    }
  }
  if (s0 <= whole && whole < s1) {  // the last step, not whole
    __syncthreads();
    if (on) parts(whole, 0);
    if (wv == 0) {
      load_rows8_below(x, (int64_t)whole * RBWD_STEP, a.T, a.H, off, v0);
      put(frags, v0);
    }
    __syncthreads();
    if (m < MT && on) mfma(frags, 0);
  }
  if (m >= MT || !on) return;
  const bool direct = a.splits == 1;
  float* out = direct ? a.dw : a.part + (int64_t)split * a.E * a.H;
  typedef float vec_t __attribute__((ext_vector_type(NC < 4 ? NC : 4)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 16 * m + 4 * g + i, h = cg * 128 + 8 * n + c0;
    if (e >= a.E || h >= a.H) continue;
#pragma unroll
    for (int c = 0; c < NC; c += 4) {
      vec_t* dst = reinterpret_cast<vec_t*>(out + (int64_t)e * a.H + h + c);
      vec_t v;
#pragma unroll
      for (int r = 0; r < (NC < 4 ? NC : 4); ++r) v[r] = acc[c + r][i];
      if (direct && a.accumulate) v = *dst + v;
      *dst = v;
    }
  }
}
// dW of a wave's columns over one range of tokens, fp32.  The waves of way 1 and up
// leave their tiles in LDS, those of way 0 add them in way order and store.  WAVES as
// above.
template <int MT, int WAVES>
__device__ __forceinline__ void route_dw(const RouteBwdArgs& a, int item,
                                         const float* __restrict__ x, float* lds) {
  using S = DwShape<MT>;
  constexpr int NC = rbwd_nc<float>(), COLS = 16 * NC, MW = S::MW, TILE = 16 * MW * COLS;
  const int split = item / a.ncg, cg = item - split * a.ncg;
  const int lane = lane_id(), n = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool on = WAVES == PROD_WAVES || wv < PROD_WAVES;
  const int half = wv % S::MH, way = wv / S::MH, m0 = half * MW;
  const int s0 = split * a.per, s1 = min(a.steps, s0 + a.per);
  f32x4_t acc[MW][NC];
#pragma unroll
  for (int m = 0; m < MW; ++m)
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[m][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // lanes past H read the row's last columns; their results are dropped below
  if (on) dw_steps<MT>(a, x, min(cg * COLS + NC * n, a.H - NC), m0, s0, way, s1, acc);
  auto each = [&](auto f) {
#pragma unroll
    for (int m = 0; m < MW; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < NC; c += 4)
          f(16 * m + 4 * g + i, NC * n + c,
            make_float4(acc[m][c][i], acc[m][c + 1][i], acc[m][c + 2][i], acc[m][c + 3][i]));
  };
  auto slot = [&](int w, int r, int c) {
    return reinterpret_cast<float4*>(lds + ((w - 1) * S::MH + half) * TILE + r * COLS + c);
  };
  if (on && way > 0) each([&](int r, int c, float4 v) { *slot(way, r, c) = v; });
  __syncthreads();
  if (way > 0) return;  // the waves that are not on as well
  const bool direct = a.splits == 1;
  float* out = direct ? a.dw : a.part + (int64_t)split * a.E * a.H;
  each([&](int r, int c, float4 v) {
    const int e = 16 * m0 + r, h = cg * COLS + c;
    if (e >= a.E || h >= a.H) return;
#pragma unroll
    for (int w = 1; w < S::WAYS; ++w) {
      const float4 o = *slot(w, r, c);
      v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
    }
    float4* dst = reinterpret_cast<float4*>(out + (int64_t)e * a.H + h);
    if (direct && a.accumulate) {
      const float4 o = *dst;
      v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
    }
    *dst = v;
  });
}

// dx of a wave's columns by 16-token tiles: the products are formed as
// (W^T)(dl^T), so a lane ends with rows 4 g + i of the tiles c = 0..7 for one
// token.  Operand row r takes columns 8 (r / 4) + 32 (r % 4) + c: the rows of a
// lane are four runs of eight columns, 8 g + 32 i, and each 16-byte store
// covers 64 contiguous bytes of a token with four lanes.
template <int MT>
__device__ __forceinline__ void route_dx(const RouteBwdArgs& a, int item,
                                         const bf16* __restrict__ w, const bf16* dx_add, bf16* dx) {
  constexpr int KS = (MT + 1) / 2, NF = KS * RBWD_DX_PARTS;
  const int range = item / a.ncg, cg = item - range * a.ncg;
  const int lane = lane_id(), n = lane & 15, g = lane >> 4;
  const int t0 = range * a.dx_tiles, t1 = min(2 * a.steps, t0 + a.dx_tiles);
  bf16x8_t wf[KS][8];
  const uint32_t w_off = rows8_off(a.H, min(cg * 128 + 8 * (n >> 2) + 32 * (n & 3), a.H - 8));
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    uint4 v[8];
    load_rows8_below(w, 32 * s, a.E, a.H, w_off, v);
#pragma unroll
    for (int c = 0; c < 8; ++c) wf[s][c] = column_frag(v, c);
  }
  const uint32_t off = (uint32_t)(n * a.H + 8 * g) * 2u;  // the lane's runs: 64 i bytes on
  const int runs = min(4, (a.H - cg * 128) / 32);         // 2 or 4 of them inside H
  // A tile's fragments and addend are asked for before the tile before it is
  // stored: loads and stores retire in one order.  Both are conditional, so their
  // number is not known and the wait before the second half of a tile's products
  // is for all of them, the stores of the tile before included.
  uint4 f[NF], add[4];
  auto load = [&](int tl) {
    const char* src = reinterpret_cast<const char*>(a.fx + (int64_t)tl * NF * 64);
    const uint32_t l16 = lane * 16u;
#pragma unroll
    for (int i = 0; i < NF; ++i) f[i] = *reinterpret_cast<const uint4*>(src + i * 1024 + l16);
    if (dx_add && tl * 16 + n < a.T) {
      const char* q = reinterpret_cast<const char*>(dx_add + (int64_t)tl * 16 * a.H + cg * 128);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < runs) add[i] = *reinterpret_cast<const uint4*>(q + 64 * i + off);
    }
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) add[i] = make_uint4(0u, 0u, 0u, 0u);
  load(t0);
  for (int tl = t0; tl < t1; ++tl) {
    f32x4_t acc[8];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int p = RBWD_DX_PARTS - 1; p >= 0; --p)
#pragma unroll
        for (int c = 0; c < 8; ++c)
          acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              wf[s][c], __builtin_bit_cast(bf16x8_t, f[s * RBWD_DX_PARTS + p]),
              s == 0 && p == RBWD_DX_PARTS - 1 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : acc[c], 0, 0, 0);
    if (dx_add) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          acc[2 * q][i] += bf16_lo(word_of(add[i], q));
          acc[2 * q + 1][i] += bf16_hi(word_of(add[i], q));
        }
    }
    if (tl + 1 < t1) load(tl + 1);
    if (tl * 16 + n < a.T) {
      char* q = reinterpret_cast<char*>(dx + (int64_t)tl * 16 * a.H + cg * 128);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < runs)
          *reinterpret_cast<uint4*>(q + 64 * i + off) =
              make_uint4(f2_to_bf16x2(acc[0][i], acc[1][i]), f2_to_bf16x2(acc[2][i], acc[3][i]),
                         f2_to_bf16x2(acc[4][i], acc[5][i]), f2_to_bf16x2(acc[6][i], acc[7][i]));
    }
  }
}
// fp32: k step 4q + r holds experts 16 q + 4 (lane / 16) + r on both sides, so
// a lane's four steps of one q are four consecutive experts of its token.
// Operand row r takes columns 4 (r / 4) + 16 (r % 4) + c: a lane ends with four
// runs of four, 4 g + 16 i, and each store covers 64 contiguous bytes of a
// token with four lanes.
template <int MT>
__device__ __forceinline__ void route_dx(const RouteBwdArgs& a, int item,
                                         const float* __restrict__ w, const float* dx_add,
                                         float* dx) {
  const int range = item / a.ncg, cg = item - range * a.ncg;
  const int lane = lane_id(), n = lane & 15, g = lane >> 4;
  const int t0 = range * a.dx_tiles, t1 = min(2 * a.steps, t0 + a.dx_tiles);
  float4 wf[MT][4];
#pragma unroll
  for (int q = 0; q < MT; ++q)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int e = 16 * q + 4 * g + r;
      wf[q][r] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (e < a.E)
        wf[q][r] = *reinterpret_cast<const float4*>(w + (int64_t)e * a.H + cg * 64 +
                                                    4 * (n >> 2) + 16 * (n & 3));
    }
  // A tile's loads go out before the products of the tile before it.  Loads and
  // stores retire in one order, and both are conditional: the wait for a tile is
  // for all that is out, the next tile's loads and earlier stores included.
  struct Tile {
    float4 d[MT], add[4];
  } b0, b1;
  auto load = [&](Tile& b, int tl) {
    const int64_t t = min(tl * 16 + n, a.T - 1);
#pragma unroll
    for (int q = 0; q < MT; ++q)
      b.d[q] = *reinterpret_cast<const float4*>(a.pad + (int64_t)(tl * 16 + n) * (16 * MT) +
                                                16 * q + 4 * g);
    if (dx_add) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        b.add[i] = *reinterpret_cast<const float4*>(dx_add + t * a.H + cg * 64 + 4 * g + 16 * i);
    }
  };
  auto products = [&](const Tile& b, int tl) {
    const int t = tl * 16 + n;
    f32x4_t acc[4];
#pragma unroll
    for (int q = 0; q < MT; ++q)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float4 d = b.d[q], v = wf[q][r];
        const float dv = r == 0 ? d.x : r == 1 ? d.y : r == 2 ? d.z : d.w;
        const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
        const bool first = q == 0 && r == 0;
        acc[0] = __builtin_amdgcn_mfma_f32_16x16x4f32(v.x, dv, first ? zero : acc[0], 0, 0, 0);
        acc[1] = __builtin_amdgcn_mfma_f32_16x16x4f32(v.y, dv, first ? zero : acc[1], 0, 0, 0);
        acc[2] = __builtin_amdgcn_mfma_f32_16x16x4f32(v.z, dv, first ? zero : acc[2], 0, 0, 0);
        acc[3] = __builtin_amdgcn_mfma_f32_16x16x4f32(v.w, dv, first ? zero : acc[3], 0, 0, 0);
      }
    if (t >= a.T) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float4 o = make_float4(acc[0][i], acc[1][i], acc[2][i], acc[3][i]);
      if (dx_add) {
        const float4 e = b.add[i];
        o = make_float4(o.x + e.x, o.y + e.y, o.z + e.z, o.w + e.w);
      }
      *reinterpret_cast<float4*>(dx + (int64_t)t * a.H + cg * 64 + 4 * g + 16 * i) = o;
    }
  };
  load(b0, t0);
  for (int tl = t0; tl < t1; tl += 2) {
    if (tl + 1 < t1) load(b1, tl + 1);
    __builtin_amdgcn_sched_barrier(0);
    products(b0, tl);
    if (tl + 1 >= t1) break;
    if (tl + 2 < t1) load(b0, tl + 2);
    __builtin_amdgcn_sched_barrier(0);
    products(b1, tl + 1);
  }
}

// Work items in contiguous eighths of the list per XCD (blocks go round-robin
// over the eight): the items of one token range share its fragments in L2.
__device__ __forceinline__ int xcd_item(int b, int n) {
  const int per = (n + 7) >> 3;
  return (b & 7) * per + (b >> 3);
}

// Blocks 0 .. dw_blocks-1 (rounded up to eights) form dW, the others dx: one
// launch, and a CU may hold a block of each (bf16, 4096 x 1536, 40 experts: 17.8 us
// for the whole call, 22.3 with a launch each).
template <typename T, int MT>
__global__ void __launch_bounds__(PROD_THREADS, 2)
route_products_kernel(RouteBwdArgs a, int dx_items, const T* __restrict__ x,
                      const T* __restrict__ w, const T* dx_add, T* dx) {
  __shared__ __align__(16) float lds[dw_lds_floats<T, MT>()];
  const int nw = (a.dw_blocks + 7) & ~7, b0 = blockIdx.x;
  if (b0 < nw) {
    const int item = xcd_item(b0, a.dw_blocks);
    if (item < a.dw_blocks) route_dw<MT, PROD_WAVES>(a, item, x, lds);
  } else {
    // fp32: dx first, so that dW's long waves have a SIMD to themselves early (2048
    // x 2048, 40 experts: 22.1 us for the call, 25.3 at one priority; a bf16 call
    // loses by it: 16384 x 3584 83, 74)
    if (sizeof(T) == 4) __builtin_amdgcn_s_setprio(3);
    const int nx = (dx_items + PROD_WAVES - 1) / PROD_WAVES;
    const int b = xcd_item(b0 - nw, nx);
    const int item = b * PROD_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (b < nx && item < dx_items) route_dx<MT>(a, item, w, dx_add, dx);
  }
}

// One or two steps of tokens: the products' blocks each form the gradient of all
// logits for themselves, in LDS, and the first one stores it, so that the call is
// one launch.  Not where dlogits is the addend too: other blocks read it.  bf16,
// 2048 columns, 64 experts: 32 tokens 7.0 us, 8.5 with the logits' gradient in a
// launch of its own; 64 tokens 9.0 both ways, and 2.6 us less of the caller's time.
template <typename T, int MT, int STEPS>
__global__ void __launch_bounds__(RBWD_THREADS, 2)
route_few_kernel(DlogitsArgs g, RouteBwdArgs a, int dx_items, const T* __restrict__ x,
                 const T* __restrict__ w, const T* dx_add, T* dx) {
  constexpr int KS = (MT + 1) / 2;
  constexpr int TILES = STEPS * (int)sizeof(rbwd_tile_t) / 4;
  constexpr int SUMS = sizeof(T) == 2 ? STEPS * DW_STEP_FLOATS : dw_lds_floats<T, MT>();
  constexpr int FX = 2 * KS * RBWD_DX_PARTS * 64, FW = MT * RBWD_DW_PARTS * 64;  // a step's
  constexpr int PACK = sizeof(T) == 2 ? (FX > FW ? FX : FW) : RBWD_STEP * 16 * MT / 4;
  __shared__ __align__(16) float lds[TILES > SUMS ? TILES : SUMS];  // the tiles, then dW's sums
  __shared__ uint4 packed[STEPS * PACK];
  rbwd_tile_t* tile = reinterpret_cast<rbwd_tile_t*>(lds);
  float* pad = sizeof(T) == 4 ? reinterpret_cast<float*>(packed) : nullptr;
  const bool for_dw = (int)blockIdx.x < a.dw_blocks;
  // the loads of all steps go out together
  const int t = threadIdx.x >> 4;
  float dl[STEPS][2 * KS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) token_dlogits(g, t + s * RBWD_STEP, dl[s]);
#pragma unroll
  for (int s = 0; s < STEPS; ++s)
    put_dlogits(g, t + s * RBWD_STEP, dl[s], blockIdx.x == 0, tile[s], MT, pad);
  __syncthreads();
  if (sizeof(T) == 2) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
      pack_dlogits<KS>(tile[s], MT, for_dw ? nullptr : packed + s * FX,
                       for_dw ? packed + s * FW : nullptr);
    __syncthreads();
  }
  a.pad = pad;
  a.fx = a.fw = packed;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (for_dw) {
    route_dw<MT, RBWD_THREADS / MOE_WAVE>(a, blockIdx.x, x, lds);  // all waves: it has barriers
  } else {
    const int item = (blockIdx.x - a.dw_blocks) * (RBWD_THREADS / MOE_WAVE) + wv;
    if (item < dx_items) route_dx<MT>(a, item, w, dx_add, dx);
  }
}

// dW = (dW +) the sum of the ranges' partials; splits = 0 clears dW.  R threads an
// element add a run of ranges each, in order, and the first adds the runs, in order.
template <int R>
__global__ void __launch_bounds__(PROD_THREADS)
route_dw_sum_kernel(int n4, int splits, const float4* __restrict__ part, int accumulate,
                    float4* __restrict__ dw) {
  constexpr int N = PROD_THREADS / R;
  __shared__ float4 runs[R][N];
  const int l = threadIdx.x % N, r = threadIdx.x / N, i = blockIdx.x * N + l;
  const int per = (splits + R - 1) / R, p1 = min(splits, (r + 1) * per);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (i < n4) {
    if (r == 0 && accumulate) s = dw[i];
#pragma unroll 8
    for (int p = r * per; p < p1; ++p) {
      const float4 v = part[(int64_t)p * n4 + i];
      s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
    }
  }
  if (R > 1) {
    runs[r][l] = s;
    __syncthreads();
    if (r > 0) return;
#pragma unroll
    for (int q = 1; q < R; ++q) {
      const float4 v = runs[q][l];
      s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
    }
  }
  if (i < n4) dw[i] = s;
}
// Eight threads an element from SUM_RUNS ranges on (bf16, 16384 x 64, 64 experts, 128
// ranges: 17.1 us for the call, 21.8 with one; 1515 x 64, 62 experts, 12 ranges: 11.8,
// 12.7; 4096 x 1536, 40 experts, 16 ranges: 18.6 both).
constexpr int SUM_RUNS = 8;
static hipError_t launch_dw_sum(int n4, int splits, const float* part, int accumulate, float* dw,
                                hipStream_t s) {
  const bool runs = splits >= SUM_RUNS;
  const int per = runs ? PROD_THREADS / 8 : PROD_THREADS;
  const auto kernel = runs ? route_dw_sum_kernel<8> : route_dw_sum_kernel<1>;
  kernel<<<(n4 + per - 1) / per, PROD_THREADS, 0, s>>>(n4, splits, (const float4*)part, accumulate,
                                                       (float4*)dw);
  return hipGetLastError();
}

int64_t route_backward_ws_bytes(const moe_dims_t& d, int T) {
  return T > 0 ? (int64_t)route_bwd_plan(d, T).total : 0;
}
int64_t route_backward_ws_bytes_up_to(const moe_dims_t& d, int T) {
  return T > 0 ? (int64_t)((route_bwd_plan(d, T).up_to + 255) & ~(size_t)255) : 0;
}

template <typename T, int MT>
static hipError_t launch_products(const RouteBwdPlan& p, const DlogitsArgs* few,
                                  const RouteBwdArgs& a, int dx_items,
                                  const void* x, const void* w, const void* dx_add, void* dx,
                                  hipStream_t s) {
  if (few) {
    constexpr int waves = RBWD_THREADS / MOE_WAVE;
    const auto kernel = a.steps == 1 ? route_few_kernel<T, MT, 1> : route_few_kernel<T, MT, 2>;
    kernel<<<a.dw_blocks + (dx_items + waves - 1) / waves, RBWD_THREADS, 0, s>>>(
        *few, a, dx_items, (const T*)x, (const T*)w, (const T*)dx_add, (T*)dx);
    return hipGetLastError();
  }
  auto run = [&](RouteBwdArgs b, int dw_blocks, int items) {
    b.dw_blocks = dw_blocks;
    const int nx = (items + PROD_WAVES - 1) / PROD_WAVES;
    route_products_kernel<T, MT><<<((dw_blocks + 7) & ~7) + ((nx + 7) & ~7), PROD_THREADS, 0, s>>>(
        b, items, (const T*)x, (const T*)w, (const T*)dx_add, (T*)dx);
    return hipGetLastError();
  };
  const bool apart = p.apart && a.dw_blocks > 0 && dx_items > 0;
  hipError_t e = run(a, a.dw_blocks, apart ? 0 : dx_items);
  if (e == hipSuccess && apart) e = run(a, 0, dx_items);
  if (e != hipSuccess || !a.dw || a.splits == 1) return e;
  return launch_dw_sum((int)((int64_t)a.E * a.H / 4), a.splits, a.part, a.accumulate, a.dw, s);
}
template <typename T>
static hipError_t launch_products_t(const RouteBwdPlan& p, const DlogitsArgs* few,
                                    const RouteBwdArgs& a, int dx_items, const void* x,
                                    const void* w, const void* dx_add, void* dx, hipStream_t s) {
  switch (p.mt) {
    case 1: return launch_products<T, 1>(p, few, a, dx_items, x, w, dx_add, dx, s);
    case 2: return launch_products<T, 2>(p, few, a, dx_items, x, w, dx_add, dx, s);
    case 3: return launch_products<T, 3>(p, few, a, dx_items, x, w, dx_add, dx, s);
    default: return launch_products<T, 4>(p, few, a, dx_items, x, w, dx_add, dx, s);
  }
}

// dx and dw may be null; x is read only for dw, w_router only for dx.  An
// empty batch only clears dw.
hipError_t launch_route_backward(const moe_dims_t& d, int T, const void* x, const void* w_router,
                                 const int32_t* ids, const float* logits, const float* dtopk_w,
                                 const float* dlogits_add, float* dlogits, const void* dx_add,
                                 void* dx, float* dw, int accumulate, void* ws, hipStream_t s) {
  if (T == 0)
    return dw ? launch_dw_sum((int)((int64_t)d.n_experts * d.hidden / 4), 0, nullptr, accumulate, dw, s)
              : hipSuccess;
  const RouteBwdPlan p = route_bwd_plan(d, T);
  const bool packs = d.dtype == MOE_BF16;
  char* base = static_cast<char*>(ws);
  float* pad = !packs && (dx || dw) ? reinterpret_cast<float*>(base + p.fx) : nullptr;
  uint4* fx = packs && dx ? reinterpret_cast<uint4*>(base + p.fx) : nullptr;
  uint4* fw = packs && dw ? reinterpret_cast<uint4*>(base + p.fw) : nullptr;
  const DlogitsArgs g{T, d.n_experts, d.top_k, d.renormalize, ids, logits, dtopk_w, dlogits_add,
                      dlogits};
  const bool few = (dx || dw) && p.steps <= 2 && p.splits == 1 && dlogits_add != dlogits;
  if (!few) {
    // up to 32 experts two a lane (16384 x 64, 8 experts: 12.6 us for the call, 13.8
    // with four)
    const auto kernel = p.ks == 1 ? route_dlogits_kernel<1> : route_dlogits_kernel<2>;
    kernel<<<p.steps, RBWD_THREADS, 0, s>>>(g, p.mt, pad, fx, fw);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || (!dx && !dw)) return e;
  }
  const RouteBwdArgs a{T, d.hidden, d.n_experts, p.ncg, p.steps, p.per, p.splits, p.dx_tiles,
                       dw ? p.splits * p.ncg : 0, pad, fx, fw,
                       p.splits > 1 ? reinterpret_cast<float*>(base + p.part) : nullptr, dw, accumulate};
  const int dx_items = dx ? (2 * p.steps + p.dx_tiles - 1) / p.dx_tiles * p.ncg : 0;
  const DlogitsArgs* in_one = few ? &g : nullptr;
  if (packs) return launch_products_t<bf16>(p, in_one, a, dx_items, x, w_router, dx_add, dx, s);
  return launch_products_t<float>(p, in_one, a, dx_items, x, w_router, dx_add, dx, s);
}

}  // namespace moe
