// The experts' gated feed-forward block for training: forward that keeps what
// its backward pass needs, and the backward pass.  Per expert, over its rows
// p (x_p = x[perm[p] / k]):
//
//   g = x W_g^T, u = x W_u^T, a = SiLU(g) u, y = a W_d^T
//   da = dy W_d; dg = da u s (1 + g (1 - s)), du = da g s, s = sigmoid(g)
//   dx = dg W_g + du W_u; dW_g = dg^T x, dW_u = du^T x, dW_d = dy^T a
//
// Five products per element: C[n][m] = sum_k A[m][k] B[n][k], m the fast axis
// of the output.  Either operand's k may be its fast axis (KMAJ) or its slow
// one, which is turned while a tile is staged into LDS.
#include <algorithm>

#include "common.h"
#include "ffn_train.h"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int TM = 64;   // outputs along m per block: one block of columns kept in 8 bits
constexpr int TN = 64;   // outputs along n per block, 16 a wave
constexpr int BK = 32;   // k per stage

template <typename T> struct mm;
template <> struct mm<bf16> {
  typedef bf16 elem_t;
  static constexpr int V = 8;         // elements of a 16-byte chunk
  static constexpr int PITCH = 40;    // LDS row, elements
  struct Frag { uint4 v; };
  __device__ static Frag load(const bf16* row, int kg) {
    return {*reinterpret_cast<const uint4*>(row + 8 * kg)};
  }
  __device__ static f32x4_t mac(const Frag& a, const Frag& b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a.v),
                                                   __builtin_bit_cast(bf16x8_t, b.v), c, 0, 0, 0);
  }
};
template <> struct mm<float> {
  typedef float elem_t;
  static constexpr int V = 4;
  static constexpr int PITCH = 36;
  struct Frag { float4 v[2]; };
  // lane group kg holds k = 4 kg..+3 and 16 + 4 kg..+3; the four groups of one
  // instruction take k = j, 4 + j, 8 + j, 12 + j, the same in both operands
  __device__ static Frag load(const float* row, int kg) {
    return {{*reinterpret_cast<const float4*>(row + 4 * kg),
             *reinterpret_cast<const float4*>(row + 16 + 4 * kg)}};
  }
  __device__ static f32x4_t mac(const Frag& a, const Frag& b, f32x4_t c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[h].x, b.v[h].x, c, 0, 0, 0);
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[h].y, b.v[h].y, c, 0, 0, 0);
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[h].z, b.v[h].z, c, 0, 0, 0);
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[h].w, b.v[h].w, c, 0, 0, 0);
    }
    return c;
  }
};

// One operand: element (r, k) at base[row(r) * ld + k] (k fast) or
// base[row(k) * ld + r]; rows are token rows, gathered through perm where
// given, of `rows` in the segment, or the rows of a weight matrix.
template <typename T> struct Operand {
  const T* base;
  int64_t ld;
  const int32_t* perm;   // token of row p: perm[p] / k (nullptr: row p itself)
  int k;
  int rows;              // rows that exist (the slow axis)
  int cols;              // elements of a row
  __device__ const T* row(int r) const {
    return base + (int64_t)(perm ? perm[r] / k : r) * ld;
  }
};

// Stage 64 outputs' worth of 32 k of an operand as [64][PITCH], k fast.
template <typename T, bool KMAJ>
__device__ __forceinline__ void stage(const Operand<T>& o, int r0, int k0, T* lds) {
  constexpr int V = mm<T>::V, PITCH = mm<T>::PITCH;
  constexpr int N = TM * BK / V / 256;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = threadIdx.x + 256 * i;
    if (KMAJ) {
      const int r = c / (BK / V), kc = c % (BK / V) * V;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r0 + r < o.rows && k0 + kc < o.cols)
        v = *reinterpret_cast<const uint4*>(o.row(r0 + r) + k0 + kc);
      *reinterpret_cast<uint4*>(lds + r * PITCH + kc) = v;
    } else {
      const int k = c / (TM / V), rc = c % (TM / V) * V;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (k0 + k < o.rows && r0 + rc < o.cols)
        v = *reinterpret_cast<const uint4*>(o.row(k0 + k) + r0 + rc);
      const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int j = 0; j < V; ++j) lds[(rc + j) * PITCH + k] = e[j];
    }
  }
}

template <typename T> struct Tile {
  T a[TM * mm<T>::PITCH], b[TN * mm<T>::PITCH];
};

// acc[i] += the products of 16 outputs m = 16 i.. with this wave's 16 outputs n
template <typename T, bool AK, bool BKM>
__device__ __forceinline__ void product(const Operand<T>& A, const Operand<T>& B, int m0, int n0,
                                        int K, Tile<T>& t, f32x4_t (&acc)[4]) {
  const int lane = lane_id(), wave = threadIdx.x / 64, r = lane & 15, kg = lane >> 4;
  for (int k0 = 0; k0 < K; k0 += BK) {
    __syncthreads();
    stage<T, AK>(A, m0, k0, t.a);
    stage<T, BKM>(B, n0, k0, t.b);
    __syncthreads();
    const auto b = mm<T>::load(t.b + (16 * wave + r) * mm<T>::PITCH, kg);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc[i] = mm<T>::mac(mm<T>::load(t.a + (16 * i + r) * mm<T>::PITCH, kg), b, acc[i]);
  }
}

// The segment that holds n-tile `tile` of the rows sorted by expert: expert,
// first row of the tile in it, its rows and start.  False past the last tile.
struct Segment { int e, row0, n, start; };
__device__ __forceinline__ bool find_segment(const int32_t* offsets, int E, int tile, Segment& s) {
  const int lane = lane_id();
  int o = 0, n = 0;
  if (lane < E) {
    o = offsets[lane];
    n = offsets[lane + 1] - o;
  }
  const int tiles = (n + TN - 1) / TN, incl = wave_incl_scan_i(tiles);
  const uint64_t in = __ballot(lane < E && tile >= incl - tiles && tile < incl);
  if (!in) return false;
  const int l = __ffsll((unsigned long long)in) - 1;
  s.e = l;
  s.row0 = (tile - __builtin_amdgcn_readlane(incl - tiles, l)) * TN;
  s.n = __builtin_amdgcn_readlane(n, l);
  s.start = __builtin_amdgcn_readlane(o, l);
  return true;
}

__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = float4{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ void store4(bf16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(f2_to_bf16x2(v[0], v[1]), f2_to_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const bf16* p, float (&v)[4]) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
}

// Gate and up of 64 channels of 64 rows, their product, and what is kept.
template <typename T>
__global__ void __launch_bounds__(256) train_gate_up_kernel(TrainArgs a) {
  __shared__ Tile<T> t;
  Segment s;
  if (!find_segment(a.offsets, a.E, blockIdx.x, s)) return;
  const int m0 = blockIdx.y * TM, I = a.I, H = a.H;
  const Operand<T> x{(const T*)a.x, H, a.perm + s.start, a.k, s.n, H};
  const int64_t we = (int64_t)s.e * I * H;
  f32x4_t g[4] = {}, u[4] = {};
  product<T, true, true>(Operand<T>{(const T*)a.w_gate + we, H, nullptr, 1, I, H}, x, m0, s.row0, H, t, g);
  product<T, true, true>(Operand<T>{(const T*)a.w_up + we, H, nullptr, 1, I, H}, x, m0, s.row0, H, t, u);
  const int lane = lane_id(), kg = lane >> 4;
  const int n = s.row0 + 16 * (threadIdx.x / 64) + (lane & 15);
  const bool live = n < s.n;
  const int64_t p = s.start + n;
  float inv[2] = {0.f, 0.f};
  if (a.keep8) {   // the lane group's maxima joined over the four groups of a row
    uint32_t top[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (m0 + 16 * i + 4 * kg + q < I) {
          top[0] = max(top[0], __float_as_uint(g[i][q]) & 0x7FFFFFFFu);
          top[1] = max(top[1], __float_as_uint(u[i][q]) & 0x7FFFFFFFu);
        }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      top[j] = max(top[j], (uint32_t)__shfl_xor((int)top[j], 16));
      top[j] = max(top[j], (uint32_t)__shfl_xor((int)top[j], 32));
      float scale;
      inv[j] = pack8_inverse(__uint_as_float(top[j]), scale);
      if (live && kg == 0) a.scale[(2 * p + j) * a.blocks + blockIdx.y] = scale;
    }
  }
  if (!live) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + 16 * i + 4 * kg;
    if (m >= I) continue;
    float gv[4], uv[4], h[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      gv[q] = g[i][q];
      uv[q] = u[i][q];
      h[q] = silu_f(gv[q]) * uv[q];
    }
    store4((T*)a.act + p * I + m, h);
    if (a.keep8) {
      *reinterpret_cast<uint32_t*>((int8_t*)a.kept + 2 * p * I + m) = pack8x4(gv, inv[0]);
      *reinterpret_cast<uint32_t*>((int8_t*)a.kept + (2 * p + 1) * I + m) = pack8x4(uv, inv[1]);
    } else if (a.kept) {
      store4((T*)a.kept + 2 * p * I + m, gv);
      store4((T*)a.kept + (2 * p + 1) * I + m, uv);
    }
  }
}

// y = a W_d^T
template <typename T>
__global__ void __launch_bounds__(256) train_down_kernel(TrainArgs a) {
  __shared__ Tile<T> t;
  Segment s;
  if (!find_segment(a.offsets, a.E, blockIdx.x, s)) return;
  const int m0 = blockIdx.y * TM, I = a.I, H = a.H;
  f32x4_t y[4] = {};
  product<T, true, true>(Operand<T>{(const T*)a.w_down + (int64_t)s.e * I * H, I, nullptr, 1, H, I},
                         Operand<T>{(const T*)a.act + (int64_t)s.start * I, I, nullptr, 1, s.n, I}, m0,
                         s.row0, I, t, y);
  const int lane = lane_id(), n = s.row0 + 16 * (threadIdx.x / 64) + (lane & 15);
  if (n >= s.n) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v[4] = {y[i][0], y[i][1], y[i][2], y[i][3]};
    store4((T*)a.y + (int64_t)(s.start + n) * H + m0 + 16 * i + 4 * (lane >> 4), v);
  }
}

// da = dy W_d, and from it and the kept gate and up: dg, du and a
template <typename T>
__global__ void __launch_bounds__(256) train_dact_kernel(TrainArgs a) {
  __shared__ Tile<T> t;
  Segment s;
  if (!find_segment(a.offsets, a.E, blockIdx.x, s)) return;
  const int m0 = blockIdx.y * TM, I = a.I, H = a.H;
  f32x4_t d[4] = {};
  product<T, false, true>(Operand<T>{(const T*)a.w_down + (int64_t)s.e * I * H, I, nullptr, 1, H, I},
                          Operand<T>{(const T*)a.dy + (int64_t)s.start * H, H, nullptr, 1, s.n, H}, m0,
                          s.row0, H, t, d);
  const int lane = lane_id(), n = s.row0 + 16 * (threadIdx.x / 64) + (lane & 15);
  if (n >= s.n) return;
  const int64_t p = s.start + n;
  float scale[2] = {1.f, 1.f};
  if (a.keep8) {
    scale[0] = a.scale[2 * p * a.blocks + blockIdx.y];
    scale[1] = a.scale[(2 * p + 1) * a.blocks + blockIdx.y];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + 16 * i + 4 * (lane >> 4);
    if (m >= I) continue;
    float g[4], u[4], h[4], dg[4], du[4];
    if (a.keep8) {
      unpack8x4(*reinterpret_cast<const uint32_t*>((const int8_t*)a.kept + 2 * p * I + m), scale[0], g);
      unpack8x4(*reinterpret_cast<const uint32_t*>((const int8_t*)a.kept + (2 * p + 1) * I + m), scale[1], u);
    } else {
      load4((const T*)a.kept + 2 * p * I + m, g);
      load4((const T*)a.kept + (2 * p + 1) * I + m, u);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) gated_grad(g[q], u[q], d[i][q], h[q], dg[q], du[q]);
    store4((T*)a.act + p * I + m, h);
    store4((T*)a.dgu + 2 * p * I + m, dg);
    store4((T*)a.dgu + (2 * p + 1) * I + m, du);
  }
}

// dx = dg W_g + du W_u
template <typename T>
__global__ void __launch_bounds__(256) train_dx_kernel(TrainArgs a) {
  __shared__ Tile<T> t;
  Segment s;
  if (!find_segment(a.offsets, a.E, blockIdx.x, s)) return;
  const int m0 = blockIdx.y * TM, I = a.I, H = a.H;
  const int64_t we = (int64_t)s.e * I * H;
  const T* rows = (const T*)a.dgu + 2 * (int64_t)s.start * I;
  f32x4_t d[4] = {};
  product<T, false, true>(Operand<T>{(const T*)a.w_gate + we, H, nullptr, 1, I, H},
                          Operand<T>{rows, 2 * I, nullptr, 1, s.n, I}, m0, s.row0, I, t, d);
  product<T, false, true>(Operand<T>{(const T*)a.w_up + we, H, nullptr, 1, I, H},
                          Operand<T>{rows + I, 2 * I, nullptr, 1, s.n, I}, m0, s.row0, I, t, d);
  const int lane = lane_id(), n = s.row0 + 16 * (threadIdx.x / 64) + (lane & 15);
  if (n >= s.n) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v[4] = {d[i][0], d[i][1], d[i][2], d[i][3]};
    store4((T*)a.dx + (int64_t)(s.start + n) * H + m0 + 16 * i + 4 * (lane >> 4), v);
  }
}

// dW_g, dW_u [I][H] (m over H, n over I) and dW_d [H][I] of one expert
template <typename T, typename D>
__global__ void __launch_bounds__(256) train_dw_kernel(TrainArgs a) {
  __shared__ Tile<T> t;
  const int e = blockIdx.z / 3, which = blockIdx.z % 3, I = a.I, H = a.H;
  const bool down = which == 2;
  D* out = (D*)a.dw[which];
  if (!out) return;
  const int M = down ? I : H, N = down ? H : I;
  // the grid covers tiles of H by tiles of I
  const int m0 = (down ? blockIdx.y : blockIdx.x) * TM, n0 = (down ? blockIdx.x : blockIdx.y) * TN;
  const int start = a.offsets ? a.offsets[e] : 0, n = a.offsets ? a.offsets[e + 1] - start : 0;
  f32x4_t d[4] = {};
  if (down)
    product<T, false, false>(Operand<T>{(const T*)a.act + (int64_t)start * I, I, nullptr, 1, n, I},
                             Operand<T>{(const T*)a.dy + (int64_t)start * H, H, nullptr, 1, n, H}, m0, n0,
                             n, t, d);
  else
    product<T, false, false>(Operand<T>{(const T*)a.x, H, a.perm + start, a.k, n, H},
                             Operand<T>{(const T*)a.dgu + (2 * (int64_t)start + which) * I, 2 * I, nullptr, 1, n, I},
                             m0, n0, n, t, d);
  const int lane = lane_id(), row = n0 + 16 * (threadIdx.x / 64) + (lane & 15);
  if (row >= N) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + 16 * i + 4 * (lane >> 4);
    if (m >= M) continue;
    float v[4] = {d[i][0], d[i][1], d[i][2], d[i][3]};
    D* to = out + (int64_t)e * I * H + (int64_t)row * M + m;
    if (a.accumulate) {
      float was[4];
      load4(to, was);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += was[q];
    }
    store4(to, v);
  }
}

}  // namespace

// Rows enough for the 256 x 256 tiles of ffn_train_gemm.hip.
static bool large(const TrainArgs& a, int P) { return P >= 64 * a.E && a.I >= 128 && a.H >= 128; }

template <typename T> static hipError_t forward(const TrainArgs& a, int P, hipStream_t s) {
  if (sizeof(T) == 2 && large(a, P)) {
    const hipError_t e = launch_train_gemm(0, a, P, s);
    return e != hipSuccess ? e : launch_train_gemm(1, a, P, s);
  }
  const int tiles = P / TN + std::min(a.E, P);
  train_gate_up_kernel<T><<<dim3(tiles, (a.I + TM - 1) / TM), 256, 0, s>>>(a);
  train_down_kernel<T><<<dim3(tiles, a.H / TM), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T> static hipError_t backward(const TrainArgs& a, int P, hipStream_t s) {
  if (sizeof(T) == 2 && P > 0 && large(a, P)) {
    hipError_t e = launch_train_gemm(2, a, P, s);
    if (e == hipSuccess && a.dx) e = launch_train_gemm(3, a, P, s);
    return e != hipSuccess ? e : launch_train_gemm(4, a, P, s);
  }
  const int tiles = P / TN + std::min(a.E, P);
  const int hi = a.H / TM, ii = (a.I + TM - 1) / TM;
  if (P > 0) {
    train_dact_kernel<T><<<dim3(tiles, ii), 256, 0, s>>>(a);
    if (a.dx) train_dx_kernel<T><<<dim3(tiles, hi), 256, 0, s>>>(a);
  }
  if (a.dw[0] || a.dw[1] || a.dw[2]) {
    if (a.dw_f32)
      train_dw_kernel<T, float><<<dim3(hi, ii, 3 * a.E), 256, 0, s>>>(a);
    else
      train_dw_kernel<T, T><<<dim3(hi, ii, 3 * a.E), 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

int64_t train_ws_bytes(const moe_dims_t& d, int64_t T) {
  return T * d.top_k * 3 * d.inter * (d.dtype == MOE_BF16 ? 2 : 4);
}

hipError_t launch_ffn_train(const TrainArgs& a, int P, bool is_bf16, hipStream_t s) {
  return is_bf16 ? forward<bf16>(a, P, s) : forward<float>(a, P, s);
}
hipError_t launch_ffn_backward(const TrainArgs& a, int P, bool is_bf16, hipStream_t s) {
  return is_bf16 ? backward<bf16>(a, P, s) : backward<float>(a, P, s);
}

}  // namespace moe
