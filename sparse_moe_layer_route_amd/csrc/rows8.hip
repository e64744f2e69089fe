// Rows kept in 8 bits and brought back: blocks of 64 columns of a row with a
// scale each (the format: ffn_train.h).
//
// Both kernels move bytes and do little else.  Where rows start on 16 bytes
// and have whole groups of 16 columns, four lanes share a block, 16 columns
// each (32 or 64 bytes in, 16 out); any other rows take 16 lanes a block that
// step over it, so that neighbouring lanes touch neighbouring elements.
#include "ffn_train.h"

namespace moe {
namespace {

template <int CTRL> __device__ __forceinline__ uint32_t umax_dpp(uint32_t v) {
  return max(v, (uint32_t)dpp_move<CTRL>((int)v, (int)v));
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const bf16* p) { return bf16_to_f(p->b); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(bf16* p, float v) { p->b = f_to_bf16(v); }

// Codes of N values, in the low byte of c: the sum with 1.5 * 2^23 rounds
// v * inv to an integer and leaves it there.  inv is rounded, so the product is
// off by up to 2^-16; where that could decide which of two codes is nearer, the
// middle between them does: 254 |v| and (2 m + 1) top are exact in 64 bits, so
// a tie is one.
template <int N>
__device__ __forceinline__ void codes_of(const float (&v)[N], float top, float inv, uint32_t (&c)[N]) {
  constexpr float SHIFT = 0x1.8p23f, CLOSE = 0.5f - 0x1p-14f;
  float far = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float b = fmaf(v[i], inv, SHIFT);
    c[i] = __float_as_uint(b);
    far = fmaxf(far, fabsf(fmaf(v[i], inv, SHIFT - b)));
  }
  if (far > CLOSE && inv > 0.0f) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float f = fabsf(v[i]) * inv, m = floorf(f);
      if (fabsf(f - m - 0.5f) < 0x1p-13f) {
        const double past = 254.0 * (double)fabsf(v[i]) - (double)(2.0f * m + 1.0f) * (double)top;
        const int n = (int)m, near = past > 0.0 || (past == 0.0 && (n & 1)) ? n + 1 : n;
        c[i] = (uint32_t)(v[i] < 0.0f ? -near : near);
      }
    }
  }
}

// The low bytes of four.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(b, a, 0x0C0C0400u) | __builtin_amdgcn_perm(d, c, 0x04000C0Cu);
}

// blocks: of a row; total: of all rows.  VEC: four lanes a block, else 16.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
rows_pack8_kernel(const T* __restrict__ src, int64_t ld, int cols, uint32_t blocks, uint32_t total,
                  int8_t* __restrict__ codes, float* __restrict__ scale) {
  constexpr int LANES = VEC ? 4 : 16, N = kKeepBlock / LANES;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t at = t / LANES;
  const int sub = threadIdx.x % LANES;
  const bool on = at < total;
  const uint32_t blk = on ? (uint32_t)at : 0u, row = blk / blocks, b = blk % blocks;
  const int col = (int)(b * kKeepBlock) + (VEC ? N * sub : sub);
  const T* from = src + (int64_t)row * ld;
  float v[N];
  if constexpr (VEC) {
    if (on && col < cols) {
      float lo[8], hi[8];
      elem<T>::load8(from + col, lo);
      elem<T>::load8(from + col + 8, hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = lo[i], v[8 + i] = hi[i];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = on && col + 16 * i < cols ? load1(from + col + 16 * i) : 0.f;
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  top = umax_dpp<0xB1>(top);   // lanes of a quad exchanged: 1, then 2 apart
  top = umax_dpp<0x4E>(top);
  if (!VEC) {
    top = max(top, (uint32_t)__shfl_xor((int)top, 4));
    top = max(top, (uint32_t)__shfl_xor((int)top, 8));
  }
  float s;
  const float inv = pack8_inverse(__uint_as_float(top), s);
  uint32_t c[N];
  codes_of(v, __uint_as_float(top), inv, c);
  if (!on) return;
  if (sub == 0) scale[blk] = s;
  int8_t* to = codes + (int64_t)row * cols + col;
  if constexpr (VEC) {
    if (col >= cols) return;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = inv > 0.0f ? low_bytes(c[4 * i], c[4 * i + 1], c[4 * i + 2], c[4 * i + 3]) : 0u;
    *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (col + 16 * i < cols) to[16 * i] = inv > 0.0f ? (int8_t)c[i] : 0;
  }
}

__device__ __forceinline__ void store16(float* p, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(p)[i] = float4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
}
__device__ __forceinline__ void store16(bf16* p, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<uint4*>(p)[i] =
        make_uint4(f2_to_bf16x2(v[8 * i], v[8 * i + 1]), f2_to_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                   f2_to_bf16x2(v[8 * i + 4], v[8 * i + 5]), f2_to_bf16x2(v[8 * i + 6], v[8 * i + 7]));
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
rows_unpack8_kernel(const int8_t* __restrict__ codes, const float* __restrict__ scale, int64_t ld,
                    int cols, uint32_t blocks, uint32_t total, T* __restrict__ dst) {
  constexpr int LANES = VEC ? 4 : 16, N = kKeepBlock / LANES;
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LANES;
  if (at >= total) return;
  const int sub = threadIdx.x % LANES;
  const uint32_t blk = (uint32_t)at, row = blk / blocks, b = blk % blocks;
  const int col = (int)(b * kKeepBlock) + (VEC ? N * sub : sub);
  if (col >= cols) return;
  const float s = scale[blk];
  const int8_t* from = codes + (int64_t)row * cols + col;
  T* to = dst + (int64_t)row * ld + col;
  if constexpr (VEC) {
    const uint4 w = *reinterpret_cast<const uint4*>(from);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      v[i] = (float)((int32_t)(ws[i / 4] << (24 - 8 * (i % 4))) >> 24) * s;
    store16(to, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (col + 16 * i < cols) store1(to + 16 * i, (float)from[16 * i] * s);
  }
}

}  // namespace

hipError_t launch_rows_pack8(int64_t rows, int64_t cols, int64_t ld, const void* src, bool is_bf16,
                             int8_t* codes, float* scale, hipStream_t s) {
  const uint32_t blocks = (uint32_t)((cols + kKeepBlock - 1) / kKeepBlock);
  const uint32_t total = (uint32_t)(rows * blocks);
  const bool vec = cols % 16 == 0 && (rows == 1 || ld * (is_bf16 ? 2 : 4) % 16 == 0);
  const unsigned grid = (unsigned)(((int64_t)total * (vec ? 4 : 16) + 255) / 256);
  if (is_bf16) {
    auto k = vec ? rows_pack8_kernel<bf16, true> : rows_pack8_kernel<bf16, false>;
    k<<<grid, 256, 0, s>>>((const bf16*)src, ld, (int)cols, blocks, total, codes, scale);
  } else {
    auto k = vec ? rows_pack8_kernel<float, true> : rows_pack8_kernel<float, false>;
    k<<<grid, 256, 0, s>>>((const float*)src, ld, (int)cols, blocks, total, codes, scale);
  }
  return hipGetLastError();
}

hipError_t launch_rows_unpack8(int64_t rows, int64_t cols, int64_t ld, const int8_t* codes,
                               const float* scale, void* dst, bool is_bf16, hipStream_t s) {
  const uint32_t blocks = (uint32_t)((cols + kKeepBlock - 1) / kKeepBlock);
  const uint32_t total = (uint32_t)(rows * blocks);
  const bool vec = cols % 16 == 0 && (rows == 1 || ld * (is_bf16 ? 2 : 4) % 16 == 0);
  const unsigned grid = (unsigned)(((int64_t)total * (vec ? 4 : 16) + 255) / 256);
  if (is_bf16) {
    auto k = vec ? rows_unpack8_kernel<bf16, true> : rows_unpack8_kernel<bf16, false>;
    k<<<grid, 256, 0, s>>>(codes, scale, ld, (int)cols, blocks, total, (bf16*)dst);
  } else {
    auto k = vec ? rows_unpack8_kernel<float, true> : rows_unpack8_kernel<float, false>;
    k<<<grid, 256, 0, s>>>(codes, scale, ld, (int)cols, blocks, total, (float*)dst);
  }
  return hipGetLastError();
}

}  // namespace moe
