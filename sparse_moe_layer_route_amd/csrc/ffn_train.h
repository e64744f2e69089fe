// What the kernels of the experts' training share: arguments, the gradient of
// the gated product, and the 8-bit form of kept rows.
#pragma once
#include "common.h"

namespace moe {

// act and dgu hold the layer's type: a bf16 layer rounds SiLU(g) u, dg and du
// once, so that the products that take them run on the bf16 matrix cores and
// their rows cost half the bytes.  Each output then carries two roundings of at
// most half a step (2^-8) instead of one: a 2-norm error of 0.0023 against 0.0017,
// 0.0026 where a sum has a single row.
struct TrainArgs {
  const void *x, *w_gate, *w_up, *w_down, *dy;   // x [T][H]; dy [P][H]
  const int32_t *offsets, *perm;
  void* kept;        // [P][2][I] rows of the layer's type, or int8
  float* scale;      // [P][2][blocks] when kept in 8 bits
  void *y, *dx;      // [P][H]
  void* dw[3];       // gate, up [E][I][H]; down [E][H][I]
  void *act, *dgu;   // workspace: SiLU(g) u [P][I]; dg and du [P][2][I]
  int E, H, I, k, blocks, pairs;   // pairs: T * k
  int keep8, dw_f32, accumulate;
  int n_dw;          // matrices whose gradients are asked for
};

// ------------------------------------------------- rows kept in 8 bits ----
// A block of 64 columns shares scale = top / 127, top its largest |value|; a
// value is kept as the nearest of -127..127 steps (ties to even).  A block
// whose top is below 2^-100 is kept as zeros (127 / top stays finite above
// it); one that holds an infinity or a NaN comes back as NaN throughout.
constexpr int kKeepBlock = 64;
constexpr float kKeepSmall = 0x1p-100f;

// 127 / top (0 where the codes are to be 0) and the scale; `top` may be the
// bits of an infinity or a NaN.
__device__ __forceinline__ float pack8_inverse(float top, float& scale) {
  const bool fine = (__float_as_uint(top) & 0x7FFFFFFFu) < 0x7F800000u;
  const bool live = fine && top >= kKeepSmall;
  scale = live ? top / 127.0f : fine ? 0.0f : __uint_as_float(0x7FC00000u);
  // next to the largest float the rounded scale's 127 steps would pass it
  if (live && 127.0f * scale > 0x1.fffffep127f) scale = __uint_as_float(__float_as_uint(scale) - 1);
  return live ? 127.0f / top : 0.0f;
}
// A block whose inverse is 0 has codes 0 whatever its values are.
__device__ __forceinline__ int pack8_code(float v, float inv) {
  return inv > 0.0f ? (int)rintf(v * inv) : 0;
}
__device__ __forceinline__ uint32_t pack8x4(const float (&v)[4], float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) w |= (uint32_t)(pack8_code(v[q], inv) & 0xFF) << (8 * q);
  return w;
}
__device__ __forceinline__ void unpack8x4(uint32_t w, float scale, float (&v)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = (float)((int32_t)(w << (24 - 8 * q)) >> 24) * scale;
}

// a = SiLU(g) u and the gradients of g and u from that of a.
__device__ __forceinline__ void gated_grad(float g, float u, float da, float& a, float& dg,
                                           float& du) {
  const float s = sigmoid_f(g), gs = g * s;
  a = gs * u;
  du = da * gs;
  dg = da * u * (s * (1.0f + (g - gs)));
}

int64_t train_ws_bytes(const moe_dims_t& d, int64_t T);
hipError_t launch_ffn_train(const TrainArgs& a, int P, bool is_bf16, hipStream_t s);
hipError_t launch_ffn_backward(const TrainArgs& a, int P, bool is_bf16, hipStream_t s);
hipError_t launch_rows_pack8(int64_t rows, int64_t cols, int64_t ld, const void* src, bool is_bf16,
                             int8_t* codes, float* scale, hipStream_t s);
hipError_t launch_rows_unpack8(int64_t rows, int64_t cols, int64_t ld, const int8_t* codes,
                               const float* scale, void* dst, bool is_bf16, hipStream_t s);

}  // namespace moe
