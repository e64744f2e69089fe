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
#include <algorithm>

#include "common.h"

namespace moe {

constexpr int RBWD_THREADS = 256;
constexpr int RBWD_SPLIT_TOKENS = 256;

// One wave per token, lane = expert; dlogits_add may be dlogits itself.
__global__ void __launch_bounds__(RBWD_THREADS)
route_dlogits_kernel(int T, int E, int k, int renorm, const int32_t* __restrict__ ids,
                     const float* __restrict__ logits, const float* __restrict__ dtopk_w,
                     const float* dlogits_add, float* dlogits) {
  const int lane = lane_id();
  const int t = blockIdx.x * (RBWD_THREADS / MOE_WAVE) + (threadIdx.x >> 6);
  if (t >= T) return;
  const bool in = lane < E;
  const int64_t o = (int64_t)t * E + lane;
  float dl = 0.f;
  if (dtopk_w) {
    const float l = in ? logits[o] : 0.f;
    float G = 0.f, n = 0.f;
    for (int j = 0; j < k; ++j) {
      const int e = ids[(int64_t)t * k + j];
      const float g = dtopk_w[(int64_t)t * k + j];
      if (e == lane && in) {
        G += g;
        n += 1.f;
      }
    }
    const bool part = in && (!renorm || n > 0.f);
    const float m = wave_max(part ? l : -__builtin_inff());
    const float z = part ? expf(l - m) : 0.f;
    const float mult = renorm ? n : 1.f;
    const float s = wave_sum(part ? mult * z : 0.f);
    const float p = part ? z / s : 0.f;
    const float c = wave_sum(n > 0.f ? G * p : 0.f);
    dl = part ? p * (G - mult * c) : 0.f;
  }
  if (in) {
    if (dlogits_add) dl += dlogits_add[o];
    dlogits[o] = dl;
  }
}

// dx: one thread per (token, eight columns), summed over the experts in order.
template <typename T>
__global__ void __launch_bounds__(RBWD_THREADS)
route_dx_kernel(uint32_t n, uint32_t units, int H, int E, const float* __restrict__ dl,
                const T* __restrict__ w, const T* dx_add, T* dx) {
  const uint32_t g = blockIdx.x * RBWD_THREADS + threadIdx.x;
  if (g >= n) return;
  const uint32_t t = g / units, u = g - t * units;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (dx_add) elem<T>::load8(dx_add + (int64_t)g * 8, acc);
  for (int e = 0; e < E; ++e) {
    float wv[8];
    elem<T>::load8(w + (int64_t)e * H + u * 8, wv);
    const float d = dl[(int64_t)t * E + e];
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = fmaf(d, wv[c], acc[c]);
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) elem<T>::store(dx, (int64_t)g * 8 + c, acc[c]);
}

// dW partials: one thread per (expert, eight columns) and range of tokens.
template <typename T>
__global__ void __launch_bounds__(RBWD_THREADS)
route_dw_kernel(int T_, int units, int H, int E, const float* __restrict__ dl,
                const T* __restrict__ x, float* __restrict__ part) {
  const int g = blockIdx.x * RBWD_THREADS + threadIdx.x;
  if (g >= E * units) return;
  const int e = g / units, u = g - e * units;
  const int t0 = blockIdx.y * RBWD_SPLIT_TOKENS, t1 = min(T_, t0 + RBWD_SPLIT_TOKENS);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int t = t0; t < t1; ++t) {
    float xv[8];
    elem<T>::load8(x + (int64_t)t * H + u * 8, xv);
    const float d = dl[(int64_t)t * E + e];
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = fmaf(d, xv[c], acc[c]);
  }
  float* o = part + ((int64_t)blockIdx.y * E + e) * H + u * 8;
#pragma unroll
  for (int c = 0; c < 8; ++c) o[c] = acc[c];
}

// dW = (dW +) the sum of the ranges' partials, in range order.
__global__ void __launch_bounds__(RBWD_THREADS)
route_dw_sum_kernel(int64_t n, int splits, const float* __restrict__ part, int accumulate,
                    float* __restrict__ dw) {
  const int64_t i = (int64_t)blockIdx.x * RBWD_THREADS + threadIdx.x;
  if (i >= n) return;
  float s = accumulate ? dw[i] : 0.f;
  for (int p = 0; p < splits; ++p) s += part[(int64_t)p * n + i];
  dw[i] = s;
}

static int dw_splits(int T) { return (T + RBWD_SPLIT_TOKENS - 1) / RBWD_SPLIT_TOKENS; }

int64_t route_backward_ws_bytes(const moe_dims_t& d, int T) {
  return (int64_t)dw_splits(T) * d.n_experts * d.hidden * 4;
}

template <typename T>
static hipError_t route_bwd_t(const moe_dims_t& d, int T_, const T* x, const T* w, const float* dl,
                              const T* dx_add, T* dx, float* dw, int accumulate, float* ws,
                              hipStream_t s) {
  const int H = d.hidden, E = d.n_experts, units = H / 8;
  if (dx && T_ > 0) {
    const uint32_t n = (uint32_t)T_ * units;
    route_dx_kernel<T><<<(n + RBWD_THREADS - 1) / RBWD_THREADS, RBWD_THREADS, 0, s>>>(
        n, units, H, E, dl, w, dx_add, dx);
  }
  if (dw) {
    const int splits = dw_splits(T_);
    if (splits > 0) route_dw_kernel<T><<<dim3((E * units + RBWD_THREADS - 1) / RBWD_THREADS, splits), RBWD_THREADS,
                         0, s>>>(T_, units, H, E, dl, x, ws);
    const int64_t n = (int64_t)E * H;
    route_dw_sum_kernel<<<(unsigned)((n + RBWD_THREADS - 1) / RBWD_THREADS), RBWD_THREADS, 0, s>>>(
        n, splits, ws, accumulate, dw);
  }
  return hipGetLastError();
}

// dx and dw may be null; x is read only for dw, w_router only for dx.  An
// empty batch only clears dw.
hipError_t launch_route_backward(const moe_dims_t& d, int T, const void* x, const void* w_router,
                                 const int32_t* ids, const float* logits, const float* dtopk_w,
                                 const float* dlogits_add, float* dlogits, const void* dx_add,
                                 void* dx, float* dw, int accumulate, void* ws, hipStream_t s) {
  if (T > 0) {
    constexpr int per = RBWD_THREADS / MOE_WAVE;
    route_dlogits_kernel<<<(T + per - 1) / per, RBWD_THREADS, 0, s>>>(
        T, d.n_experts, d.top_k, d.renormalize, ids, logits, dtopk_w, dlogits_add, dlogits);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (d.dtype == MOE_BF16)
    return route_bwd_t<bf16>(d, T, (const bf16*)x, (const bf16*)w_router, dlogits,
                             (const bf16*)dx_add, (bf16*)dx, dw, accumulate, (float*)ws, s);
  return route_bwd_t<float>(d, T, (const float*)x, (const float*)w_router, dlogits,
                            (const float*)dx_add, (float*)dx, dw, accumulate, (float*)ws, s);
}

}  // namespace moe
