// Distillation from a teacher's top logits, with its gradient.  Per row, with
// z = student / tau over V classes, q = softmax(z), and the teacher's K entries
// (id_k, t_k):
//   p_k = softmax over the K entries of t_k / tau, or, when the log-sum-exp of
//   all of the teacher's t / tau is given, exp(t_k / tau - lse_teacher) with
//   the rest p_T = 1 - sum p on one tail class that joins the classes outside
//   the K (log q_T = lse_tail - lse).
//   KL = sum_k p_k (log p_k - log q_{id_k}) + p_T (log p_T - log q_T)
//   dKL/dz_v = q_v M - sum_{k: id_k = v} p_k      for a teacher's class
//            = exp(z_v - lse_tail) (q_T M - p_T)  for the others
//   (M = sum p + p_T; 1 unless the row has no entry, or no class outside).
// The classes outside the K are summed in 32 bits against their own maximum;
// the K entries, whose p and q nearly cancel in a trained student, and the
// joins are in 64 bits, so q sums to one to 64-bit accuracy and the error of
// the loss is that of lse_tail times (q_T - p_T) only.
#include <algorithm>

#include "common.h"

namespace moe {

constexpr int DISTILL_THREADS = 256;
constexpr double NEG_INF = -__builtin_huge_val();

struct DistillArgs {
  int T, V, K;
  int64_t ld;
  const int32_t* ids;
  const float* t_logits;
  const float* t_lse;    // may be null
  const float* token_w;  // may be null
  double inv_tau;
  float c_hi, c_lo;  // log2(e) / tau in two parts
  float scale;
  float* loss;
};

__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}
__device__ __forceinline__ double wave_max_d(double v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v = fmax(v, __shfl_xor(v, m, 64));
  return v;
}

// exp((s - m) / tau): the difference is exact or rounded once, and the factor
// log2(e) / tau is held in two floats, so no error is common to all terms.
// Below -1e30 the result is 0 anyway; the clamp keeps inf * c_lo out and lets
// NaN through.
__device__ __forceinline__ float distill_exp(float s, float m, float c_hi, float c_lo) {
  float d = s - m;
  d = d < -1e30f ? -1e30f : d;
  return __builtin_amdgcn_exp2f(fmaf(d, c_hi, d * c_lo));
}

__device__ __forceinline__ double log_add(double a, double b) {
  if (a != a || b != b) return a + b;  // fmax and fmin would drop a NaN
  const double hi = fmax(a, b), lo = fmin(a, b);
  return hi == NEG_INF ? hi : hi + log1p(exp(lo - hi));
}

template <typename T>
__global__ void __launch_bounds__(DISTILL_THREADS)
distill_kernel(DistillArgs a, const T* student, T* dstudent) {
  extern __shared__ double smem[];
  const int K = a.K, V = a.V, tid = threadIdx.x, lane = lane_id(), wv = tid >> 6;
  constexpr int NW = DISTILL_THREADS / MOE_WAVE;
  double* s_p = smem;              // [K]
  double* s_z = s_p + K;           // [K]
  int32_t* s_id = (int32_t*)(s_z + K);  // [K]
  uint32_t* bits = (uint32_t*)(s_id + K);  // [(V + 31) / 32]: teacher's classes
  __shared__ int s_dup;
  __shared__ float s_f[NW];
  __shared__ double s_head[4];
  const int64_t t = blockIdx.x;
  const T* row = student + t * a.ld;
  T* drow = dstudent ? dstudent + t * a.ld : nullptr;
  const double c = (double)a.scale * (a.token_w ? (double)a.token_w[t] : 1.0);
  auto clear = [&] {
    if (tid == 0) a.loss[t] = 0.f;
    if (drow)
      for (int v = tid; v < V; v += DISTILL_THREADS) elem<T>::store(drow, v, 0.f);
  };
  if (c == 0.0) return clear();  // a masked row is not read
  if (tid == 0) s_dup = 0;
  for (int i = tid; i < (V + 31) / 32; i += DISTILL_THREADS) bits[i] = 0u;
  __syncthreads();
  for (int i = tid; i < K; i += DISTILL_THREADS) {
    const int id = a.ids[t * K + i];
    const bool ok = (unsigned)id < (unsigned)V;
    s_id[i] = ok ? id : -1;
    if (ok) {
      const uint32_t bit = 1u << (id & 31);
      if (atomicOr(&bits[id >> 5], bit) & bit) s_dup = 1;
      s_z[i] = (double)elem<T>::load(row, id) * a.inv_tau;
      s_p[i] = (double)a.t_logits[t * K + i] * a.inv_tau;
    }
  }
  __syncthreads();
  // own(i): entry i is the first of its class (a class counts once in q)
  auto own = [&](int i) {
    if (s_id[i] < 0) return false;
    if (s_dup)
      for (int j = 0; j < i; ++j)
        if (s_id[j] == s_id[i]) return false;
    return true;
  };
  if (wv == 0) {
    double m = NEG_INF, zm = NEG_INF;
    for (int i = lane; i < K; i += 64)
      if (s_id[i] >= 0) {
        m = fmax(m, s_p[i]);
        zm = fmax(zm, s_z[i]);
      }
    m = wave_max_d(m);
    zm = wave_max_d(zm);
    // log p = (t / tau - ref) - log_sum, in this order: beside a maximum of the
    // type's lowest value the logarithm would be lost
    double ref = m, log_sum = 0.0;
    if (a.t_lse) {
      ref = (double)a.t_lse[t];
    } else if (m > NEG_INF) {
      double e = 0.0;
      for (int i = lane; i < K; i += 64)
        if (s_id[i] >= 0) e += exp(s_p[i] - m);
      log_sum = log(wave_sum_d(e));
    }
    double mass = 0.0, hs = 0.0, cnt = 0.0;
    for (int i = lane; i < K; i += 64) {
      if (s_id[i] < 0) continue;
      // s_p becomes log p
      s_p[i] = s_p[i] == NEG_INF ? NEG_INF : (s_p[i] - ref) - log_sum;
      mass += exp(s_p[i]);
      if (own(i)) {
        cnt += 1.0;
        if (s_z[i] != NEG_INF) hs += exp(s_z[i] - zm);
      }
    }
    mass = wave_sum_d(mass);
    hs = wave_sum_d(hs);
    cnt = wave_sum_d(cnt);
    if (lane == 0) {
      s_head[0] = mass;
      s_head[1] = hs == 0.0 ? NEG_INF : log(hs);
      s_head[2] = cnt;
      s_head[3] = zm;
    }
  }
  float m = -__builtin_inff();
  for (int v = tid; v < V; v += DISTILL_THREADS)
    if (!((bits[v >> 5] >> (v & 31)) & 1u)) m = fmaxf(m, elem<T>::load(row, v));
  m = wave_max(m);
  if (lane == 0) s_f[wv] = m;
  __syncthreads();
  m = s_f[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) m = fmaxf(m, s_f[w]);
  __syncthreads();
  const float ms = m == -__builtin_inff() ? 0.f : m;
  float sum = 0.f;
  for (int v = tid; v < V; v += DISTILL_THREADS)
    if (!((bits[v >> 5] >> (v & 31)) & 1u)) sum += distill_exp(elem<T>::load(row, v), ms, a.c_hi, a.c_lo);
  sum = wave_sum(sum);
  if (lane == 0) s_f[wv] = sum;
  __syncthreads();
  double S = 0.0;
#pragma unroll
  for (int w = 0; w < NW; ++w) S += (double)s_f[w];
  const bool has_tail = s_head[2] < (double)V;
  const double mass = s_head[0];
  if (!a.t_lse && mass == 0.0) return clear();  // no entry to learn from
  // all against the larger of the two maxima (all -inf: NaN from here on)
  const double zt = (double)m * a.inv_tau, top = fmax(zt, s_head[3]);
  const double lse_t = S == 0.0 ? NEG_INF : (zt - top) + log(S);
  const double lse = log_add(lse_t, (s_head[3] - top) + s_head[1]);
  const double qt = has_tail ? exp(lse_t - lse) : 0.0;
  const double pt = a.t_lse && has_tail ? fmax(0.0, 1.0 - mass) : 0.0;
  const double M = mass + pt, g = c * a.inv_tau;
  if (wv == 0) {
    double kl = 0.0;
    for (int i = lane; i < K; i += 64)
      if (s_id[i] >= 0 && s_p[i] != NEG_INF) kl += exp(s_p[i]) * (s_p[i] - (s_z[i] - top) + lse);
    kl = wave_sum_d(kl);
    if (lane == 0) {
      if (pt > 0.0) kl += pt * (log(pt) - lse_t + lse);
      a.loss[t] = (float)(c * kl);
    }
  }
  if (!drow) return;
  __syncthreads();  // every read of the row that crosses threads is done
  const float f = (float)(S == 0.0 ? 0.0 * qt : g * (qt * M - pt) / S);
  for (int v = tid; v < V; v += DISTILL_THREADS)
    if (!((bits[v >> 5] >> (v & 31)) & 1u))
      elem<T>::store(drow, v, f * distill_exp(elem<T>::load(row, v), ms, a.c_hi, a.c_lo));
  for (int i = tid; i < K; i += DISTILL_THREADS) {
    if (!own(i)) continue;
    double p = exp(s_p[i]);
    if (s_dup)
      for (int j = i + 1; j < K; ++j)
        if (s_id[j] == s_id[i]) p += exp(s_p[j]);
    elem<T>::store(drow, s_id[i], (float)(g * (exp((s_z[i] - top) - lse) * M - p)));
  }
}

int64_t distill_ws_bytes(int T, int V) {
  (void)T;
  (void)V;
  return 0;
}

hipError_t launch_distill(int T, int V, int64_t ld, int K, const void* student, bool is_bf16,
                          const int32_t* ids, const float* t_logits, const float* t_lse,
                          const float* token_w, float tau, float scale, float* loss,
                          void* dstudent, void* ws, hipStream_t s) {
  (void)ws;
  const double c = 1.4426950408889634 / (double)tau;
  DistillArgs a{T, V, K, ld, ids, t_logits, t_lse, token_w, 1.0 / (double)tau, (float)c,
                (float)(c - (double)(float)c), scale, loss};
  const size_t lds = (size_t)K * 20 + (size_t)((V + 31) / 32) * 4;
  if (is_bf16)
    distill_kernel<bf16><<<T, DISTILL_THREADS, lds, s>>>(a, (const bf16*)student, (bf16*)dstudent);
  else
    distill_kernel<float><<<T, DISTILL_THREADS, lds, s>>>(a, (const float*)student,
                                                          (float*)dstudent);
  return hipGetLastError();
}

}  // namespace moe
