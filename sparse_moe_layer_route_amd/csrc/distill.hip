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
//
// The student's row is the traffic: read once, its gradient written once.
//   wave kernel   V <= 512 and K <= 64 (a router over its experts): one wave
//                 per row, the row in registers, no barriers.
//   block kernel  one block per row, which it holds in registers as loaded
//                 (bf16 stays packed) between the maximum, the sum and the
//                 gradient, so memory sees it once.  Exponentials are formed
//                 twice rather than kept: that would double the registers.
//   two launches  rows cut into segments, a block each, when the rows alone
//                 would not fill the GPU or are longer than a block holds: the
//                 first leaves each segment's sums in the workspace, the second
//                 joins them and reads its segment again.
// A row is walked in units of 16 bytes of memory, whatever its alignment; the
// elements of the first and last unit that belong to other rows, and the
// teacher's classes, are marked in a bitmap in LDS that the loops test a unit
// at a time.
#include <algorithm>
#include <cmath>

#include "common.h"

namespace moe {

constexpr double NEG_INF = -__builtin_huge_val();

struct DistillArgs {
  int T, V, K;
  int64_t ld;
  const int32_t* ids;
  const float* t_logits;
  const float* t_lse;    // may be null
  const float* token_w;  // may be null
  double inv_tau;
  float c_hi, c_lo;  // log2(e) / tau = c_hi + c_lo, c_lo > 0
  float scale;
  float* loss;
  int segs, seg_units;    // of a row; seg_units 16-byte units each
  struct SegStat* stats;  // [T][segs]
};

// What a segment of a row brings to the row's sums.
struct SegStat {
  float m, s;  // tail: maximum logit, sum of exp((logit - m) / tau)
  double zm, hs;  // teacher's classes: maximum z, sum of exp(z - zm), each class once
  double A, P;  // sum of p (log p - (z - ref)) with ref = zm (0 if that is -inf), sum of p
  double cnt;   // number of the teacher's classes
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
// s = -inf gives 0 (both parts of the factor are positive), NaN stays NaN.
__device__ __forceinline__ float distill_exp(float s, float m, const DistillArgs& a) {
  const float d = s - m;
  return __builtin_amdgcn_exp2f(fmaf(d, a.c_hi, d * a.c_lo));
}

__device__ __forceinline__ double log_add(double a, double b) {
  if (a != a || b != b) return a + b;  // fmax and fmin would drop a NaN
  const double hi = fmax(a, b), lo = fmin(a, b);
  return hi == NEG_INF ? hi : hi + log1p(exp(lo - hi));
}

// Everything the gradient needs of a row, and its loss.
struct RowResult {
  double top, lse;  // lse of z - top
  double M;
  float m, f;  // a tail class's gradient is f exp((logit - m) / tau)
  float loss;
};

// Joined sums of a row (every lane of the wave passes and gets the same).
//   m, S: tail; zm, hs: teacher's classes; A: sum of p (log p - (z - top))
__device__ __forceinline__ RowResult finish_row(const DistillArgs& a, double c, double mass, float m,
                                                double S, double zm, double hs, double A, double top,
                                                bool has_tail) {
  RowResult r;
  // all against the larger of the two maxima (all -inf: NaN from here on)
  const double zt = (double)m * a.inv_tau;
  const double lse_t = S == 0.0 ? NEG_INF : (zt - top) + log(S);
  const double lse_h = hs == 0.0 ? NEG_INF : (zm - top) + log(hs);
  const double lse = log_add(lse_t, lse_h);
  const double qt = has_tail ? exp(lse_t - lse) : 0.0;
  const double pt = a.t_lse && has_tail ? fmax(0.0, 1.0 - mass) : 0.0;
  double kl = A + mass * lse;
  if (pt > 0.0) kl += pt * (log(pt) - lse_t + lse);
  const double g = c * a.inv_tau;
  r.top = top;
  r.lse = lse;
  r.M = mass + pt;
  r.m = m == -__builtin_inff() ? 0.f : m;
  r.f = (float)(S == 0.0 ? 0.0 * qt : g * (qt * r.M - pt) / S);
  r.loss = (float)(c * kl);
  return r;
}

// ------------------------------------------------------ one wave per row ---
constexpr int DISTILL_WAVE_V = 512;  // 8 elements a lane
constexpr int DISTILL_WAVES = 4;     // rows of a block

template <typename T, int NE>
__global__ void __launch_bounds__(DISTILL_WAVES * MOE_WAVE)
distill_wave_kernel(DistillArgs a, const T* student, T* dstudent) {
  __shared__ uint32_t s_bits[DISTILL_WAVES][NE * 2];
  const int lane = lane_id(), wv = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * DISTILL_WAVES + wv;
  if (t >= a.T) return;  // no barrier below
  const T* row = student + t * a.ld;
  T* drow = dstudent ? dstudent + t * a.ld : nullptr;
  uint32_t* bits = s_bits[wv];
  const double c = (double)a.scale * (a.token_w ? (double)a.token_w[t] : 1.0);
  auto clear = [&] {
    if (lane == 0) a.loss[t] = 0.f;
    if (drow)
      for (int v = lane; v < a.V; v += 64) elem<T>::store(drow, v, 0.f);
  };
  if (c == 0.0) return clear();  // a masked row is not read
  float s[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int v = lane + 64 * i;
    s[i] = v < a.V ? elem<T>::load(row, v) : 0.f;
  }
  // lane k holds entry k
  const bool slot = lane < a.K;
  const int id = slot ? a.ids[t * a.K + lane] : -1;
  const double u = slot ? (double)a.t_logits[t * a.K + lane] * a.inv_tau : 0.0;
  const double t_lse = a.t_lse ? (double)a.t_lse[t] : 0.0;
  if (lane < NE * 2) bits[lane] = 0u;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  const bool ok = (unsigned)id < (unsigned)a.V;
  uint32_t old = 0u;
  if (ok) old = atomicOr(&bits[id >> 5], 1u << (id & 31));
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const bool dup = __any(ok && ((old >> (id & 31)) & 1u));
  const double z = ok ? (double)elem<T>::load(row, id) * a.inv_tau : NEG_INF;
  // own: the first entry of its class; more: the masses of the later ones
  bool own = ok;
  if (dup)
    for (int j = 0; j < a.K; ++j) {
      const int idj = __shfl(id, j);  // by the whole wave
      if (j < lane && idj == id) own = false;
    }
  // teacher: log p = (u - ref) - log_sum, in this order (beside a maximum of
  // the type's lowest value the logarithm would be lost)
  const double um = wave_max_d(ok ? u : NEG_INF);
  const bool has_p = ok && u != NEG_INF;
  double ref = t_lse, log_sum = 0.0;
  if (!a.t_lse) {
    ref = um;
    if (um > NEG_INF || um != um) log_sum = log(wave_sum_d(has_p ? exp(u - um) : 0.0));
  }
  const double lp = has_p ? (u - ref) - log_sum : NEG_INF;
  const double p = has_p ? exp(lp) : 0.0;
  const double mass = wave_sum_d(p);
  if (!a.t_lse && mass == 0.0) return clear();  // no entry to learn from
  double p_class = p;
  if (dup)
    for (int j = 0; j < a.K; ++j) {
      const double pj = __shfl(p, j);
      const int idj = __shfl(id, j);
      if (j != lane && idj == id) p_class += pj;
    }
  const double zm = wave_max_d(z);
  const double hs = wave_sum_d(own && z != NEG_INF ? exp(z - zm) : 0.0);
  const int cnt = __popcll(__ballot(own));
  // tail
  float m = -__builtin_inff(), sum = 0.f;
  bool tail[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int v = lane + 64 * i;
    tail[i] = v < a.V && !((bits[v >> 5] >> (v & 31)) & 1u);
    if (tail[i]) m = fmaxf(m, s[i]);
  }
  m = wave_max(m);
  const float ms = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    s[i] = tail[i] ? distill_exp(s[i], ms, a) : 0.f;
    sum += s[i];
  }
  const double S = (double)wave_sum(sum);
  const double top = fmax((double)m * a.inv_tau, zm);
  const double A = wave_sum_d(has_p ? p * (lp - (z - top)) : 0.0);
  const RowResult r = finish_row(a, c, mass, m, S, zm, hs, A, top, cnt < a.V);
  if (lane == 0) a.loss[t] = r.loss;
  if (!drow) return;
#pragma unroll
  for (int i = 0; i < NE; ++i)
    if (tail[i]) elem<T>::store(drow, lane + 64 * i, r.f * s[i]);
  if (own)
    elem<T>::store(drow, id, (float)(c * a.inv_tau * (exp((z - r.top) - r.lse) * r.M - p_class)));
}

// ------------------------------------------------- one block per segment ---
template <typename T> struct raw_unit {
  static constexpr int EPU = 16 / sizeof(T);  // elements of a unit
};
__device__ __forceinline__ float unit_elem(const uint4& v, int i, bf16) {
  const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
  return i & 1 ? bf16_hi(w) : bf16_lo(w);
}
__device__ __forceinline__ float unit_elem(const uint4& v, int i, float) {
  return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
}
__device__ __forceinline__ uint4 make_unit(const float (&o)[8], bf16) {
  return make_uint4(f2_to_bf16x2(o[0], o[1]), f2_to_bf16x2(o[2], o[3]), f2_to_bf16x2(o[4], o[5]),
                    f2_to_bf16x2(o[6], o[7]));
}
__device__ __forceinline__ uint4 make_unit(const float (&o)[4], float) {
  return make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]),
                    __float_as_uint(o[3]));
}

enum { DISTILL_ROW = 0, DISTILL_STATS = 1, DISTILL_GRAD = 2 };

// Segment blockIdx.x of row blockIdx.y (DISTILL_ROW: row blockIdx.x), NT
// threads of at most NU units each.
template <typename T, int NT, int NU, int PHASE>
__global__ void __launch_bounds__(NT)
distill_block_kernel(DistillArgs a, const T* student, T* dstudent) {
  constexpr int EPU = raw_unit<T>::EPU, NW = NT / MOE_WAVE;
  constexpr uint32_t ALL = (1u << EPU) - 1u;
  extern __shared__ double smem[];
  const int K = a.K, V = a.V, tid = threadIdx.x, lane = lane_id(), wv = tid >> 6;
  double* s_lp = smem;                   // [K] log p
  double* s_z = s_lp + K;                // [K] z of this segment's entries
  int32_t* s_id = (int32_t*)(s_z + K);   // [K] class, -1 where skipped
  uint32_t* bits = (uint32_t*)(s_id + K);  // this segment's marked elements
  __shared__ int s_dup;
  __shared__ float s_max[NW], s_sum[NW];
  __shared__ double s_mass;
  __shared__ SegStat s_stat;
  __shared__ RowResult s_row;
  const int64_t t = PHASE == DISTILL_ROW ? blockIdx.x : blockIdx.y;
  const int seg = PHASE == DISTILL_ROW ? 0 : blockIdx.x;
  const T* row = student + t * a.ld;
  T* drow = dstudent ? dstudent + t * a.ld : nullptr;
  // unit u holds elements u * EPU - ph .. +EPU-1 of the row
  const int ph = (int)((t * a.ld) & (EPU - 1));
  const int u0 = seg * a.seg_units, u1 = min(u0 + a.seg_units, (V + ph + EPU - 1) / EPU);
  const int n_units = max(u1 - u0, 0);
  const double c = (double)a.scale * (a.token_w ? (double)a.token_w[t] : 1.0);
  auto whole = [&](int u) { return u * EPU >= ph && (u + 1) * EPU <= V + ph; };
  auto clear = [&] {
    if (PHASE == DISTILL_STATS) return;
    if (tid == 0 && seg == 0) a.loss[t] = 0.f;
    if (!drow) return;
    for (int u = u0 + tid; u < u1; u += NT) {
      if (whole(u))
        *reinterpret_cast<uint4*>(drow + (u * EPU - ph)) = make_uint4(0u, 0u, 0u, 0u);
      else
        for (int v = max(u * EPU - ph, 0); v < min((u + 1) * EPU - ph, V); ++v)
          elem<T>::store(drow, v, 0.f);
    }
  };
  if (c == 0.0) return clear();  // a masked row is not read
  uint4 x[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = u0 + i * NT + tid;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (u >= u1) continue;
    if (whole(u)) {
      x[i] = *reinterpret_cast<const uint4*>(row + (u * EPU - ph));
    } else {  // the elements of other rows are marked below
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < EPU; ++e) {
        const int v = u * EPU - ph + e;
        if (v < 0 || v >= V) continue;
        if (sizeof(T) == 2)
          w[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[v] << (16 * (e & 1));
        else
          w[e] = reinterpret_cast<const uint32_t*>(row)[v];
      }
      x[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if (tid == 0) s_dup = 0;
  for (int i = tid; i < (n_units * EPU + 31) / 32; i += NT) bits[i] = 0u;
  __syncthreads();
  // bit of element v: v + ph - u0 * EPU
  const int b0 = u0 * EPU - ph, nb = n_units * EPU;
  for (int i = tid; i < K; i += NT) {
    const int id = a.ids[t * K + i];
    const bool ok = (unsigned)id < (unsigned)V;
    s_id[i] = ok ? id : -1;
    s_lp[i] = (double)a.t_logits[t * K + i] * a.inv_tau;
    const int b = id - b0;
    if (ok && b >= 0 && b < nb) {
      const uint32_t bit = 1u << (b & 31);
      if (atomicOr(&bits[b >> 5], bit) & bit) s_dup = 1;
      s_z[i] = (double)elem<T>::load(row, id) * a.inv_tau;
    }
  }
  // the elements of other rows in the first and the last unit
  if (tid < EPU && n_units > 0) {
    if (tid < -b0) atomicOr(&bits[0], 1u << tid);
    const int b = nb - EPU + tid;
    if (b + b0 >= V) atomicOr(&bits[b >> 5], 1u << (b & 31));
  }
  __syncthreads();
  auto here = [&](int i) { return s_id[i] >= 0 && s_id[i] >= b0 && s_id[i] < b0 + nb; };
  auto own = [&](int i) {  // the first entry of its class
    if (s_dup)
      for (int j = 0; j < i; ++j)
        if (s_id[j] == s_id[i]) return false;
    return true;
  };
  auto marks = [&](int i) -> uint32_t {  // of the thread's unit i
    const int q = (i * NT + tid) * EPU;
    return (bits[q >> 5] >> (q & 31)) & ALL;
  };
  if (wv == 0) {
    double um = NEG_INF;
    for (int i = lane; i < K; i += 64)
      if (s_id[i] >= 0) um = fmax(um, s_lp[i]);
    um = wave_max_d(um);
    // log p = (u - ref) - log_sum, in this order: beside a maximum of the
    // type's lowest value the logarithm would be lost
    double ref = um, log_sum = 0.0;
    if (a.t_lse) {
      ref = (double)a.t_lse[t];
    } else {
      double e = 0.0;
      for (int i = lane; i < K; i += 64)
        if (s_id[i] >= 0 && s_lp[i] != NEG_INF) e += exp(s_lp[i] - um);
      log_sum = log(wave_sum_d(e));
    }
    double mass = 0.0, zm = NEG_INF;
    for (int i = lane; i < K; i += 64) {
      if (s_id[i] < 0) continue;
      s_lp[i] = s_lp[i] == NEG_INF ? NEG_INF : (s_lp[i] - ref) - log_sum;
      mass += exp(s_lp[i]);
      if (here(i)) zm = fmax(zm, s_z[i]);
    }
    mass = wave_sum_d(mass);
    if (lane == 0) s_mass = mass;
    if (PHASE != DISTILL_GRAD) {
      zm = wave_max_d(zm);
      const double zr = zm == NEG_INF ? 0.0 : zm;
      double hs = 0.0, A = 0.0, P = 0.0, cnt = 0.0;
      for (int i = lane; i < K; i += 64) {
        if (!here(i)) continue;
        if (own(i)) {
          cnt += 1.0;
          if (s_z[i] != NEG_INF) hs += exp(s_z[i] - zm);
        }
        if (s_lp[i] != NEG_INF) {
          const double p = exp(s_lp[i]);
          P += p;
          A += p * (s_lp[i] - (s_z[i] - zr));
        }
      }
      hs = wave_sum_d(hs);
      A = wave_sum_d(A);
      P = wave_sum_d(P);
      cnt = wave_sum_d(cnt);
      if (lane == 0) {
        s_stat.zm = zm;
        s_stat.hs = hs;
        s_stat.A = A;
        s_stat.P = P;
        s_stat.cnt = cnt;
      }
    }
  }
  if (PHASE != DISTILL_GRAD) {
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (u0 + i * NT + tid >= u1) continue;
      const uint32_t k = marks(i);
      if (k == 0u) {
#pragma unroll
        for (int e = 0; e < EPU; ++e) m = fmaxf(m, unit_elem(x[i], e, T{}));
      } else {
#pragma unroll
        for (int e = 0; e < EPU; ++e)
          if (!((k >> e) & 1u)) m = fmaxf(m, unit_elem(x[i], e, T{}));
      }
    }
    m = wave_max(m);
    if (lane == 0) s_max[wv] = m;
    __syncthreads();
    m = s_max[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) m = fmaxf(m, s_max[w]);
    const float ms = m == -__builtin_inff() ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (u0 + i * NT + tid >= u1) continue;
      const uint32_t k = marks(i);
      if (k == 0u) {
#pragma unroll
        for (int e = 0; e < EPU; ++e) sum += distill_exp(unit_elem(x[i], e, T{}), ms, a);
      } else {
#pragma unroll
        for (int e = 0; e < EPU; ++e)
          if (!((k >> e) & 1u)) sum += distill_exp(unit_elem(x[i], e, T{}), ms, a);
      }
    }
    sum = wave_sum(sum);
    if (lane == 0) s_sum[wv] = sum;
    __syncthreads();
    if (tid == 0) {
      double S = 0.0;
#pragma unroll
      for (int w = 0; w < NW; ++w) S += (double)s_sum[w];
      s_stat.m = m;
      s_stat.s = (float)S;
      if (PHASE == DISTILL_STATS) a.stats[t * a.segs + seg] = s_stat;
    }
    if (PHASE == DISTILL_STATS) return;
  }
  __syncthreads();
  const double mass = s_mass;
  if (!a.t_lse && mass == 0.0) return clear();  // no entry to learn from
  if (wv == 0) {
    // join the segments (one: the block's own)
    const SegStat* st = PHASE == DISTILL_ROW ? &s_stat : a.stats + t * a.segs;
    const int n = PHASE == DISTILL_ROW ? 1 : a.segs;
    float m = -__builtin_inff();
    double zm = NEG_INF;
    for (int i = lane; i < n; i += 64) {
      m = fmaxf(m, st[i].m);
      zm = fmax(zm, st[i].zm);
    }
    m = wave_max(m);
    zm = wave_max_d(zm);
    const double top = fmax((double)m * a.inv_tau, zm);
    double S = 0.0, hs = 0.0, A = 0.0, cnt = 0.0;
    for (int i = lane; i < n; i += 64) {
      const SegStat q = st[i];
      if (q.s != 0.f) S += (double)q.s * exp(((double)q.m - (double)m) * a.inv_tau);
      if (q.hs != 0.0) hs += q.hs * exp(q.zm - zm);
      if (q.P != 0.0) A += q.A - q.P * ((q.zm == NEG_INF ? 0.0 : q.zm) - top);
      cnt += q.cnt;
    }
    S = wave_sum_d(S);
    hs = wave_sum_d(hs);
    A = wave_sum_d(A);
    cnt = wave_sum_d(cnt);
    const RowResult r = finish_row(a, c, mass, m, S, zm, hs, A, top, cnt < (double)V);
    if (lane == 0) {
      s_row = r;
      if (seg == 0) a.loss[t] = r.loss;
    }
  }
  if (!drow) return;
  __syncthreads();
  const RowResult r = s_row;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = u0 + i * NT + tid;
    if (u >= u1) continue;
    const uint32_t k = marks(i);
    float o[EPU];
#pragma unroll
    for (int e = 0; e < EPU; ++e) o[e] = r.f * distill_exp(unit_elem(x[i], e, T{}), r.m, a);
    if (k == 0u) {
      *reinterpret_cast<uint4*>(drow + (u * EPU - ph)) = make_unit(o, T{});
    } else {
#pragma unroll
      for (int e = 0; e < EPU; ++e)
        if (!((k >> e) & 1u)) elem<T>::store(drow, u * EPU - ph + e, o[e]);
    }
  }
  for (int i = tid; i < K; i += NT) {
    if (!here(i) || !own(i)) continue;
    double p = exp(s_lp[i]);
    if (s_dup)
      for (int j = i + 1; j < K; ++j)
        if (s_id[j] == s_id[i]) p += exp(s_lp[j]);
    elem<T>::store(drow, s_id[i],
                   (float)(c * a.inv_tau * (exp((s_z[i] - r.top) - r.lse) * r.M - p)));
  }
}

// Segments of a call's rows: 1 when a block holds a row and the rows fill the
// GPU, or a row is too short to be worth two launches.
constexpr int SEG_NT = 256, SEG_NU = 8;
constexpr int ROW_UNITS = 1024 * 16;  // of the largest one-block kernel
#ifndef DISTILL_FILL
#define DISTILL_FILL 256
#endif
#ifndef DISTILL_SEG_BLOCKS
#define DISTILL_SEG_BLOCKS 512
#endif
#ifndef DISTILL_SPLIT_UNITS
#define DISTILL_SPLIT_UNITS 4096
#endif

static void distill_segments(int T, int units, int* segs, int* seg_units) {
  *segs = 1;
  *seg_units = units;
  if (units <= ROW_UNITS && (T >= DISTILL_FILL || units < DISTILL_SPLIT_UNITS)) return;
  const int64_t want = ((int64_t)T * units + DISTILL_SEG_BLOCKS - 1) / DISTILL_SEG_BLOCKS;
  const int64_t per = (want + SEG_NT - 1) / SEG_NT * SEG_NT;
  *seg_units = (int)std::min<int64_t>(std::max<int64_t>(per, SEG_NT), SEG_NT * SEG_NU);
  *segs = (units + *seg_units - 1) / *seg_units;
}

// Most units a row of V elements of `bytes` can touch.
static int row_units(int V, int bytes) {
  const int epu = 16 / bytes;
  return (V + epu - 1 + epu - 1) / epu;
}

int64_t distill_ws_bytes(int T, int V) {
  int64_t most = 0;
  for (int bytes = 2; bytes <= 4; bytes += 2) {
    int segs, seg_units;
    distill_segments(T, row_units(V, bytes), &segs, &seg_units);
    if (segs > 1) most = std::max<int64_t>(most, (int64_t)T * segs * (int64_t)sizeof(SegStat));
  }
  return most;
}

template <typename T, int NT, int NU, int PHASE>
static void block_launch(const DistillArgs& a, dim3 grid, const T* student, T* dstudent, hipStream_t s) {
  const size_t lds = (size_t)a.K * 20 + (size_t)(a.seg_units * raw_unit<T>::EPU + 31) / 32 * 4;
  distill_block_kernel<T, NT, NU, PHASE><<<grid, NT, lds, s>>>(a, student, dstudent);
}

template <typename T>
static hipError_t distill_t(DistillArgs a, const T* student, T* dstudent, void* ws, hipStream_t s) {
  if (a.V <= DISTILL_WAVE_V && a.K <= MOE_WAVE) {
    const int grid = (a.T + DISTILL_WAVES - 1) / DISTILL_WAVES, thr = DISTILL_WAVES * MOE_WAVE;
    if (a.V <= 64)
      distill_wave_kernel<T, 1><<<grid, thr, 0, s>>>(a, student, dstudent);
    else
      distill_wave_kernel<T, 8><<<grid, thr, 0, s>>>(a, student, dstudent);
    return hipGetLastError();
  }
  const int units = row_units(a.V, sizeof(T));
  distill_segments(a.T, units, &a.segs, &a.seg_units);
  if (a.segs > 1) {
    a.stats = (SegStat*)ws;
    // rows on the grid's second axis, a bounded number of them a launch
    constexpr int MAX_Y = 32768;
    for (int t0 = 0; t0 < a.T; t0 += MAX_Y) {
      DistillArgs b = a;
      const int n = std::min(MAX_Y, a.T - t0);
      b.T = n;
      b.ids += (int64_t)t0 * a.K;
      b.t_logits += (int64_t)t0 * a.K;
      if (b.t_lse) b.t_lse += t0;
      if (b.token_w) b.token_w += t0;
      b.loss += t0;
      b.stats += (int64_t)t0 * a.segs;
      const int64_t at = (int64_t)t0 * a.ld;
      block_launch<T, SEG_NT, SEG_NU, DISTILL_STATS>(b, dim3(a.segs, n), student + at, nullptr, s);
      hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      block_launch<T, SEG_NT, SEG_NU, DISTILL_GRAD>(b, dim3(dstudent ? a.segs : 1, n), student + at,
                                                    dstudent ? dstudent + at : nullptr, s);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
  }
  if (units <= 256 * 4)
    block_launch<T, 256, 4, DISTILL_ROW>(a, a.T, student, dstudent, s);
  else if (units <= 256 * 16)
    block_launch<T, 256, 16, DISTILL_ROW>(a, a.T, student, dstudent, s);
  else
    block_launch<T, 1024, 16, DISTILL_ROW>(a, a.T, student, dstudent, s);
  return hipGetLastError();
}

hipError_t launch_distill(int T, int V, int64_t ld, int K, const void* student, bool is_bf16,
                          const int32_t* ids, const float* t_logits, const float* t_lse,
                          const float* token_w, float tau, float scale, float* loss,
                          void* dstudent, void* ws, hipStream_t s) {
  const double c = 1.4426950408889634 / (double)tau;
  float hi = (float)c;
  if ((double)hi >= c) hi = std::nextafter(hi, 0.f);
  DistillArgs a{T, V, K, ld, ids, t_logits, t_lse, token_w, 1.0 / (double)tau, hi,
                (float)(c - (double)hi), scale, loss, 1, 0, nullptr};
  if (is_bf16) return distill_t(a, (const bf16*)student, (bf16*)dstudent, ws, s);
  return distill_t(a, (const float*)student, (float*)dstudent, ws, s);
}

}  // namespace moe
