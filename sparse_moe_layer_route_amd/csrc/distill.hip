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
//   group kernel  short rows (a router over its experts): 16 or 64 lanes per
//                 row, the row in registers, no barriers.
//   block kernel  one block per row, which it holds in registers between the
//                 maximum, the sum and the gradient, so memory sees it once.
//   two launches  rows cut into segments, a block each, when the rows alone
//                 would not fill the GPU or are longer than a block holds: the
//                 first leaves each segment's sums in the workspace, the second
//                 joins them and reads its segment again.
// A block walks a row in units of 16 bytes of memory, whatever its alignment.
// The teacher's classes, and the elements of other rows in the first and last
// unit, are set to -inf in the registers before the passes, which then need no
// tests; the teacher's classes get their own gradient after a barrier.
#include <algorithm>

#include "common.h"

// z = logit / tau is compared and subtracted in several places: as a rounded
// value, the same in all of them.  Fused into a subtraction its rounding error
// would be left over, which beside logits of the type's lowest value is huge.
#pragma clang fp contract(off)

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
  float c;  // log2(e) / tau
  float scale;
  float* loss;
  int segs, seg_units;    // of a row; seg_units 16-byte units each
  struct SegStat* stats;  // [T][segs]
};

// What a segment of a row brings to the row's sums.  e = exp(d) is a teacher's
// entry before it is normalised: d = u / tau minus the entries' largest (minus
// lse_teacher where that is given, and e is p).
struct SegStat {
  float m, s;  // tail: maximum logit, sum of exp((logit - m) / tau)
  double zm, hs;  // teacher's classes: maximum z, sum of exp(z - zm), each class once
  double A, P;  // sum of e (d - (z - ref)) with ref = zm (0 if that is -inf), sum of e
  int cnt;      // number of the teacher's classes
};

// The wave reductions of common.h on doubles, a half at a time.
template <int CTRL, int ROWS, bool BOUND_ZERO>
__device__ __forceinline__ double dpp_move_d(double old, double v) {
  const int2 o = __builtin_bit_cast(int2, old), x = __builtin_bit_cast(int2, v);
  return __builtin_bit_cast(double, int2{dpp_move<CTRL, ROWS, BOUND_ZERO>(o.x, x.x),
                                         dpp_move<CTRL, ROWS, BOUND_ZERO>(o.y, x.y)});
}
__device__ __forceinline__ double lane63_d(double v) {
  const int2 x = __builtin_bit_cast(int2, v);
  return __builtin_bit_cast(double, int2{__builtin_amdgcn_readlane(x.x, 63),
                                         __builtin_amdgcn_readlane(x.y, 63)});
}
__device__ __forceinline__ double wave_sum_d(double v) {
  v += dpp_move_d<0x111, 0xf, true>(0.0, v);
  v += dpp_move_d<0x112, 0xf, true>(0.0, v);
  v += dpp_move_d<0x114, 0xf, true>(0.0, v);
  v += dpp_move_d<0x118, 0xf, true>(0.0, v);
  v += dpp_move_d<0x142, 0xa, false>(0.0, v);
  v += dpp_move_d<0x143, 0xc, false>(0.0, v);
  return lane63_d(v);
}
__device__ __forceinline__ double wave_max_d(double v) {
  v = fmax(v, dpp_move_d<0x111, 0xf, false>(v, v));
  v = fmax(v, dpp_move_d<0x112, 0xf, false>(v, v));
  v = fmax(v, dpp_move_d<0x114, 0xf, false>(v, v));
  v = fmax(v, dpp_move_d<0x118, 0xf, false>(v, v));
  v = fmax(v, dpp_move_d<0x142, 0xa, false>(v, v));
  v = fmax(v, dpp_move_d<0x143, 0xc, false>(v, v));
  return lane63_d(v);
}

// exp((s - m) / tau).  The difference first: s and m of the type's lowest value
// then still give 1, and the rounding of the factor counts by |s - m| only.
__device__ __forceinline__ float distill_exp(float s, float m, const DistillArgs& a) {
  return __builtin_amdgcn_exp2f((s - m) * a.c);
}

// Everything the gradient needs of a row, and its loss.
struct RowResult {
  double zm, qh;  // a teacher's class: q = exp(z - zm) qh
  double M, norm;  // p = e norm
  float m, f;  // a tail class's gradient is f exp((logit - m) / tau)
  float loss;
};

// From the joined sums of a row: sum of e; m, S of the tail; zm, hs of the
// teacher's classes; A = sum of e (d - (z - top)), top = max(m / tau, zm).  All is
// taken relative to top, and log p = d - log(sum) in this order: beside a
// maximum of the type's lowest value a logarithm would be lost.  All -inf: NaN
// from here on.
// The row's values are in every lane; of two exponentials, three quotients and
// two logarithms each lane of four takes one: one call of each in the chain that
// the row's other waves wait for.
__device__ __forceinline__ RowResult finish_row(const DistillArgs& a, double c, double sum, float m,
                                                double S, double zm, double hs, double A, double top,
                                                bool has_tail) {
  RowResult r;
  const int l = threadIdx.x & 3;
  auto lane0 = [](double v) { return dpp_move_d<0x00, 0xf, false>(v, v); };  // quad_perm 0,0,0,0
  auto lane1 = [](double v) { return dpp_move_d<0x55, 0xf, false>(v, v); };  // quad_perm 1,1,1,1
  auto lane2 = [](double v) { return dpp_move_d<0xAA, 0xf, false>(v, v); };  // quad_perm 2,2,2,2
  const double dt = (double)m * a.inv_tau - top;
  const double ev = exp(l == 0 ? dt : zm - top);
  const double et = lane0(ev), eh = lane1(ev), W = S * et + hs * eh;
  const double iv = 1.0 / (l == 0 ? W : l == 1 ? S : sum);
  const double iW = lane0(iv), iS = lane1(iv);
  r.norm = a.t_lse ? 1.0 : lane2(iv);
  const double mass = sum * r.norm;
  const double pt = a.t_lse && has_tail ? fmax(0.0, 1.0 - mass) : 0.0;
  const double lv = log(l == 0 ? W : a.t_lse ? pt * W * iS : sum);
  const double lW = lane0(lv), l1 = lane1(lv);
  double kl = A * r.norm + mass * lW;
  if (!a.t_lse) kl -= mass * l1;
  if (pt > 0.0) kl += pt * (l1 - dt);
  const double g = c * a.inv_tau;
  r.zm = zm;
  r.qh = eh * iW;
  r.M = mass + pt;
  r.m = m == -__builtin_inff() ? 0.f : m;
  r.f = (float)(S == 0.0 ? 0.0 * W : g * (r.M * et * iW - pt * iS));
  r.loss = (float)(c * kl);
  return r;
}
// Gradient of a teacher's class: ez = exp(z - zm), p its entries' mass.
__device__ __forceinline__ float head_grad(const DistillArgs& a, double c, const RowResult& r, double ez,
                                           double p) {
  return (float)(c * a.inv_tau * (ez * r.qh * r.M - p));
}

// --------------------------------------------- a group of lanes per row ---
// Reductions over groups of 16 or 64 lanes, the result in every lane.  Within
// 16: exchanges by 1, 2, then mirrored halves and rows.
template <int G> __device__ __forceinline__ double group_sum_d(double v) {
  if (G == 64) return wave_sum_d(v);
  v += dpp_move_d<0xB1, 0xf, false>(v, v);   // quad_perm 1,0,3,2
  v += dpp_move_d<0x4E, 0xf, false>(v, v);   // quad_perm 2,3,0,1
  v += dpp_move_d<0x141, 0xf, false>(v, v);  // row_half_mirror
  v += dpp_move_d<0x140, 0xf, false>(v, v);  // row_mirror
  return v;
}
template <int G> __device__ __forceinline__ double group_max_d(double v) {
  if (G == 64) return wave_max_d(v);
  v = fmax(v, dpp_move_d<0xB1, 0xf, false>(v, v));
  v = fmax(v, dpp_move_d<0x4E, 0xf, false>(v, v));
  v = fmax(v, dpp_move_d<0x141, 0xf, false>(v, v));
  v = fmax(v, dpp_move_d<0x140, 0xf, false>(v, v));
  return v;
}
template <int CTRL> __device__ __forceinline__ float dpp_move_f(float v) {
  const int x = __float_as_int(v);
  return __int_as_float(dpp_move<CTRL, 0xf, false>(x, x));
}
template <int G> __device__ __forceinline__ float group_max(float v) {
  if (G == 64) return wave_max(v);
  v = fmaxf(v, dpp_move_f<0xB1>(v));
  v = fmaxf(v, dpp_move_f<0x4E>(v));
  v = fmaxf(v, dpp_move_f<0x141>(v));
  return fmaxf(v, dpp_move_f<0x140>(v));
}
template <int G> __device__ __forceinline__ float group_sum(float v) {
  if (G == 64) return wave_sum(v);
  v += dpp_move_f<0xB1>(v);
  v += dpp_move_f<0x4E>(v);
  v += dpp_move_f<0x141>(v);
  return v + dpp_move_f<0x140>(v);
}

constexpr int GROUP_THREADS = 256;

// Rows of at most G * NE classes and G teacher entries, G lanes each.  4096 x 40
// fp32, 8 entries (1.6 MB): 4.5 us, a launch and one chain of a row's steps;
// 16384 x 500 bf16, 40 entries: 25 us, bound by some 800 vector instructions a
// row, half of them the entries' 64-bit steps.
template <typename T, int G, int NE>
__global__ void __launch_bounds__(GROUP_THREADS)
distill_group_kernel(DistillArgs a, const T* student, T* dstudent) {
  constexpr int ROWS = GROUP_THREADS / G, WORDS = (G * NE + 31) / 32;
  __shared__ uint32_t s_bits[ROWS][WORDS];
  const int l = threadIdx.x % G, base = lane_id() - l;  // lane in the group, its first lane
  const int64_t t = (int64_t)blockIdx.x * ROWS + threadIdx.x / G;
  if (t >= a.T) return;  // no barrier below, and no exchange between groups
  const T* row = student + t * a.ld;
  T* drow = dstudent ? dstudent + t * a.ld : nullptr;
  uint32_t* bits = s_bits[threadIdx.x / G];
  const double c = (double)a.scale * (a.token_w ? (double)a.token_w[t] : 1.0);
  auto clear = [&] {
    if (l == 0) a.loss[t] = 0.f;
    if (drow)
      for (int v = l; v < a.V; v += G) elem<T>::store(drow, v, 0.f);
  };
  if (c == 0.0) return clear();  // a masked row is not read
  float s[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int v = l + G * i;
    s[i] = v < a.V ? elem<T>::load(row, v) : 0.f;
  }
  // lane k holds entry k
  const bool slot = l < a.K;
  const int id = slot ? a.ids[t * a.K + l] : -1;
  const double u = slot ? (double)a.t_logits[t * a.K + l] * a.inv_tau : 0.0;
  const double t_lse = a.t_lse ? (double)a.t_lse[t] : 0.0;
  for (int i = l; i < WORDS; i += G) bits[i] = 0u;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  const bool ok = (unsigned)id < (unsigned)a.V;
  uint32_t old = 0u;
  if (ok) old = atomicOr(&bits[id >> 5], 1u << (id & 31));
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const bool dup = __any(ok && ((old >> (id & 31)) & 1u));
  const double z = ok ? (double)elem<T>::load(row, id) * a.inv_tau : NEG_INF;
  // own: the first entry of its class
  bool own = ok;
  if (dup)
    for (int j = 0; j < a.K; ++j) {
      const int idj = __shfl(id, base + j);  // by the whole group
      if (j < l && idj == id) own = false;
    }
  const bool has_p = ok && u != NEG_INF;
  const double d = u - (a.t_lse ? t_lse : group_max_d<G>(ok ? u : NEG_INF));
  const double e = has_p ? exp(d) : 0.0, psum = group_sum_d<G>(e);
  if (!a.t_lse && psum == 0.0) return clear();  // no entry to learn from
  double e_class = e;
  if (dup)
    for (int j = 0; j < a.K; ++j) {
      const double ej = __shfl(e, base + j);
      const int idj = __shfl(id, base + j);
      if (j != l && idj == id) e_class += ej;
    }
  const double zm = group_max_d<G>(z);
  const double ez = z != NEG_INF ? exp(z - zm) : 0.0;
  const double hs = group_sum_d<G>(own ? ez : 0.0);
  const int cnt = __popcll((__ballot(own) >> base) & (~0ull >> (64 - G)));
  // tail
  float m = -__builtin_inff(), sum = 0.f;
  bool tail[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int v = l + G * i;
    tail[i] = v < a.V && !((bits[v >> 5] >> (v & 31)) & 1u);
    if (tail[i]) m = fmaxf(m, s[i]);
  }
  m = group_max<G>(m);
  const float ms = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    s[i] = tail[i] ? distill_exp(s[i], ms, a) : 0.f;
    sum += s[i];
  }
  const double S = (double)group_sum<G>(sum);
  const double top = fmax((double)m * a.inv_tau, zm);
  // an entry whose p underflows counts nothing, whatever the student says (0 * inf)
  const double A = group_sum_d<G>(e != 0.0 ? e * (d - (z - top)) : 0.0);
  const RowResult r = finish_row(a, c, psum, m, S, zm, hs, A, top, cnt < a.V);
  if (l == 0) a.loss[t] = r.loss;
  if (!drow) return;
#pragma unroll
  for (int i = 0; i < NE; ++i)
    if (tail[i]) elem<T>::store(drow, l + G * i, r.f * s[i]);
  if (own) elem<T>::store(drow, id, head_grad(a, c, r, ez, e_class * r.norm));
}

// ------------------------------------------------- one block per segment ---
template <typename T> struct raw_unit {
  static constexpr int EPU = 16 / sizeof(T);  // elements of a unit
};
__device__ __forceinline__ uint32_t unit_word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ float unit_elem(const uint4& v, int i, bf16) {
  return i & 1 ? bf16_hi(unit_word(v, i >> 1)) : bf16_lo(unit_word(v, i >> 1));
}
__device__ __forceinline__ float unit_elem(const uint4& v, int i, float) {
  return __uint_as_float(unit_word(v, i));
}
__device__ __forceinline__ uint4 make_unit(const float (&o)[8], bf16) {
  return make_uint4(f2_to_bf16x2(o[0], o[1]), f2_to_bf16x2(o[2], o[3]), f2_to_bf16x2(o[4], o[5]),
                    f2_to_bf16x2(o[6], o[7]));
}
__device__ __forceinline__ uint4 make_unit(const float (&o)[4], float) {
  return make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]),
                    __float_as_uint(o[3]));
}
// -inf into the elements whose bit is set.
__device__ __forceinline__ uint32_t mask_word(uint32_t w, uint32_t k, bf16) {
  if (k & 1u) w = (w & 0xFFFF0000u) | 0xFF80u;
  if (k & 2u) w = (w & 0xFFFFu) | 0xFF800000u;
  return w;
}
__device__ __forceinline__ uint32_t mask_word(uint32_t w, uint32_t k, float) {
  return (k & 1u) ? 0xFF800000u : w;
}
template <typename T> __device__ __forceinline__ uint4 mask_unit(const uint4& v, uint32_t k) {
  constexpr int PER = 4 / sizeof(T);  // elements of a word
  return make_uint4(mask_word(v.x, k, T{}), mask_word(v.y, k >> PER, T{}),
                    mask_word(v.z, k >> (2 * PER), T{}), mask_word(v.w, k >> (3 * PER), T{}));
}

enum { DISTILL_ROW = 0, DISTILL_STATS = 1, DISTILL_GRAD = 2 };

// Maximum of a thread's units.  bf16 pairs are compared as they are stored:
// as signed integers positive values keep their order and beat negative ones,
// so the result is the maximum wherever it is not negative (a NaN of positive
// sign comes out, and through; a negative one reaches the sum).
template <int NU> __device__ __forceinline__ float units_max(const uint4 (&x)[NU], float) {
  float m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) m = fmaxf(m, unit_elem(x[i], e, 0.f));
  return m;
}
template <int NU> __device__ __forceinline__ float units_max(const uint4 (&x)[NU], bf16) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  s16x2 k = {-32768, -32768};
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int w = 0; w < 4; ++w)
      k = __builtin_elementwise_max(k, __builtin_bit_cast(s16x2, unit_word(x[i], w)));
  const int b = max((int)k.x, (int)k.y);
  if (b >= 0) return bf16_to_f((uint16_t)b);
  float m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, unit_elem(x[i], e, bf16{}));
  return m;
}

// Segment blockIdx.x of row blockIdx.y (DISTILL_ROW: row blockIdx.x), NT
// threads of at most NU units each.  OCC: waves a SIMD should hold.
// 2048 x 32000 bf16, 64 entries, a tenth of the rows masked (250 MB): 59 us over
// changing inputs, 4.2 TB/s (50 replayed on one set, part of which stays in the
// caches); vector instructions (15 an element) are issued in half of a CU's busy
// cycles, beside the loads and stores of other rows.  Cut rows, 7 x 100003 fp32: 11.2 us, two launches.
template <typename T, int NT, int NU, int PHASE, int OCC>
__global__ void __launch_bounds__(NT, OCC)
distill_block_kernel(DistillArgs a, const T* student, T* dstudent) {
  constexpr int EPU = raw_unit<T>::EPU, NW = NT / MOE_WAVE;
  constexpr uint32_t ALL = (1u << EPU) - 1u;
  // the sum's exponentials are kept for the gradient where they fit
  constexpr bool KEEP = PHASE == DISTILL_ROW && NU * EPU <= 64;
  extern __shared__ double smem[];
  const int K = a.K, V = a.V, tid = threadIdx.x, lane = lane_id(), wv = tid >> 6;
  double* s_e = smem;                    // [K] the teacher's u / tau, then e
  double* s_z = s_e + K;                 // [K] this segment's entries: z, then exp(z - zm)
  int32_t* s_id = (int32_t*)(s_z + K);   // [K] class, -1 where skipped
  uint32_t* bits = (uint32_t*)(s_id + K);  // this segment's marked elements
  __shared__ int s_dup;
  __shared__ float s_max[NW], s_sum[NW];
  __shared__ double s_psum;
  __shared__ SegStat s_stat;
  __shared__ RowResult s_row;
  const int64_t t = PHASE == DISTILL_ROW ? blockIdx.x : blockIdx.y;
  const int seg = PHASE == DISTILL_ROW ? 0 : blockIdx.x;
  const T* row = student + t * a.ld;
  T* drow = dstudent ? dstudent + t * a.ld : nullptr;
  // unit u holds elements u * EPU - ph .. +EPU-1 of the row; the first and the
  // last may hold elements of other rows too
  const int ph = (int)((t * a.ld) & (EPU - 1));
  const int all_units = (V + ph + EPU - 1) / EPU;
  const int u0 = seg * a.seg_units, u1 = min(u0 + a.seg_units, all_units);
  const int n_units = max(u1 - u0, 0);
  const int edge0 = ph ? 0 : -1, edge1 = (V + ph) % EPU ? all_units - 1 : -1;
  const double c = (double)a.scale * (a.token_w ? (double)a.token_w[t] : 1.0);
  auto put = [&](int u, const float (&o)[EPU]) {
    if (u != edge0 && u != edge1) {
      *reinterpret_cast<uint4*>(drow + (u * EPU - ph)) = make_unit(o, T{});
    } else {
#pragma unroll
      for (int e = 0; e < EPU; ++e)
        if ((unsigned)(u * EPU - ph + e) < (unsigned)V) elem<T>::store(drow, u * EPU - ph + e, o[e]);
    }
  };
  auto clear = [&] {
    if (PHASE == DISTILL_STATS) return;
    if (tid == 0 && seg == 0) a.loss[t] = 0.f;
    if (!drow) return;
    float o[EPU];
#pragma unroll
    for (int e = 0; e < EPU; ++e) o[e] = 0.f;
    for (int u = u0 + tid; u < u1; u += NT) put(u, o);
  };
  if (c == 0.0) return clear();  // a masked row is not read
  // the first NT entries before the row: loads retire in order
  const int id0 = tid < K ? a.ids[t * K + tid] : -1;
  const float t0 = tid < K ? a.t_logits[t * K + tid] : 0.f;
  // whole units, with what they hold of other rows (masked below); threads past
  // the segment load its last one.  A unit that passes the buffer's end (the last
  // one of the last row) is put together from its elements.
  const bool end = u1 == all_units && u1 > u0 &&
                   t * a.ld - ph + (int64_t)all_units * EPU > (a.T - 1) * a.ld + V;
  const int n_whole = n_units - end;
  uint4 x[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    if (i * NT < n_whole) {
      const int u = u0 + min(i * NT + tid, n_whole - 1);
      x[i] = *reinterpret_cast<const uint4*>(row + (u * EPU - ph));
    } else {
      x[i] = mask_unit<T>(make_uint4(0u, 0u, 0u, 0u), ALL);
    }
  }
  if (end) {
    T el[EPU];
#pragma unroll
    for (int e = 0; e < EPU; ++e) el[e] = row[min(max((u1 - 1) * EPU - ph + e, 0), V - 1)];
    uint4 last;
    __builtin_memcpy(&last, el, 16);
#pragma unroll
    for (int i = 0; i < NU; ++i)
      if (i * NT + tid == n_whole) x[i] = last;
  }
  if (tid == 0) s_dup = 0;
  for (int i = tid; i < (n_units * EPU + 31) / 32; i += NT) bits[i] = 0u;
  __syncthreads();
  // bit of element v: v - b0
  const int b0 = u0 * EPU - ph, nb = n_units * EPU;
  for (int i = tid; i < K; i += NT) {
    const int id = i < NT ? id0 : a.ids[t * K + i];
    const bool ok = (unsigned)id < (unsigned)V;
    s_id[i] = ok ? id : -1;
    s_e[i] = (double)(i < NT ? t0 : a.t_logits[t * K + i]) * a.inv_tau;
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
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    if (i * NT >= n_units) continue;
    const int u = i * NT + tid, q = min(u, n_units - 1) * EPU;
    const uint32_t k = u < n_units ? (bits[q >> 5] >> (q & 31)) & ALL : ALL;
    if (k) x[i] = mask_unit<T>(x[i], k);
  }
  // The teacher's entries, by the block's last wave while the others form the
  // tail's sum: one exponential an entry for p and one for its class.
  auto teacher = [&] {
    double ref, zm = NEG_INF;
    if (a.t_lse) {
      ref = (double)a.t_lse[t];
    } else {
      double um = NEG_INF;
      for (int i = lane; i < K; i += 64)
        if (s_id[i] >= 0) um = fmax(um, s_e[i]);
      ref = wave_max_d(um);
    }
    if (PHASE != DISTILL_GRAD) {
      for (int i = lane; i < K; i += 64)
        if (here(i)) zm = fmax(zm, s_z[i]);
      zm = wave_max_d(zm);
    }
    const double zr = zm == NEG_INF ? 0.0 : zm;
    double psum = 0.0, hs = 0.0, A = 0.0, P = 0.0;
    int cnt = 0;
    for (int i0 = 0; i0 < K; i0 += 64) {
      const int i = i0 + lane;
      const bool ok = i < K && s_id[i] >= 0, in = ok && here(i), first = in && own(i);
      const double d = ok && s_e[i] != NEG_INF ? s_e[i] - ref : NEG_INF;
      const double e = exp(d);
      if (ok) s_e[i] = e;
      psum += e;
      if (PHASE == DISTILL_GRAD) continue;
      cnt += __popcll(__ballot(first));
      const double z = in ? s_z[i] : NEG_INF;
      const double ez = z == NEG_INF ? 0.0 : exp(z - zm);
      if (first) hs += ez;
      if (in && e != 0.0) {  // e may underflow where the student is -inf
        P += e;
        A += e * (d - (z - zr));
      }
      if (PHASE == DISTILL_ROW && in) s_z[i] = ez;
    }
    psum = wave_sum_d(psum);
    if (lane == 0) s_psum = psum;
    if (PHASE != DISTILL_GRAD) {
      hs = wave_sum_d(hs);
      A = wave_sum_d(A);
      P = PHASE == DISTILL_ROW ? psum : wave_sum_d(P);
      if (lane == 0) {
        s_stat.zm = zm;
        s_stat.hs = hs;
        s_stat.A = A;
        s_stat.P = P;
        s_stat.cnt = cnt;
      }
    }
  };
  float ex[KEEP ? NU : 1][EPU];
  float m;
  double S = 0.0;
  if (PHASE != DISTILL_GRAD) {
    m = wave_max(units_max(x, T{}));
    if (lane == 0) s_max[wv] = m;
    __syncthreads();
    if (wv == NW - 1) teacher();
    m = s_max[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) m = fmaxf(m, s_max[w]);
    const float ms = m == -__builtin_inff() ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (i * NT < n_units) {
#pragma unroll
        for (int e = 0; e < EPU; ++e) {
          const float v = distill_exp(unit_elem(x[i], e, T{}), ms, a);
          if (KEEP) ex[KEEP ? i : 0][e] = v;
          sum += v;
        }
      }
    }
    sum = wave_sum(sum);
    if (lane == 0) s_sum[wv] = sum;
  } else if (wv == NW - 1) {
    teacher();
  }
  // meanwhile, the second launch: the first wave joins the segments
  double zm, top, hs, A;
  int cnt;
  if (PHASE == DISTILL_GRAD && wv == 0) {
    const SegStat* st = a.stats + t * a.segs;
    m = -__builtin_inff();
    zm = NEG_INF;
    for (int i = lane; i < a.segs; i += 64) {
      m = fmaxf(m, st[i].m);
      zm = fmax(zm, st[i].zm);
    }
    m = wave_max(m);
    zm = wave_max_d(zm);
    top = fmax((double)m * a.inv_tau, zm);
    hs = A = 0.0;
    cnt = 0;
    for (int i = lane; i < a.segs; i += 64) {
      const SegStat q = st[i];
      if (q.s != 0.f) S += (double)q.s * exp(((double)q.m - (double)m) * a.inv_tau);
      if (q.hs != 0.0) hs += q.hs * exp(q.zm - zm);
      if (q.P != 0.0) A += q.A - q.P * ((q.zm == NEG_INF ? 0.0 : q.zm) - top);
      cnt += q.cnt;
    }
    S = wave_sum_d(S);
    hs = wave_sum_d(hs);
    A = wave_sum_d(A);
    cnt = __builtin_amdgcn_readlane(wave_incl_scan_i(cnt), 63);
  }
  __syncthreads();
  if (PHASE != DISTILL_GRAD && wv == 0) {
#pragma unroll
    for (int w = 0; w < NW; ++w) S += (double)s_sum[w];
    S = (double)(float)S;
  }
  if (PHASE == DISTILL_STATS) {
    if (tid == 0) {
      SegStat q = s_stat;
      q.m = m;
      q.s = (float)S;
      a.stats[t * a.segs + seg] = q;
    }
    return;
  }
  const double psum = s_psum;
  if (!a.t_lse && psum == 0.0) return clear();  // no entry to learn from
  if (wv == 0) {
    if (PHASE == DISTILL_ROW) {
      zm = s_stat.zm;
      top = fmax((double)m * a.inv_tau, zm);
      hs = s_stat.hs;
      A = psum == 0.0 ? 0.0 : s_stat.A - psum * ((zm == NEG_INF ? 0.0 : zm) - top);
      cnt = s_stat.cnt;
    }
    const RowResult r = finish_row(a, c, psum, m, S, zm, hs, A, top, cnt < V);
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
    float o[EPU];
#pragma unroll
    for (int e = 0; e < EPU; ++e)
      o[e] = r.f * (KEEP ? ex[KEEP ? i : 0][e] : distill_exp(unit_elem(x[i], e, T{}), r.m, a));
    put(u, o);
  }
  __syncthreads();  // the teacher's classes over what the units wrote there
  for (int i = tid; i < K; i += NT) {
    if (!here(i) || !own(i)) continue;
    double e = s_e[i];
    if (s_dup)
      for (int j = i + 1; j < K; ++j)
        if (s_id[j] == s_id[i]) e += s_e[j];
    const double z = s_z[i];
    const double ez = PHASE == DISTILL_ROW ? z : z == NEG_INF ? 0.0 : exp(z - r.zm);
    elem<T>::store(drow, s_id[i], head_grad(a, c, r, ez, e * r.norm));
  }
}

// Segments of a call's rows.  One block holds rows of up to ROW_UNITS units;
// longer ones are cut.  Below that, rows of more than HALF_ROW_UNITS are cut as
// well while they are few (8 x 65000 bf16: 10.3 us cut, 14.0 whole; 32 x 128000:
// 14.0 and 21.7; 80 x 65000: 16.6 and 16.0; 240 x 128000: 49 and 38), into about
// SEG_BLOCKS segments in all.
constexpr int FEW_WAVES = 4 * 1024;  // waves that four a SIMD hold
constexpr int SEG_NT = 256, SEG_NU = 8, SEG_BLOCKS = 512, SEG_TOKENS = 64;
constexpr int ROW_UNITS = 1024 * 16, HALF_ROW_UNITS = 512 * 8;

static void distill_segments(int T, int units, int* segs, int* seg_units) {
  *segs = 1;
  *seg_units = units;
  if (units <= HALF_ROW_UNITS || (units <= ROW_UNITS && T >= SEG_TOKENS)) return;
  const int64_t want = ((int64_t)T * units + SEG_BLOCKS - 1) / SEG_BLOCKS;
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
// Enough for any T' <= T: few rows are cut where many are not.
int64_t distill_ws_bytes_up_to(int T, int V) {
  int64_t most = distill_ws_bytes(T, V);
  for (int t = 1; t <= std::min(T, SEG_TOKENS); ++t) most = std::max(most, distill_ws_bytes(t, V));
  return most;
}

template <typename T, int NT, int NU, int PHASE, int OCC>
static void block_launch(const DistillArgs& a, dim3 grid, const T* student, T* dstudent, hipStream_t s) {
  const size_t lds = (size_t)a.K * 20 + (size_t)(a.seg_units * raw_unit<T>::EPU + 31) / 32 * 4;
  distill_block_kernel<T, NT, NU, PHASE, OCC><<<grid, NT, lds, s>>>(a, student, dstudent);
}

template <typename T, int NT, int NU>
static hipError_t row_launch(const DistillArgs& a, const T* student, T* dstudent, hipStream_t s) {
  block_launch<T, NT, NU, DISTILL_ROW, 4>(a, a.T, student, dstudent, s);
  return hipGetLastError();
}

template <typename T>
static hipError_t distill_t(DistillArgs a, const T* student, T* dstudent, void* ws, hipStream_t s) {
  auto group = [&](auto kernel, int rows) {
    kernel<<<(a.T + rows - 1) / rows, GROUP_THREADS, 0, s>>>(a, student, dstudent);
    return hipGetLastError();
  };
  // 16 lanes a row where they hold its entries (4096 x 40 fp32: 4.5 us, 7.3 with
  // 64 lanes, 8.8 with a block), and longer rows when there are many (16384 x 500
  // bf16: 23, 25 and 29; 5000 x 500 fp32: 10.8, 10.9 and 12.2; 300 x 500 bf16:
  // 10.2, 5.7 and 6.2), else a wave
  if (a.K <= 16 && a.V <= 64) return group(distill_group_kernel<T, 16, 4>, GROUP_THREADS / 16);
  if (a.K <= 16 && a.V <= 512 && a.T > FEW_WAVES)
    return group(distill_group_kernel<T, 16, 32>, GROUP_THREADS / 16);
  if (a.K <= 64 && a.V <= 512) return group(distill_group_kernel<T, 64, 8>, GROUP_THREADS / 64);
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
      block_launch<T, SEG_NT, SEG_NU, DISTILL_STATS, 1>(b, dim3(a.segs, n), student + at, nullptr, s);
      hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      block_launch<T, SEG_NT, SEG_NU, DISTILL_GRAD, 1>(b, dim3(dstudent ? a.segs : 1, n), student + at,
                                                    dstudent ? dstudent + at : nullptr, s);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
  }
  // A small block of eight units a thread: a row's chain of small steps (its
  // entries, joins, barriers) then overlaps that of more other rows on the CU
  // (8192 x 2000 fp32: 33 us with 64 threads, 37 with 128, 45 with 256).  As
  // long as all rows are on the GPU at once anyway (four waves a SIMD), four
  // units and twice the threads shorten the chain (10 x 15000 bf16: 8.1 us with
  // eight, 6.9 with four; 500 x 15001: 13.8, 13.0; 1000 x 15001: 19.4, 21.2).
  // Rows of up to 256 units have a wave either way (16384 x 2000 bf16: 51, 48).
  const bool few = (int64_t)a.T * ((units + 255) / 256) <= FEW_WAVES;
  if (units <= 256) return row_launch<T, 64, 4>(a, student, dstudent, s);
  if (units <= 512)
    return few ? row_launch<T, 128, 4>(a, student, dstudent, s)
               : row_launch<T, 64, 8>(a, student, dstudent, s);
  if (units <= 1024)
    return few ? row_launch<T, 256, 4>(a, student, dstudent, s)
               : row_launch<T, 128, 8>(a, student, dstudent, s);
  if (units <= 2048)
    return few ? row_launch<T, 512, 4>(a, student, dstudent, s)
               : row_launch<T, 256, 8>(a, student, dstudent, s);
  if (units <= 4096) {
    if (few) return row_launch<T, 1024, 4>(a, student, dstudent, s);
    // fp32 rows keep sixteen units' exponentials in registers as well (2000 x
    // 16000: 55 us, 61 with eight); bf16 rows hold twice as many a unit (2048 x
    // 32000: 66 us, 61 with eight)
    if constexpr (sizeof(T) == 4) return row_launch<T, 256, 16>(a, student, dstudent, s);
    return row_launch<T, 512, 8>(a, student, dstudent, s);
  }
  // two blocks a CU, so that one reads while the other sums and writes (1000 x
  // 65000 bf16: 65 us, 83 with 1024 threads of half the units)
  if (units <= 8192) return row_launch<T, 512, 16>(a, student, dstudent, s);
  return row_launch<T, 1024, 16>(a, student, dstudent, s);
}

hipError_t launch_distill(int T, int V, int64_t ld, int K, const void* student, bool is_bf16,
                          const int32_t* ids, const float* t_logits, const float* t_lse,
                          const float* token_w, float tau, float scale, float* loss,
                          void* dstudent, void* ws, hipStream_t s) {
  DistillArgs a{T, V, K, ld, ids, t_logits, t_lse, token_w, 1.0 / (double)tau,
                (float)(1.4426950408889634 / (double)tau), scale, loss, 1, 0, nullptr};
  if (is_bf16) return distill_t(a, (const bf16*)student, (bf16*)dstudent, ws, s);
  return distill_t(a, (const float*)student, (float*)dstudent, ws, s);
}

}  // namespace moe
