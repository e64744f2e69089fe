// Tokens sorted by expert and back, with the slot weights applied, and the
// gradient:
//   dispatch             x_perm[inv[t,j]] = x[t]
//   undispatch           out[t] = add[t] + sum_j w[t,j] y_perm[inv[t,j]]
//   undispatch backward  dy_perm[inv[t,j]] = w[t,j] dout[t],
//                        dw[t,j] = <dout[t], y_perm[inv[t,j]]>
// The gradient of dispatch is undispatch without weights.  All three walk the
// tokens, not the sorted rows: x, out and dout move once, and each sorted row
// is touched by exactly one token, so nothing is accumulated in memory and the
// sums run over the slots in slot order.  Every kernel is bound by the bytes
// of the T*k sorted rows.  A row is cut into units of 16 bytes of the layer's type
// (hidden % 64 == 0, so a row is whole units; fp32 rows beside a bf16 layer have
// 32 bytes a unit).
// Slots with inv outside 0..T*k-1 (pairs that are not computed) move nothing.
#include <algorithm>

#include "common.h"

namespace moe {

constexpr int DISPATCH_THREADS = 256;

// 16 bytes that are read once (load_once below): they do not stay in the caches.
__device__ __forceinline__ uint4 load_stream(const void* p) {
  typedef uint32_t v4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const v4*>(p)));
}

// N elements as loaded: 16 bytes of the layer's type (8 bf16, 4 fp32), and as
// many elements of fp32 rows beside a bf16 layer (32 bytes).
template <typename T, int N> struct unit;
template <> struct unit<bf16, 8> {
  uint4 a;
  __device__ __forceinline__ void load(const bf16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void load_once(const bf16* p) { a = load_stream(p); }
  __device__ __forceinline__ void store(bf16* p) const { *reinterpret_cast<uint4*>(p) = a; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_uint4(f2_to_bf16x2(v[0], v[1]), f2_to_bf16x2(v[2], v[3]), f2_to_bf16x2(v[4], v[5]),
                   f2_to_bf16x2(v[6], v[7]));
  }
};
template <int N> struct unit<float, N> {
  float4 a[N / 4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) a[i] = reinterpret_cast<const float4*>(p)[i];
  }
  __device__ __forceinline__ void load_once(const float* p) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) a[i] = __builtin_bit_cast(float4, load_stream(p + 4 * i));
  }
  __device__ __forceinline__ void store(float* p) const {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) reinterpret_cast<float4*>(p)[i] = a[i];
  }
  __device__ __forceinline__ void get(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      v[4 * i] = a[i].x; v[4 * i + 1] = a[i].y; v[4 * i + 2] = a[i].z; v[4 * i + 3] = a[i].w;
    }
  }
  __device__ __forceinline__ void set(const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      a[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
};
template <typename T> constexpr int unit_elems() { return 16 / (int)sizeof(T); }

// One thread per (token, unit), flat over the batch: a unit is read once and
// stored to its k rows, 64 lanes on 1 KiB of each.  4096 x 1536 bf16 top-8
// (113 MB): 21.0 us, 5.4 TB/s, what a copy of that size reaches; 8 x 2048 top-6:
// 3.1 us, a launch.
template <typename T>
__global__ void __launch_bounds__(DISPATCH_THREADS)
dispatch_kernel(uint32_t n, uint32_t units, int H, int k, uint32_t P, const T* __restrict__ x,
                const int32_t* __restrict__ inv, T* __restrict__ x_perm) {
  const uint32_t g = blockIdx.x * DISPATCH_THREADS + threadIdx.x;
  if (g >= n) return;
  const uint32_t t = g / units, u = g - t * units;
  constexpr int N = unit_elems<T>();
  unit<T, N> v;
  v.load(x + (int64_t)g * N);
  for (int j = 0; j < k; ++j) {
    const uint32_t row = (uint32_t)inv[(int64_t)t * k + j];
    if (row < P) v.store(x_perm + (int64_t)row * H + u * N);
  }
}

// One thread per (token, unit): the loads of all slots' rows go out together,
// then the sum runs in slot order in fp32 and is rounded once.  add may be
// out itself (a thread reads its unit before it writes it).
// ONCE: the rows are read past the caches.
// 6007 x 2048 bf16 top-6, a tenth of the pairs missing (182 MB): 32.2 us, 5.7
// TB/s; 256 x 3584 top-8 on fp32 rows (33 MB): 7.0 us.
template <typename T, typename Ty, bool ONCE>
__global__ void __launch_bounds__(DISPATCH_THREADS)
undispatch_kernel(uint32_t n, uint32_t units, int H, int k, uint32_t P,
                  const Ty* __restrict__ y_perm, const int32_t* __restrict__ inv,
                  const float* __restrict__ topk_w, const T* add, T* out) {
  const uint32_t g = blockIdx.x * DISPATCH_THREADS + threadIdx.x;
  if (g >= n) return;
  const uint32_t t = g / units, u = g - t * units;
  constexpr int N = unit_elems<T>();
  float acc[N];
#pragma unroll
  for (int c = 0; c < N; ++c) acc[c] = 0.f;
  if (add) {
    unit<T, N> a;
    a.load(add + (int64_t)g * N);
    a.get(acc);
  }
  unit<Ty, N> v[MOE_MAX_TOPK];
  float w[MOE_MAX_TOPK];
  bool live[MOE_MAX_TOPK];
#pragma unroll
  for (int j = 0; j < MOE_MAX_TOPK; ++j) {
    const int64_t o = (int64_t)t * k + j;
    const uint32_t row = j < k ? (uint32_t)inv[o] : 0xFFFFFFFFu;
    live[j] = row < P;
    w[j] = 1.f;
    if (live[j]) {
      const Ty* p = y_perm + (int64_t)row * H + u * N;
      if (ONCE)
        v[j].load_once(p);
      else
        v[j].load(p);
      if (topk_w) w[j] = topk_w[o];
    }
  }
#pragma unroll
  for (int j = 0; j < MOE_MAX_TOPK; ++j) {
    if (!live[j]) continue;
    float f[N];
    v[j].get(f);
#pragma unroll
    for (int c = 0; c < N; ++c) acc[c] = fmaf(w[j], f[c], acc[c]);
  }
  unit<T, N> o;
  o.set(acc);
  o.store(out + (int64_t)g * N);
}

// One group of G lanes per token (up to a wave: the power of two that covers the
// row's units; 256: a block).  Each lane walks its units, U of them with up to
// KM slots' rows in flight, then the lanes' partial dots meet in a fixed tree
// (and a block's four waves in wave order).
// ONCE: y_perm is read past the caches.
// 4096 x 1536 bf16 top-8, both gradients (214 MB): 45.0 us, 4.8 TB/s, as much
// read as written; 333 x 256 fp32 top-2: 3.4 us, a launch.
template <typename T, typename Ty, int G, int KM, bool DY, bool DW, bool ONCE>
__global__ void __launch_bounds__(DISPATCH_THREADS)
undispatch_bwd_kernel(int T_, int units, int H, int k, uint32_t P, const T* __restrict__ dout,
                      const Ty* __restrict__ y_perm, const int32_t* __restrict__ inv,
                      const float* __restrict__ topk_w, Ty* __restrict__ dy_perm,
                      float* __restrict__ dtopk_w) {
  constexpr int N = unit_elems<T>(), U = MOE_MAX_TOPK / KM;
  const int l = threadIdx.x % G;
  const int t = blockIdx.x * (DISPATCH_THREADS / G) + threadIdx.x / G;
  if (t >= T_) return;  // whole groups leave together
  uint32_t row[KM];
  float w[KM], dot[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    const int64_t o = (int64_t)t * k + j;
    row[j] = j < k ? (uint32_t)inv[o] : 0xFFFFFFFFu;
    w[j] = DY && j < k ? topk_w[o] : 0.f;
    dot[j] = 0.f;
  }
  for (int u0 = l; u0 < units; u0 += U * G) {
    unit<T, N> d[U];
    unit<Ty, N> y[U][KM];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int u = u0 + q * G;
      if (q > 0 && u >= units) break;
      d[q].load(dout + (int64_t)t * H + u * N);
      if (DW) {
#pragma unroll
        for (int j = 0; j < KM; ++j)
          if (row[j] < P) {
            const Ty* p = y_perm + (int64_t)row[j] * H + u * N;
            if (ONCE)
              y[q][j].load_once(p);
            else
              y[q][j].load(p);
          }
      }
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int u = u0 + q * G;
      if (q > 0 && u >= units) break;
      float df[N];
      d[q].get(df);
#pragma unroll
      for (int j = 0; j < KM; ++j) {
        if (row[j] >= P) continue;
        if (DW) {
          float f[N];
          y[q][j].get(f);
#pragma unroll
          for (int c = 0; c < N; ++c) dot[j] = fmaf(df[c], f[c], dot[j]);
        }
        if (DY) {
          float o[N];
#pragma unroll
          for (int c = 0; c < N; ++c) o[c] = w[j] * df[c];
          unit<Ty, N> ov;
          ov.set(o);
          ov.store(dy_perm + (int64_t)row[j] * H + u * N);
        }
      }
    }
  }
  if (!DW) return;
  __shared__ float part[KM][DISPATCH_THREADS / MOE_WAVE];
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    float s = dot[j];
#pragma unroll
    for (int m = (G < MOE_WAVE ? G : MOE_WAVE) / 2; m > 0; m >>= 1) s += __shfl_xor(s, m, 64);
    if (G <= MOE_WAVE) {
      if (l == 0 && j < k) dtopk_w[(int64_t)t * k + j] = s;
    } else if (l % MOE_WAVE == 0) {
      part[j][l / MOE_WAVE] = s;
    }
  }
  if (G > MOE_WAVE) {
    __syncthreads();
    if (l < k) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < DISPATCH_THREADS / MOE_WAVE; ++v) s += part[l][v];
      dtopk_w[(int64_t)t * k + l] = s;
    }
  }
}

template <typename T>
static void dispatch_t(const moe_dims_t& d, int T_, const void* x, const int32_t* inv, void* x_perm,
                       hipStream_t s) {
  const uint32_t units = d.hidden / unit_elems<T>(), n = (uint32_t)T_ * units;
  dispatch_kernel<T><<<(n + DISPATCH_THREADS - 1) / DISPATCH_THREADS, DISPATCH_THREADS, 0, s>>>(
      n, units, d.hidden, d.top_k, (uint32_t)T_ * d.top_k, (const T*)x, inv, (T*)x_perm);
}

hipError_t launch_dispatch(const moe_dims_t& d, int T, const void* x, const int32_t* inv,
                           void* x_perm, hipStream_t s) {
  if (d.dtype == MOE_BF16)
    dispatch_t<bf16>(d, T, x, inv, x_perm, s);
  else
    dispatch_t<float>(d, T, x, inv, x_perm, s);
  return hipGetLastError();
}

// Bytes of sorted rows from which reading them past the caches gains, also right
// after the kernel that wrote them, whose last rows the caches still hold (with
// that kernel, bf16 rows: 67 MB 33.0 us without, 34.8 with; 101 MB 51.5, 49.9; 147 MB
// 79, 72; fp32 rows beside a bf16 layer, two loads a unit: 101 MB 50.0, 53.7; 134
// MB 75, 69).  Stores are not treated so: their reader loses more than they gain.
template <typename T, typename Ty> constexpr size_t once_bytes() {
  return (size_t)(sizeof(T) == sizeof(Ty) ? 80 : 128) << 20;
}
template <typename T, typename Ty>
static void undispatch_t(const moe_dims_t& d, int T_, const void* y, const int32_t* inv,
                         const float* w, const void* add, void* out, hipStream_t s) {
  const uint32_t units = d.hidden / unit_elems<T>(), n = (uint32_t)T_ * units;
  const size_t bytes = (size_t)T_ * d.top_k * d.hidden * sizeof(Ty);
  const auto kernel = bytes >= once_bytes<T, Ty>() ? undispatch_kernel<T, Ty, true>
                                                   : undispatch_kernel<T, Ty, false>;
  kernel<<<(n + DISPATCH_THREADS - 1) / DISPATCH_THREADS, DISPATCH_THREADS, 0, s>>>(
      n, units, d.hidden, d.top_k, (uint32_t)T_ * d.top_k, (const Ty*)y, inv, w, (const T*)add,
      (T*)out);
}

hipError_t launch_undispatch(const moe_dims_t& d, int T, const void* y_perm, bool rows_bf16,
                             const int32_t* inv, const float* topk_w, const void* add, void* out,
                             hipStream_t s) {
  if (d.dtype != MOE_BF16)
    undispatch_t<float, float>(d, T, y_perm, inv, topk_w, add, out, s);
  else if (rows_bf16)
    undispatch_t<bf16, bf16>(d, T, y_perm, inv, topk_w, add, out, s);
  else
    undispatch_t<bf16, float>(d, T, y_perm, inv, topk_w, add, out, s);
  return hipGetLastError();
}

struct UndispatchBwd {
  const moe_dims_t& d;
  int T;
  const void *dout, *y_perm;
  const int32_t* inv;
  const float* w;
  void* dy;
  float* dw;
  hipStream_t s;
};

// Reading y_perm past the caches gains from less on here, since dy_perm is as much
// again (with the kernel that wrote the rows, bf16: 34 MB 25.2 us without, 25.9 with;
// 49 MB 37.3, 35.8; 67 MB 52.4, 50.7; 246 MB 189, 170).  fp32 rows beside a bf16 layer
// lose at every size (201 MB 149, 160); rows below a wave of units keep the plain
// loads.
constexpr size_t BWD_ONCE_BYTES = (size_t)40 << 20;
template <typename T, typename Ty, int G, int KM, bool DY, bool DW>
static void bwd_launch(const UndispatchBwd& a) {
  constexpr int per = DISPATCH_THREADS / G;
  constexpr bool MAY = DW && G >= MOE_WAVE && sizeof(T) == sizeof(Ty);
  const bool once = MAY && (size_t)a.T * a.d.top_k * a.d.hidden * sizeof(Ty) >= BWD_ONCE_BYTES;
  const auto kernel = once ? undispatch_bwd_kernel<T, Ty, G, KM, DY, DW, MAY>
                           : undispatch_bwd_kernel<T, Ty, G, KM, DY, DW, false>;
  kernel<<<(a.T + per - 1) / per, DISPATCH_THREADS, 0, a.s>>>(
      a.T, a.d.hidden / unit_elems<T>(), a.d.hidden, a.d.top_k, (uint32_t)a.T * a.d.top_k,
      (const T*)a.dout, (const Ty*)a.y_perm, a.inv, a.w, (Ty*)a.dy, a.dw);
}
template <typename T, typename Ty, int G, int KM>
static void bwd_outputs(const UndispatchBwd& a) {
  if (a.dy && a.dw)
    bwd_launch<T, Ty, G, KM, true, true>(a);
  else if (a.dy)
    bwd_launch<T, Ty, G, KM, true, false>(a);
  else
    bwd_launch<T, Ty, G, KM, false, true>(a);
}
// Short rows: as many lanes as units (16384 x 64 top-8: 9.7 us with 16 lanes a
// token, 20 with 64; fp32 8192 x 128 top-4: 10.2 with 32, 13.4 with 64).
// A block per token for rows of more than a wave's units, when there are few
// tokens (256 x 4096 top-8: 11.3 us against 14.6 with a wave per token) or its
// waves are nearly always busy (2048 x 2048: 31 against 37); a row that leaves
// many of them idle is better off with a wave (16384 x 1088, 136 units: 26
// against 50).
template <typename T, typename Ty, int KM>
static void bwd_group(const UndispatchBwd& a) {
  const int units = a.d.hidden / unit_elems<T>(), B = DISPATCH_THREADS;
  const bool full = 8 * units >= 7 * ((units + B - 1) / B * B);
  if (units <= 16)
    bwd_outputs<T, Ty, 16, KM>(a);
  else if (units <= 32)
    bwd_outputs<T, Ty, 32, KM>(a);
  else if (units > MOE_WAVE && (full || a.T <= 1024))
    bwd_outputs<T, Ty, DISPATCH_THREADS, KM>(a);
  else
    bwd_outputs<T, Ty, MOE_WAVE, KM>(a);
}
// Up to two slots: four units of a lane at once, to have as many loads in
// flight as eight slots have (8192 x 1536 top-2: 27.6 us against 29.5).
template <typename T, typename Ty>
static void bwd_slots(const UndispatchBwd& a) {
  if (a.d.top_k <= 2)
    bwd_group<T, Ty, 2>(a);
  else
    bwd_group<T, Ty, MOE_MAX_TOPK>(a);
}

// At least one of dy and dw is not null; y_perm is read only for dw, topk_w
// only for dy.
hipError_t launch_undispatch_backward(const moe_dims_t& d, int T, const void* dout,
                                      const void* y_perm, bool rows_bf16, const int32_t* inv,
                                      const float* topk_w, void* dy, float* dw, hipStream_t s) {
  const UndispatchBwd a{d, T, dout, y_perm, inv, topk_w, dy, dw, s};
  if (d.dtype != MOE_BF16)
    bwd_slots<float, float>(a);
  else if (rows_bf16)
    bwd_slots<bf16, bf16>(a);
  else
    bwd_slots<bf16, float>(a);
  return hipGetLastError();
}

}  // namespace moe
