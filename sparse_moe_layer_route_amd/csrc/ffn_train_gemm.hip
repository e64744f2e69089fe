// The products of the experts' training on the matrix cores.
//
//   C[n][m] = sum_k A[m][k] B[n][k], m the fast axis of the output
//
//   GATE_UP  m: channels of W_g and of W_u       n: token rows    k: H
//   DOWN     m: H (W_d)                          n: token rows    k: I
//   DACT     m: I (W_d turned)                   n: token rows    k: H
//   DX       m: H (W_g, then W_u, turned)        n: token rows    k: I, twice
//   DW       m: H (x) or I (a), both turned      n: I (dg, du) or H (dy), turned; k: the expert's rows
//
// A block is four waves, WM x WN of them, each with 16 MI outputs along m and
// 16 NJ along n; v_mfma_f32_16x16x32_bf16, or v_mfma_f32_16x16x4_f32 for fp32
// layers.  Stages of 64 bytes of k (32 bf16, 16 fp32) go from memory to LDS
// directly into a ring; a wave's fragments for the next stage are read beside
// the matrix instructions of the present one.  An operand whose k is its fast
// axis lies in LDS by rows of 64 bytes, 16-byte chunk c of row r at c ^ (r / 2
// % 4).  One whose k is the slow axis lies by rows of its outputs: bf16 with
// 32-byte chunk p of row k at p ^ (k % 4 + 4 (k / 8 % 2)), turned on its way to
// the registers by the transposing LDS read; fp32 with 64-byte chunk p of row
// k at p ^ (k / 4 % 4), read a value at a time.  Either way the lanes that LDS
// serves together cover all its banks.
//
// Blocks are persistent: the stages of a block's tiles form one stream, so the
// next tile's first stages load while the present one's outputs are formed.
#include <algorithm>

#include "common.h"
#include "ffn_train.h"
#include "ffn_train_shapes.h"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// DACT8, GATE_UP8: gate and up kept in 8 bits; DW_ANY: gradients of the
// weights in fp32, or added to what is there
enum { GATE_UP, GATE_UP8, DOWN, DACT, DACT8, DX, DW, DW_ANY };

constexpr int STAGING = 2048;       // LDS of a wave's outputs: 16 rows x 64 bf16
constexpr int NXCD = 8;

__device__ __attribute__((aligned(16))) const uint32_t zero_chunk[4] = {0, 0, 0, 0};

// 16 bytes a lane from `from` to LDS, lane l at `to` + 16 l.  Outside the
// compiler's wait counting (it would drain all loads before the next LDS
// read): landing is waited for by count, below.  M0, which holds the LDS
// address, is reserved to such code: nothing else in these kernels uses it.
__device__ __forceinline__ void dma16(const void* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               : : "v"(from), "s"(to) : "memory");
}
template <int N> __device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N > 63 ? 63 : N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// All waves of the block; no LDS access moves to the other side.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

typedef __attribute__((address_space(3))) u32x4 lds16_t;
typedef __attribute__((address_space(3))) u32x2 lds8_t;
typedef __attribute__((address_space(3))) uint32_t lds4_t;
typedef __attribute__((address_space(3))) s16x4 lds_turn_t;

__device__ __forceinline__ u32x4 read16(uint32_t at) { return *(const lds16_t*)(uintptr_t)at; }
__device__ __forceinline__ u32x2 read8(uint32_t at) { return *(const lds8_t*)(uintptr_t)at; }
__device__ __forceinline__ uint32_t read4(uint32_t at) { return *(const lds4_t*)(uintptr_t)at; }
__device__ __forceinline__ void write8(uint32_t at, uint32_t lo, uint32_t hi) {
  *(lds8_t*)(uintptr_t)at = u32x2{lo, hi};
}

// Fragments: 16 bytes of k of one output a lane.  turned<PITCH>: from rows k
// PITCH bytes apart, of which this lane's address points into the first.
template <typename T> struct frag;
template <> struct frag<bf16> {
  template <int PITCH> __device__ static u32x4 turned(uint32_t at) {   // rows k..k+3, k+4..k+7 of 16 outputs
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_turn_t*)(uintptr_t)at);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_turn_t*)(uintptr_t)(at + 4 * PITCH));
    return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};
template <> struct frag<float> {
  template <int PITCH> __device__ static u32x4 turned(uint32_t at) {
    return u32x4{read4(at), read4(at + PITCH), read4(at + 2 * PITCH), read4(at + 3 * PITCH)};
  }
};

// c += a b.  The accumulators stay in the accumulation half of the register
// file: left to itself the compiler moves them to the other and back in every
// step.  It knows nothing of the hazards between these instructions and others:
// the accumulators are cleared by a matrix instruction too (0 * 0 + 0), never
// by moves that the compiler might place next to one, and before they are
// read, and after they are cleared, matrix_done waits for longer than any of
// them takes to write its results.
template <typename T> __device__ __forceinline__ void mac(const u32x4& a, const u32x4& b, f32x4_t& c) {
  if constexpr (sizeof(T) == 2) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)      // k = 4 kg + q of the four lane groups kg
      asm volatile("v_mfma_f32_16x16x4_f32 %0, %1, %2, %0" : "+a"(c) : "v"(a[q]), "v"(b[q]));
  }
}
__device__ __forceinline__ void clear_acc(const u32x4& zeros, f32x4_t& c) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %1, 0" : "=a"(c) : "v"(zeros));
}
__device__ __forceinline__ void matrix_done() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }
__device__ __forceinline__ float acc_read(float v) {
  float r;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(r) : "a"(v));
  return r;
}
__device__ __forceinline__ void acc_read4(const f32x4_t& v, float (&r)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) r[q] = acc_read(v[q]);
}

// The lane, as a value that nothing derived from is kept in registers for the
// next use across the steps in between.
__device__ __forceinline__ int fresh_lane() {
  int l = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  asm volatile("" : "+v"(l));
  return l;
}

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const bf16* p, float (&v)[4]) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = float4{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ void store4(bf16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(f2_to_bf16x2(v[0], v[1]), f2_to_bf16x2(v[2], v[3]));
}

// One tile of the launch: expert, its first row and rows, n and m origins, and
// for DW which matrix.
struct Meta { int e, start, n, n0, m0, which; };

// The sizes that follow from a block's shape.
template <typename T, int WM_, int WN_, int MI_, int NJ_> struct Shape {
  typedef T type;
  static constexpr int WM = WM_, WN = WN_, MI = MI_, NJ = NJ_;
  static_assert(WM * WN == 4, "four waves");
  static constexpr int SZ = sizeof(T), BK = 64 / SZ, CH = 16 / SZ;   // k of a stage, of a 16-byte chunk
  static constexpr int TM = 16 * MI * WM, TN = 16 * NJ * WN;
  static constexpr int A_STAGE = TM * 64, B_STAGE = TN * 64, SLOT = A_STAGE + B_STAGE;
  static constexpr int NA = TM / 64, NB = TN / 64, LOADS = NA + NB;  // a wave's load instructions a stage
  // 256 x 256: a block fills a CU's registers; 256 x 128: two blocks fill its
  // LDS; 128 x 64: more, for streams of weights that pass once
  static constexpr int RING = NJ == 8 ? 4 : NJ == 4 || MI == 8 ? 3 : 4;
  static constexpr int PER_CU = NJ == 8 ? 1 : NJ == 4 ? 2 : MI == 8 ? 3 : 4;
};

template <int MODE, typename S>
__global__ void __launch_bounds__(256, S::PER_CU) train_gemm_kernel(TrainArgs a) {
  typedef typename S::type T;
  constexpr int MI = S::MI, NJ = S::NJ, BK = S::BK, CH = S::CH, SZ = S::SZ, TM = S::TM, TN = S::TN;
  constexpr int A_STAGE = S::A_STAGE, SLOT = S::SLOT, NA = S::NA, NB = S::NB, RING = S::RING, LOADS = S::LOADS;
  constexpr bool GU = MODE == GATE_UP || MODE == GATE_UP8, DA = MODE == DACT || MODE == DACT8;
  constexpr bool DWS = MODE == DW || MODE == DW_ANY;
  constexpr bool AT = DA || MODE == DX || DWS, BT = DWS;   // operands whose k is the slow axis
  __shared__ __attribute__((aligned(1024))) char ring[RING * SLOT];
  __shared__ __attribute__((aligned(16))) char staging[4][STAGING];

  const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv % S::WM, wn = wv / S::WM, r16 = lane & 15, kg = lane >> 4;
  const int H = a.H, I = a.I;

  // ---- this block's tiles: its XCD's share, every nbx-th ------------------
  constexpr int MSTEP = GU ? TM / 2 : TM;              // GATE_UP: as many channels of either matrix
  const int tiles_m = ((GU || DA ? I : H) + MSTEP - 1) / MSTEP;
  // DW: tiles of dW_g or dW_u (m over H), and of dW_d (m over I)
  const int per_gu = DWS ? ((H + TM - 1) / TM) * ((I + TN - 1) / TN) : 0;
  const int per_d = DWS ? ((I + TM - 1) / TM) * ((H + TN - 1) / TN) : 0;
  const bool any_d = DWS && a.dw[2] != nullptr;
  const int n_gu = DWS ? a.n_dw - any_d : 0;
  int off = 0, cnt = 0;
  if (lane < a.E && a.offsets) {
    off = a.offsets[lane];
    cnt = a.offsets[lane + 1] - off;
  }
  const int mine = lane < a.E ? (DWS ? per_gu * n_gu + (any_d ? per_d : 0) : (cnt + TN - 1) / TN * tiles_m) : 0;
  const int incl = wave_incl_scan_i(mine);
  const int total = __builtin_amdgcn_readlane(incl, 63);
  const int nbx = gridDim.x / NXCD, xcd = blockIdx.x % NXCD, bi = blockIdx.x / NXCD;
  const int per_x = (total + NXCD - 1) / NXCD;
  const int first = xcd * per_x + bi, past = min(total, (xcd + 1) * per_x);
  if (first >= past) return;
  const int n_my = (past - first + nbx - 1) / nbx;

  auto decode = [&](int j) __attribute__((always_inline)) {
    const int t = first + j * nbx;
    const uint64_t in = __ballot(t >= incl - mine && t < incl);
    Meta m;
    m.e = __builtin_ctzll(in);
    const int r = t - (__builtin_amdgcn_readlane(incl, m.e) - __builtin_amdgcn_readlane(mine, m.e));
    m.start = __builtin_amdgcn_readlane(off, m.e);
    m.n = __builtin_amdgcn_readlane(cnt, m.e);
    if constexpr (DWS) {
      const int w = r / per_gu;
      const bool down = w >= n_gu;
      const int q = down ? r - n_gu * per_gu : r - w * per_gu;
      m.which = down ? 2 : a.dw[0] ? w : 1;
      const int nm = ((down ? I : H) + TM - 1) / TM;
      m.m0 = q % nm * TM;
      m.n0 = q / nm * TN;
    } else {
      m.which = 0;
      m.m0 = r % tiles_m * MSTEP;
      m.n0 = r / tiles_m * TN;
    }
    return m;
  };
  // pairs of stages of a tile (DX: of each of its two halves)
  const int pairs_i = (I + 2 * BK - 1) / (2 * BK);
  auto pairs_of = [&](const Meta& m) __attribute__((always_inline)) {
    return DWS ? max(1, (m.n + 2 * BK - 1) / (2 * BK))
           : MODE == DX ? 2 * pairs_i : MODE == DOWN ? pairs_i : H / (2 * BK);
  };
  // stages of kept rows that follow a tile's own (DACT, bf16)
  constexpr bool STREAMED = DA && SZ == 2 && NJ >= 4;
  constexpr int EXTRA = !STREAMED ? 0 : MODE == DACT ? 2 * NJ : NJ;
  static_assert(MI == 8 || (!GU && EXTRA == 0), "a wave has 64 channels of either matrix, kept rows 128");
  static_assert(EXTRA % 2 == 0 && (EXTRA == 0 || EXTRA >= RING), "pairs of stages, a ring of them");

  // ---- loading stream -----------------------------------------------------
  // A wave moves a quarter of either operand's stage in instructions of 1 KiB:
  // of its rows (k fast) or of its k (k slow).  The stream's position is a
  // pair of stages of a tile; it ends with the block's last tile.
  const uint32_t ring0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)&ring[0];
  int dj = 0, dpair = 0, dpairs;
  bool more = true;
  Meta dm = decode(0);
  const char* pa[NA];                  // this lane's next 16 bytes, by instruction
  const char* pb[NB];                  // (DW's pa: its column, the rows being looked up)
  int64_t step_a = 0, step_b = 0;
  const int kchunk = (lane & 3) ^ ((lane >> 3) & 3);    // k fast: the 16-byte chunk this lane moves
  constexpr int KW = BK / 4;                            // k slow: k of a wave
  constexpr int AL = TM * SZ / 16, BL = TN * SZ / 16;   // lanes of a row
  const int slow_a = KW * wv + lane / AL, slow_b = KW * wv + lane / BL;   // + 64 / AL q, 64 / BL q
  // the output whose chunk lies at 16-byte place j of row k
  auto slow_col = [&](int k, int j, int width) __attribute__((always_inline)) {
    if constexpr (SZ == 4) return 4 * (j ^ (((k >> 2) & 3) << 2));
    const int f = (k & 3) | (width >= 128 ? ((k >> 3) & 1) << 2 : 0);
    return 16 * ((j >> 1) ^ f) + 8 * (j & 1);
  };
  // DW: the pairs of a wave's rows of x are looked up through scalar loads a
  // step before they are loaded; perm_s is a.perm in the constant address space
  typedef int32_t ints_t __attribute__((ext_vector_type(KW), aligned(4)));
  const __attribute__((address_space(4))) int32_t* perm_s =
      (const __attribute__((address_space(4))) int32_t*)(uintptr_t)a.perm;
  // p / k, p < 2^25: the high word of p ceil(2^32 / k)
  const uint32_t per_k = (uint32_t)(((1ull << 32) + a.k - 1) / a.k);
  ints_t pairs_at;
  auto look_up = [&](int stage) __attribute__((always_inline)) {
    if (!DWS) return;
    const int p = dm.start + BK * stage + KW * wv;
    if (dm.which == 2 || dm.n == 0) {    // rows of the sorted buffers themselves
#pragma unroll
      for (int i = 0; i < KW; ++i) pairs_at[i] = p + i;
    } else if (p + KW <= a.pairs) {
      pairs_at = *(const __attribute__((address_space(4))) ints_t*)(perm_s + p);
    } else {
#pragma unroll
      for (int i = 0; i < KW; ++i) pairs_at[i] = perm_s[min(p + i, a.pairs - 1)];
    }
  };
  auto row_at = [&](int i) __attribute__((always_inline)) {
    const uint32_t p = (uint32_t)pairs_at[i];
    return (int)(dm.which == 2 || a.k == 1 ? p : __umulhi(p, per_k));
  };
  auto set_tile = [&]() __attribute__((always_inline)) {
    const int64_t we = (int64_t)dm.e * I * H;
    // from the lane afresh: held since the last tile these would cost registers
    const int lane = fresh_lane(), kchunk = (lane & 3) ^ ((lane >> 3) & 3);
    const int slow_a = KW * wv + lane / AL, slow_b = KW * wv + lane / BL;
    auto col_a = [&](int q) __attribute__((always_inline)) { return slow_col(slow_a + 64 / AL * q, lane % AL, TM); };
    auto col_b = [&](int q) __attribute__((always_inline)) { return slow_col(slow_b + 64 / BL * q, lane % BL, TN); };
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      const int r = 16 * NA * wv + 16 * q + (lane >> 2);  // k fast: row of the tile
      const int64_t k = slow_a + 64 / AL * q;
      if (GU) {                                           // 64 channels of W_g, 64 of W_u for each wave's part
        const int ch = min(dm.m0 + (r >> 7) * 64 + (r & 63), I - 1);
        pa[q] = (const char*)((const T*)((r >> 6) & 1 ? a.w_up : a.w_gate) + we + (int64_t)ch * H + CH * kchunk);
      } else if (MODE == DOWN) {
        pa[q] = (const char*)((const T*)a.w_down + we + (int64_t)min(dm.m0 + r, H - 1) * I + CH * kchunk);
      } else if (DA) {
        pa[q] = (const char*)((const T*)a.w_down + we + k * I + min(dm.m0 + col_a(q), I - CH));
      } else if (MODE == DX) {                            // W_g, then W_u
        pa[q] = (const char*)((const T*)(dpair >= pairs_i ? a.w_up : a.w_gate) + we + k * H +
                              min(dm.m0 + col_a(q), H - CH));
      } else {
        const bool down = dm.which == 2;
        pa[q] = (const char*)((const T*)(down ? a.act : a.x) + min(dm.m0 + col_a(q), (down ? I : H) - CH));
      }
    }
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int64_t row = dm.start + min(dm.n0 + 16 * NB * wv + 16 * q + (lane >> 2), dm.n - 1);
      if (GU) {
        pb[q] = (const char*)((const T*)a.x + (int64_t)(a.perm[row] / a.k) * H + CH * kchunk);
      } else if (MODE == DOWN) {
        pb[q] = (const char*)((const T*)a.act + row * I + CH * kchunk);
      } else if (DA) {
        pb[q] = (const char*)((const T*)a.dy + row * H + CH * kchunk);
      } else if (MODE == DX) {
        pb[q] = (const char*)((const T*)a.dgu + (2 * row + (dpair >= pairs_i)) * I + CH * kchunk);
      } else {
        const bool down = dm.which == 2;
        pb[q] = (const char*)((const T*)(down ? a.dy : a.dgu) +
                              (int64_t)(dm.start + slow_b + 64 / BL * q) * (down ? H : 2 * I) + (down ? 0 : dm.which * I) +
                              min(dm.n0 + col_b(q), (down ? H : I) - CH));
      }
    }
    step_a = !AT ? 64 : DWS ? (int64_t)SZ * (dm.which == 2 ? I : H) : (int64_t)SZ * BK * (MODE == DX ? H : I);
    step_b = !BT ? 64 : (int64_t)SZ * BK * (dm.which == 2 ? H : 2 * I);
    dpairs = pairs_of(dm);
  };
  auto load_a = [&](uint32_t slot, int stage) __attribute__((always_inline)) {
    const uint32_t to = ring0 + slot + 1024 * NA * wv;
    const int k0 = BK * (MODE == DX && stage >= 2 * pairs_i ? stage - 2 * pairs_i : stage);
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      const char* p = pa[q];
      if constexpr (DWS) {
        constexpr int R = 64 / AL;                        // rows of an instruction
        int row = row_at(R * q);
#pragma unroll
        for (int i = 1; i < R; ++i) row = lane >= i * AL ? row_at(R * q + i) : row;
        p += (int64_t)row * step_a;
      } else {
        pa[q] += step_a;
      }
      bool live = true;
      if (MODE == DOWN) live = k0 + CH * kchunk < I;
      if (MODE == DX) live = k0 + slow_a + 64 / AL * q < I;
      if (DWS) live = k0 + slow_a + 64 / AL * q < dm.n;
      dma16(live ? p : (const char*)zero_chunk, to + 1024 * q);
    }
  };
  auto load_b = [&](uint32_t slot, int stage) __attribute__((always_inline)) {
    const uint32_t to = ring0 + slot + A_STAGE + 1024 * NB * wv;
    const int k0 = BK * (MODE == DX && stage >= 2 * pairs_i ? stage - 2 * pairs_i : stage);
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      bool live = true;
      if (MODE == DOWN || MODE == DX) live = k0 + CH * kchunk < I;
      if (DWS) live = k0 + slow_b + 64 / BL * q < dm.n;
      dma16(live ? pb[q] : (const char*)zero_chunk, to + 1024 * q);
      pb[q] += step_b;
    }
  };
  // Stage e of kept rows into this wave's own 4 KiB of a slot: 16 rows x 64
  // channels (8 bits: 128) of g, then of u, rows of 128 bytes with 16-byte
  // chunk c of row r at c ^ (r % 8)
  constexpr int KEPT_LOADS = 4;
  auto load_kept = [&](uint32_t slot, int e) __attribute__((always_inline)) {
    const uint32_t to = ring0 + slot + 4096 * wv;
    const int row0 = dm.n0 + 16 * NJ * wn + 16 * (MODE == DACT ? e >> 1 : e);
    const int c0 = dm.m0 + 128 * wm + (MODE == DACT ? 64 * (e & 1) : 0);
    const int l = fresh_lane(), c = (l & 7) ^ (l >> 3);
#pragma unroll
    for (int q = 0; q < KEPT_LOADS; ++q) {
      const int64_t p = dm.start + min(row0 + 8 * (q & 1) + (l >> 3), dm.n - 1);
      const int64_t at = (2 * p + (q >> 1)) * I;
      dma16(MODE == DACT ? (const char*)((const T*)a.kept + at + min(c0 + 8 * c, I - 8))
                         : (const char*)a.kept + at + min(c0 + 16 * c, I - 16),
            to + 1024 * q);
    }
  };
  // half of the stream's pair into a slot; the second half moves on
  auto load_stage = [&](uint32_t slot, int odd) __attribute__((always_inline)) {
    if (EXTRA > 0 && dpair >= dpairs) {
      load_kept(slot, 2 * (dpair - dpairs) + odd);
    } else {
      load_a(slot, 2 * dpair + odd);
      load_b(slot, 2 * dpair + odd);
    }
  };
  auto next_pair = [&]() __attribute__((always_inline)) {
    ++dpair;
    bool fresh = MODE == DX && dpair == pairs_i;
    if (dpair == dpairs + EXTRA / 2) {
      if (dj + 1 < n_my) {
        ++dj;
        dm = decode(dj);
        dpair = 0;
        fresh = true;
      } else {
        more = false;
      }
    }
    if (fresh) set_tile();
    look_up(2 * dpair);
  };

  // ---- fragments ----------------------------------------------------------
  u32x4 fa[MI], fb[2][NJ];
  f32x4_t acc[MI][NJ];
  const uint32_t straight = (uint32_t)(r16 * 64 + ((kg ^ ((r16 >> 1) & 3)) * 16));
  // k slow: tile `first` of the wave, in rows of `width` outputs
  auto turned = [&](int width, int first) __attribute__((always_inline)) {
    if constexpr (SZ == 4) return (uint32_t)(4 * kg * width * 4 + ((first ^ kg) << 6) + r16 * 4);
    const int f = ((r16 >> 2) & 3) | (width >= 128 ? (kg & 1) << 2 : 0);
    return (uint32_t)((8 * kg + (r16 >> 2)) * width * 2 + ((first ^ f) << 5) + (r16 & 3) * 8);
  };
  constexpr int TILE_BITS = SZ == 4 ? 6 : 5;           // log2 of a tile's 16 outputs in bytes
  const uint32_t base_a = ring0 + (AT ? turned(TM, MI * wm) : straight + wm * 1024 * MI);
  const uint32_t base_b = ring0 + A_STAGE + (BT ? turned(TN, NJ * wn) : straight + wn * 1024 * NJ);
  auto read_a = [&](int i, uint32_t slot) __attribute__((always_inline)) {
    return AT ? frag<T>::template turned<TM * SZ>((base_a ^ (i << TILE_BITS)) + slot) : read16(base_a + slot + 1024 * i);
  };
  auto read_b = [&](int i, uint32_t slot) __attribute__((always_inline)) {
    return BT ? frag<T>::template turned<TN * SZ>((base_b ^ (i << TILE_BITS)) + slot) : read16(base_b + slot + 1024 * i);
  };
  auto clear = [&]() __attribute__((always_inline)) {
    u32x4 zeros = {0u, 0u, 0u, 0u};
    asm volatile("s_nop 3" : "+v"(zeros));       // written by moves: let them settle
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) clear_acc(zeros, acc[i][j]);
    matrix_done();
  };
  // fp32: what the accumulators have reached is put aside every FLUSH pairs of
  // stages (512 k), so that a long sum's error grows with the root of its parts
  // rather than of its terms (4128 terms: 1.2e-6 of the result without)
  constexpr int FLUSH = 16;
  f32x4_t aside[SZ == 4 ? MI : 1][SZ == 4 ? NJ : 1] = {};
  auto put_aside = [&]() __attribute__((always_inline)) {
    if constexpr (SZ == 4) {
      matrix_done();
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          float v[4];
          acc_read4(acc[i][j], v);
#pragma unroll
          for (int q = 0; q < 4; ++q) aside[i][j][q] += v[q];
        }
      clear();
    }
  };
  auto sum4 = [&](int i, int j, float (&v)[4]) __attribute__((always_inline)) {
    acc_read4(acc[i][j], v);
    if constexpr (SZ == 4)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += aside[i][j][q];
  };
  auto after = [&](uint32_t slot) __attribute__((always_inline)) {
    return slot == (RING - 1) * SLOT ? 0u : slot + SLOT;
  };
  // fewest loads that a stage of the stream may have
  constexpr int FEWEST = EXTRA > 0 && KEPT_LOADS < LOADS ? KEPT_LOADS : LOADS;

  // One stage: the matrix instructions of its fragments (B's set P); the next
  // stage's are read in their places as they fall free; half ODD of the
  // stream's pair is loaded into this stage's slot, whose fragments were read
  // a step ago.  Before the barrier the loads that the next step reads have
  // landed: of the RING stages beyond the present one, all but the last RING - 2.
#define STEP(P, ODD)                                                                           \
  {                                                                                            \
    const uint32_t from = after(slot);                                                         \
    const bool loading = more, keeping = EXTRA > 0 && dpair >= dpairs;                         \
    _Pragma("unroll") for (int i = 0; i < MI; ++i) {                                           \
      _Pragma("unroll") for (int j = 0; j < NJ; ++j) mac<T>(fa[i], fb[P][j], acc[i][j]);       \
      fa[i] = read_a(i, from);                                                                 \
      if (i < NJ) fb[1 - (P)][i] = read_b(i, from);                                            \
      if (i == 1 && loading) {                                                                 \
        load_stage(slot, ODD);                                                                 \
        if (ODD) next_pair(); else look_up(2 * dpair + 1);                                     \
      }                                                                                        \
      __builtin_amdgcn_sched_barrier(0);                                                       \
    }                                                                                          \
    wait_lds();                                                                                \
    if (!loading) wait_loads<0>();                                                             \
    else if (settled > 0) --settled;                                                           \
    else if (keeping) wait_loads<(RING - 2) * FEWEST>();                                       \
    else wait_loads<(RING - 2) * LOADS>();                                                     \
    meet();                                                                                    \
    slot = from;                                                                               \
  }

  // ---- outputs ------------------------------------------------------------
  const uint32_t mine0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)&staging[wv][0];
#include "ffn_train_gemm_out.h"

  uint32_t slot = 0;                   // of the present stage
  set_tile();
  look_up(0);
#pragma unroll
  for (int st = 0; st < RING; ++st)
    if (more) {
      load_stage(st * SLOT, st & 1);
      if (st & 1) next_pair(); else look_up(2 * dpair + 1);
    }
  if (!more) wait_loads<0>();
  else wait_loads<(RING - 2) * FEWEST>();                // stages 0 and 1
  meet();
  auto first_fragments = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[i] = read_a(i, slot);
#pragma unroll
    for (int j = 0; j < NJ; ++j) fb[0][j] = read_b(j, slot);
    wait_lds();
    meet();      // the slot may be filled again
  };
  first_fragments();
  clear();
  int settled = 0;                     // steps whose loads have landed already
  for (int cj = 0; cj < n_my; ++cj) {
    const Meta cm = decode(cj);
    const int pairs = pairs_of(cm);
    before_tile(cm);
    for (int p = 0; p < pairs; ++p) {
      STEP(0, RING & 1)
      STEP(1, 1 - (RING & 1))
      if (SZ == 4 && (p + 1) % FLUSH == 0 && p + 1 < pairs) put_aside();
    }
    if constexpr (EXTRA > 0) {
      // The kept rows' stages follow: a wave works on its own part of each and
      // the slot is filled again once all are done.  A wave whose outputs are
      // all there issues ST stores a stage; of any other only loads are counted.
      constexpr int ST = MODE == DACT ? 6 : 12;
      const int left = cm.n - cm.n0 - 16 * NJ * wn, cols = I - cm.m0 - 16 * MI * wm;
      const bool full = left >= 16 * NJ && cols >= 128;
      matrix_done();
      settle_scales();
#pragma unroll
      for (int e = 0; e < EXTRA; ++e) {
        if (e >= 2) {
          if (!more) wait_loads<0>();
          else if (full && e == 2) wait_loads<FEWEST * (RING - 1) + 2 * ST>();
          else if (full) wait_loads<(FEWEST + ST) * (RING - 1)>();
          else wait_loads<FEWEST * (RING - 1)>();
        }
        if (left > 0 && cols > 0) gradients(cm, e, slot);
        meet();
        if (more) {
          load_stage(slot, (e + RING) & 1);
          if ((e + RING) & 1) next_pair(); else look_up(2 * dpair + 1);
        }
        slot = after(slot);
      }
      if (!more) wait_loads<0>();
      else if (full) wait_loads<(RING - 2) * (FEWEST + ST)>();
      else wait_loads<(RING - 2) * FEWEST>();
      meet();
      first_fragments();
    } else {
      // what is in flight lands before the first store, so that the next steps
      // need not wait for the stores behind it
      wait_loads<0>();
      settled = RING - 2;
      matrix_done();
      outputs(cm);
      if constexpr (GU || DA) first_fragments();   // read again: they are not held across the outputs
    }
    clear();
    if constexpr (SZ == 4)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) aside[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  wait_loads<0>();                     // no load outlives the block's LDS
#undef STEP
}

template <int MODE, typename S> void go(const TrainArgs& a, int64_t tiles, hipStream_t s) {
  // Persistent: the CUs' share, a multiple of the XCDs.
  const int64_t g = std::min<int64_t>(tiles, S::PER_CU * kTrainCus);
  train_gemm_kernel<MODE, S><<<(unsigned)((g + NXCD - 1) / NXCD * NXCD), 256, 0, s>>>(a);
}

// A launch is known when this is compiled, so that only the shapes its rule
// can choose are.
template <train_launch W, typename S> void launch(TrainArgs a, int P, hipStream_t s) {
  constexpr int TM = S::TM, TN = S::TN;
  auto row_tiles = [&](int width, int m) { return train_row_tiles(P, a.E, width, TN, m); };
  if constexpr (W == TRAIN_GATE_UP) {
    static_assert(S::MI == 8, "a wave has 64 channels of either matrix");
    if (a.keep8) go<GATE_UP8, S>(a, row_tiles(a.I, TM / 2), s);
    else go<GATE_UP, S>(a, row_tiles(a.I, TM / 2), s);
  } else if constexpr (W == TRAIN_DOWN) {
    go<DOWN, S>(a, row_tiles(a.H, TM), s);
  } else if constexpr (W == TRAIN_DACT) {
    if (a.keep8) go<DACT8, S>(a, row_tiles(a.I, TM), s);
    else go<DACT, S>(a, row_tiles(a.I, TM), s);
  } else if constexpr (W == TRAIN_DX) {
    go<DX, S>(a, row_tiles(a.H, TM), s);
  } else {
    a.n_dw = (a.dw[0] != nullptr) + (a.dw[1] != nullptr) + (a.dw[2] != nullptr);
    if (!a.n_dw) return;
    const int64_t mh = (a.H + TM - 1) / TM, mi = (a.I + TM - 1) / TM;
    const int64_t tiles = a.E * a.n_dw * std::max(mh * ((a.I + TN - 1) / TN), mi * ((a.H + TN - 1) / TN));
    if (a.dw_f32 || a.accumulate) go<DW_ANY, S>(a, tiles, s);
    else if constexpr (S::SZ == 2) go<DW, S>(a, tiles, s);
  }
}

template <train_launch W> void launch_any(const TrainArgs& a, int P, bool is_bf16, hipStream_t s) {
  const train_shape shape = train_shape_of(W, is_bf16, P, a.E, a.H, a.I);
  if (is_bf16) {
    if constexpr (W == TRAIN_DX)
      if (shape == SHAPE_256x256) return launch<W, Shape<bf16, 2, 2, 8, 8>>(a, P, s);
    if constexpr (W == TRAIN_DOWN)
      if (shape == SHAPE_64x64) return launch<W, Shape<bf16, 1, 4, 4, 1>>(a, P, s);
    if (shape == SHAPE_256x128) return launch<W, Shape<bf16, 2, 2, 8, 4>>(a, P, s);
    launch<W, Shape<bf16, 1, 4, 8, 1>>(a, P, s);
  } else {
    if constexpr (W != TRAIN_GATE_UP)
      if (shape == SHAPE_64x64) return launch<W, Shape<float, 1, 4, 4, 1>>(a, P, s);
    launch<W, Shape<float, 1, 4, 8, 1>>(a, P, s);
  }
}

}  // namespace

int64_t train_ws_bytes(const moe_dims_t& d, int64_t T) {
  return T * d.top_k * 3 * d.inter * (d.dtype == MOE_BF16 ? 2 : 4);
}

hipError_t launch_ffn_train(const TrainArgs& a, int P, bool is_bf16, hipStream_t s) {
  launch_any<TRAIN_GATE_UP>(a, P, is_bf16, s);
  launch_any<TRAIN_DOWN>(a, P, is_bf16, s);
  return hipGetLastError();
}

hipError_t launch_ffn_backward(const TrainArgs& a, int P, bool is_bf16, hipStream_t s) {
  if (P > 0) {
    launch_any<TRAIN_DACT>(a, P, is_bf16, s);
    if (a.dx) launch_any<TRAIN_DX>(a, P, is_bf16, s);
  }
  launch_any<TRAIN_DW>(a, P, is_bf16, s);
  return hipGetLastError();
}

}  // namespace moe
