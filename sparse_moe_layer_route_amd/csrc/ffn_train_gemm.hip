// The products of the experts' training on the matrix cores, bf16, for
// experts with many rows: 256 x 256 outputs a block, v_mfma_f32_16x16x32_bf16.
//
//   C[n][m] = sum_k A[m][k] B[n][k], m the fast axis of the output
//
//   GATE_UP  m: 128 channels of W_g and of W_u   n: token rows    k: H
//   DOWN     m: H (W_d)                          n: token rows    k: I
//   DACT     m: I (W_d turned)                   n: token rows    k: H
//   DX       m: H (W_g, then W_u, turned)        n: token rows    k: I, twice
//   DW       m: H (x) or I (a), both turned      n: I (dg, du) or H (dy), turned; k: the expert's rows
//
// Four waves, one a SIMD, of 128 x 128 outputs each (256 accumulators a lane):
// per 32 k a wave reads 16 fragments from LDS for 64 matrix instructions, a
// quarter less LDS traffic than eight waves of 128 x 64 would need, and LDS
// reads and the arriving tiles share its 128 bytes a cycle.  Stages of 32 k
// (32 KiB) go from memory to LDS directly into a ring of four; three are in
// flight while a wave's fragments for the next stage are read beside the
// matrix instructions of the present one.  An operand whose k is its fast
// axis lies in LDS by rows of 64 bytes, 16-byte chunk c of row r at c ^ (r / 2
// % 4); one whose k is the slow axis by rows of 256 outputs (512 bytes),
// 32-byte chunk p of row k at p ^ (k % 4 + 4 (k / 8 % 2)), and is turned on
// its way to the registers by the transposing LDS read.  Either way the lanes
// that LDS serves together cover all its banks.
//
// Blocks are persistent: the stages of a block's tiles form one stream, so the
// next tile's first stages load while the present one's outputs are formed.
#include <stdlib.h>

#include <algorithm>

#include "common.h"
#include "ffn_train.h"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// GATE_UP8, DACT8: gate and up kept in 8 bits; DW_ANY: gradients of the
// weights in fp32, or added to what is there
enum { GATE_UP, GATE_UP8, DOWN, DACT, DACT8, DX, DW, DW_ANY };

constexpr int TM = 256;             // outputs of a block along m
constexpr int A_STAGE = TM * 64;    // bytes of 32 k of A
constexpr int STAGING = 2048;       // a wave's: 16 rows x 64 bf16
constexpr int NXCD = 8;
constexpr int CUS = 256;

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
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

typedef __attribute__((address_space(3))) u32x4 lds16_t;
typedef __attribute__((address_space(3))) u32x2 lds8_t;
typedef __attribute__((address_space(3))) uint32_t lds4_t;
typedef __attribute__((address_space(3))) s16x4 lds_turn_t;

__device__ __forceinline__ u32x4 read16(uint32_t at) { return *(const lds16_t*)(uintptr_t)at; }
__device__ __forceinline__ u32x2 read8(uint32_t at) { return *(const lds8_t*)(uintptr_t)at; }
__device__ __forceinline__ void write8(uint32_t at, uint32_t lo, uint32_t hi) {
  *(lds8_t*)(uintptr_t)at = u32x2{lo, hi};
}
// Rows k..k+3 and k+4..k+7 (PITCH bytes apart) of 16 outputs: this lane's output, its 8 k.
template <int PITCH> __device__ __forceinline__ bf16x8_t read_turned(uint32_t at) {
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_turn_t*)(uintptr_t)at);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_turn_t*)(uintptr_t)(at + 4 * PITCH));
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The accumulators stay in the accumulation half of the register file: left to
// itself the compiler moves them to the other and back in every step.  Before
// they are read, and after they are cleared, matrix_done waits as many cycles
// as the longest of the hazards between these instructions takes.
__device__ __forceinline__ void mac(const bf16x8_t& a, const bf16x8_t& b, f32x4_t& c) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
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
__device__ __forceinline__ void matrix_done() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

constexpr int most(int n) { return n > 63 ? 63 : n; }   // the counter's range

// One tile of the launch: expert, its first row and rows, n and m origins, and
// for DW which matrix.
struct Meta { int e, start, n, n0, m0, which; };

// NJ: a wave's outputs along n in sixteens; 4: two blocks a CU, 8: one.
template <int MODE, int NJ>
__global__ void __launch_bounds__(256, NJ == 4 ? 2 : 1) train_gemm_kernel(TrainArgs a) {
  constexpr bool GU = MODE == GATE_UP || MODE == GATE_UP8, DA = MODE == DACT || MODE == DACT8;
  constexpr bool DWS = MODE == DW || MODE == DW_ANY;
  constexpr bool AT = DA || MODE == DX || DWS, BT = DWS;   // operands whose k is the slow axis
  constexpr int TN = 32 * NJ, B_STAGE = TN * 64, SLOT = A_STAGE + B_STAGE, RING = NJ == 4 ? 3 : 4;
  constexpr int NB = NJ / 2, LOADS = 4 + NB;               // a wave's load instructions a stage, B's and all
  __shared__ __attribute__((aligned(1024))) char ring[RING * SLOT];
  __shared__ __attribute__((aligned(16))) char staging[4][STAGING];

  const int lane = lane_id(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wv & 1, wn = wv >> 1, r16 = lane & 15, kg = lane >> 4;
  const int H = a.H, I = a.I;

  // ---- this block's tiles: its XCD's share, every nbx-th ------------------
  const int tiles_m = GU ? (I + 127) / 128 : DA ? (I + TM - 1) / TM : (H + TM - 1) / TM;
  // DW: tiles of dW_g or dW_u (m over H), and of dW_d (m over I)
  const int per_gu = DWS ? ((H + TM - 1) / TM) * ((I + TN - 1) / TN) : 0;
  const int per_d = DWS ? ((I + TM - 1) / TM) * ((H + TN - 1) / TN) : 0;
  const bool any_d = DWS && a.dw[2] != nullptr;
  const int n_gu = DWS ? a.n_dw - any_d : 0;
  int off = 0, cnt = 0;
  if (lane < a.E) {
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
      m.m0 = r % tiles_m * (GU ? 128 : TM);
      m.n0 = r / tiles_m * TN;
    }
    return m;
  };
  // pairs of stages of a tile (DX: of each of its two halves)
  const int pairs_i = (I + 63) / 64;
  auto pairs_of = [&](const Meta& m) __attribute__((always_inline)) {
    return DWS ? max(1, (m.n + 63) / 64) : MODE == DX ? 2 * pairs_i : MODE == DOWN ? pairs_i : H / 64;
  };
  // stages of kept rows that follow a tile's own (DACT)
  constexpr int EXTRA = MODE == DACT ? 2 * NJ : MODE == DACT8 ? NJ : 0;

  // ---- loading stream -----------------------------------------------------
  // Wave w moves rows 64 w..+63 of A and a quarter of B's (k fast), or k 8 w..+7
  // of either (k slow), in instructions of 1 KiB.  The stream's
  // position is a pair of stages of a tile; it ends with the block's last tile.
  const uint32_t ring0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)&ring[0];
  int dj = 0, dpair = 0, dpairs;
  bool more = true;
  Meta dm = decode(0);
  const char* pa[4];                   // this lane's next 16 bytes, by instruction
  const char* pb[NB];                  // (DW's pa: its column, the rows being looked up)
  int64_t step_a = 0, step_b = 0;
  const int kchunk = (lane & 3) ^ ((lane >> 3) & 3);    // k fast: the 16-byte chunk this lane moves
  const int slow_k0 = 8 * wv + (lane >> 5);             // k slow: row (+ 2 q) this lane moves
  auto slow_col = [&](int q) __attribute__((always_inline)) {
    const int k = slow_k0 + 2 * q, f = (k & 3) | (((k >> 3) & 1) << 2);
    return 16 * (((lane & 31) >> 1) ^ f) + 8 * (lane & 1);
  };
  constexpr int BL = TN / 8;                            // B's: lanes of a row
  const int slow_kb0 = 8 * wv + lane / BL;              // (+ 64 / BL q)
  auto slow_col_b = [&](int q) __attribute__((always_inline)) {
    const int k = slow_kb0 + 64 / BL * q, f = (k & 3) | (((k >> 3) & 1) << 2);
    return 16 * (((lane % BL) >> 1) ^ f) + 8 * (lane & 1);
  };
  // DW: x's rows of a stage are looked up through scalar loads a stage ahead
  const __attribute__((address_space(4))) int32_t* perm_s =
      (const __attribute__((address_space(4))) int32_t*)(uintptr_t)a.perm;
  // p / k, p < 2^25: the high word of p ceil(2^32 / k)
  const uint32_t per_k = (uint32_t)(((1ull << 32) + a.k - 1) / a.k);
  int rows[8];
  auto look_up = [&](int stage) __attribute__((always_inline)) {
    if (!DWS) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int p = min(dm.start + 32 * stage + 8 * wv + i, a.pairs - 1);
      const uint32_t t = (uint32_t)perm_s[p];
      rows[i] = dm.which == 2 ? p : (int)(a.k == 1 ? t : __umulhi(t, per_k));
    }
  };
  auto set_tile = [&]() __attribute__((always_inline)) {
    const int64_t we = (int64_t)dm.e * I * H;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = 64 * wv + 16 * q + (lane >> 2);       // k fast: row of the tile
      const int64_t k = slow_k0 + 2 * q;
      if (GU) {
        const int ch = min(dm.m0 + (r >> 7) * 64 + (r & 63), I - 1);
        pa[q] = (const char*)((const bf16*)((r >> 6) & 1 ? a.w_up : a.w_gate) + we + (int64_t)ch * H + 8 * kchunk);
      } else if (MODE == DOWN) {
        pa[q] = (const char*)((const bf16*)a.w_down + we + (int64_t)min(dm.m0 + r, H - 1) * I + 8 * kchunk);
      } else if (DA) {
        pa[q] = (const char*)((const bf16*)a.w_down + we + k * I + min(dm.m0 + slow_col(q), I - 8));
      } else if (MODE == DX) {                            // W_g, then W_u
        pa[q] = (const char*)((const bf16*)(dpair >= pairs_i ? a.w_up : a.w_gate) + we + k * H +
                              min(dm.m0 + slow_col(q), H - 8));
      } else {
        const bool down = dm.which == 2;
        pa[q] = (const char*)((const bf16*)(down ? a.act : a.x) + min(dm.m0 + slow_col(q), (down ? I : H) - 8));
      }
    }
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int64_t row = dm.start + min(dm.n0 + 16 * NB * wv + 16 * q + (lane >> 2), dm.n - 1);
      if (GU) {
        pb[q] = (const char*)((const bf16*)a.x + (int64_t)(a.perm[row] / a.k) * H + 8 * kchunk);
      } else if (MODE == DOWN) {
        pb[q] = (const char*)((const bf16*)a.act + row * I + 8 * kchunk);
      } else if (DA) {
        pb[q] = (const char*)((const bf16*)a.dy + row * H + 8 * kchunk);
      } else if (MODE == DX) {
        pb[q] = (const char*)((const bf16*)a.dgu + (2 * row + (dpair >= pairs_i)) * I + 8 * kchunk);
      } else {
        const bool down = dm.which == 2;
        pb[q] = (const char*)((const bf16*)(down ? a.dy : a.dgu) +
                              (int64_t)(dm.start + slow_kb0 + 64 / BL * q) * (down ? H : 2 * I) + (down ? 0 : dm.which * I) +
                              min(dm.n0 + slow_col_b(q), (down ? H : I) - 8));
      }
    }
    step_a = !AT ? 64 : DWS ? 2 * (int64_t)(dm.which == 2 ? I : H) : 64 * (int64_t)(MODE == DX ? H : I);
    step_b = !BT ? 64 : 64 * (int64_t)(dm.which == 2 ? H : 2 * I);
    dpairs = pairs_of(dm);
  };
  auto load_a = [&](uint32_t slot, int stage) __attribute__((always_inline)) {
    const uint32_t to = ring0 + slot + 4096 * wv;
    const int k0 = 32 * (MODE == DX && stage >= 2 * pairs_i ? stage - 2 * pairs_i : stage);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const char* p = pa[q];
      if (DWS) p += (int64_t)(lane < 32 ? rows[2 * q] : rows[2 * q + 1]) * step_a;
      else pa[q] += step_a;
      bool live = true;
      if (MODE == DOWN) live = k0 + 8 * kchunk < I;
      if (MODE == DX) live = k0 + slow_k0 + 2 * q < I;
      if (DWS) live = k0 + slow_k0 + 2 * q < dm.n;
      dma16(live ? p : (const char*)zero_chunk, to + 1024 * q);
    }
  };
  auto load_b = [&](uint32_t slot, int stage) __attribute__((always_inline)) {
    const uint32_t to = ring0 + slot + A_STAGE + 1024 * NB * wv;
    const int k0 = 32 * (MODE == DX && stage >= 2 * pairs_i ? stage - 2 * pairs_i : stage);
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      bool live = true;
      if (MODE == DOWN || MODE == DX) live = k0 + 8 * kchunk < I;
      if (DWS) live = k0 + slow_kb0 + 64 / BL * q < dm.n;
      dma16(live ? pb[q] : (const char*)zero_chunk, to + 1024 * q);
      pb[q] += step_b;
    }
  };
  // DACT: stage e of kept rows into this wave's own 4 KiB of a slot: 16 rows x
  // 64 channels (8 bits: 128) of g, then of u, rows of 128 bytes with 16-byte
  // chunk c of row r at c ^ (r % 8)
  auto load_kept = [&](uint32_t slot, int e) __attribute__((always_inline)) {
    const uint32_t to = ring0 + slot + 4096 * wv;
    const int row0 = dm.n0 + 16 * NJ * wn + 16 * (MODE == DACT ? e >> 1 : e);
    const int c0 = dm.m0 + 128 * wm + (MODE == DACT ? 64 * (e & 1) : 0);
    const int l = fresh_lane(), c = (l & 7) ^ (l >> 3);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t p = dm.start + min(row0 + 8 * (q & 1) + (l >> 3), dm.n - 1);
      const int64_t at = (2 * p + (q >> 1)) * I;
      dma16(MODE == DACT ? (const char*)((const bf16*)a.kept + at + min(c0 + 8 * c, I - 8))
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
  bf16x8_t fa[8], fb[2][NJ];
  f32x4_t acc[8][NJ];
  const uint32_t f = ((r16 >> 2) & 3) | ((kg & 1) << 2);
  const uint32_t straight = (uint32_t)(r16 * 64 + ((kg ^ ((r16 >> 1) & 3)) * 16));
  auto turned = [&](uint32_t pitch, uint32_t first) __attribute__((always_inline)) {
    return (uint32_t)((8 * kg + (r16 >> 2)) * pitch + ((first ^ f) << 5) + (r16 & 3) * 8);
  };
  const uint32_t base_a = ring0 + (AT ? turned(512, 8 * wm) : straight + wm * 8192);
  const uint32_t base_b = ring0 + A_STAGE + (BT ? turned(2 * TN, NJ * wn) : straight + wn * 1024 * NJ);
  auto read_a = [&](int i, uint32_t slot) __attribute__((always_inline)) {
    return AT ? read_turned<512>((base_a ^ (i << 5)) + slot)
              : __builtin_bit_cast(bf16x8_t, read16(base_a + slot + 1024 * i));
  };
  auto read_b = [&](int i, uint32_t slot) __attribute__((always_inline)) {
    return BT ? read_turned<2 * TN>((base_b ^ (i << 5)) + slot)
              : __builtin_bit_cast(bf16x8_t, read16(base_b + slot + 1024 * i));
  };
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    matrix_done();
  };
  auto after = [&](uint32_t slot) __attribute__((always_inline)) {
    return slot == (RING - 1) * SLOT ? 0u : slot + SLOT;
  };

  // One stage: the matrix instructions of its fragments (B's set P); the next
  // stage's are read in their places as they fall free; half ODD of the
  // stream's pair is loaded into this stage's slot, whose fragments were read
  // a step ago.  Before the barrier the loads that the next step reads have
  // landed: of the RING stages beyond the present one, all but the last RING - 2.
#define STEP(P, ODD)                                                                           \
  {                                                                                            \
    const uint32_t from = after(slot);                                                         \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) {                                            \
      _Pragma("unroll") for (int j = 0; j < NJ; ++j) mac(fa[i], fb[P][j], acc[i][j]);           \
      fa[i] = read_a(i, from);                                                                 \
      if (i < NJ) fb[1 - (P)][i] = read_b(i, from);                                            \
      if (i == 1 && more) load_stage(slot, ODD);                                               \
      __builtin_amdgcn_sched_barrier(0);                                                       \
    }                                                                                          \
    wait_lds();                                                                                \
    if (!more) wait_loads<0>();                                                                \
    else if (settled > 0) --settled;                                                           \
    else if (EXTRA > 0 && dpair >= dpairs) wait_loads<(RING - 2) * 4>();                       \
    else wait_loads<(RING - 2) * LOADS>();                                                     \
    if (ODD) { if (more) next_pair(); } else look_up(2 * dpair + 1);                           \
    __builtin_amdgcn_s_barrier();                                                              \
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
  else if (EXTRA > 0 && (dpair >= dpairs || dj > 0)) wait_loads<(RING - 2) * 4>();
  else wait_loads<(RING - 2) * LOADS>();     // stages 0 and 1
  __builtin_amdgcn_s_barrier();
  auto first_fragments = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) fa[i] = read_a(i, slot);
#pragma unroll
    for (int j = 0; j < NJ; ++j) fb[0][j] = read_b(j, slot);
    wait_lds();
    __builtin_amdgcn_s_barrier();      // the slot may be filled again
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
    }
    if constexpr (DA) {
      // The kept rows' stages follow: a wave works on its own part of each and
      // the slot is filled again once all are done.  A wave whose outputs are
      // all there issues S stores a stage; of any other only loads (four a
      // stage at least) are counted.
      constexpr int S = MODE == DACT ? 6 : 12;
      const int left = cm.n - cm.n0 - 16 * NJ * wn, cols = I - cm.m0 - 128 * wm;
      const bool full = left >= 16 * NJ && cols >= 128;
      matrix_done();
#pragma unroll
      for (int e = 0; e < EXTRA; ++e) {
        if (e >= 2) {
          if (!more) wait_loads<0>();
          else if (full && e == 2) wait_loads<most(4 * (RING - 1) + 2 * S)>();
          else if (full) wait_loads<most(4 * (RING - 1) + (RING - 1) * S)>();
          else wait_loads<4 * (RING - 1)>();
        }
        if (left > 0 && cols > 0) gradients(cm, e, slot);
        __builtin_amdgcn_s_barrier();
        if (more) {
          load_stage(slot, (e + RING) & 1);
          if ((e + RING) & 1) next_pair(); else look_up(2 * dpair + 1);
        }
        slot = after(slot);
      }
      if (!more) wait_loads<0>();
      else if (dj > cj + 1 || dpair >= dpairs) wait_loads<4 * (RING - 2)>();
      else if (full) wait_loads<most((RING - 2) * (LOADS + S))>();
      else wait_loads<(RING - 2) * LOADS>();
      __builtin_amdgcn_s_barrier();
      first_fragments();
    } else {
      // what is in flight lands before the first store, so that the next step
      // need not wait for the stores behind it
      wait_loads<0>();
      settled = RING - 2;
      matrix_done();
      outputs(cm);
      if constexpr (GU) first_fragments();   // read again: they are not held across the outputs
    }
    clear();
  }
  wait_loads<0>();                     // no load outlives the block's LDS
#undef STEP
}

}  // namespace

template <int MODE, int NJ>
static void go(const TrainArgs& a, int64_t tiles, hipStream_t s) {
  // persistent: the CUs' share, a multiple of the XCDs
  const int64_t g = std::min<int64_t>(tiles, NJ == 4 ? 2 * CUS : CUS);
  train_gemm_kernel<MODE, NJ><<<(unsigned)((g + NXCD - 1) / NXCD * NXCD), 256, 0, s>>>(a);
}

template <int NJ> static void launch(int which, TrainArgs a, int P, hipStream_t s) {
  constexpr int TN = 32 * NJ;
  const int64_t row_tiles = P / TN + std::min(a.E, P);       // an upper bound
  const int64_t mh = (a.H + TM - 1) / TM, mi = (a.I + TM - 1) / TM;
  if constexpr (NJ == 8) {
    go<DX, NJ>(a, row_tiles * mh, s);
  } else if (which == 0) {
    const int64_t tiles = row_tiles * ((a.I + 127) / 128);
    if (a.keep8) go<GATE_UP8, NJ>(a, tiles, s);
    else go<GATE_UP, NJ>(a, tiles, s);
  } else if (which == 1) {
    go<DOWN, NJ>(a, row_tiles * mh, s);
  } else if (which == 2) {
    if (a.keep8) go<DACT8, NJ>(a, row_tiles * mi, s);
    else go<DACT, NJ>(a, row_tiles * mi, s);
  } else if (which == 3) {
    go<DX, NJ>(a, row_tiles * mh, s);
  } else {
    a.n_dw = (a.dw[0] != nullptr) + (a.dw[1] != nullptr) + (a.dw[2] != nullptr);
    if (!a.n_dw) return;
    const int64_t tiles = a.E * a.n_dw * std::max(mh * ((a.I + TN - 1) / TN), mi * ((a.H + TN - 1) / TN));
    if (a.dw_f32 || a.accumulate) go<DW_ANY, NJ>(a, tiles, s);
    else go<DW, NJ>(a, tiles, s);
  }
}

hipError_t launch_train_gemm(int which, const TrainArgs& a, int P, hipStream_t s) {
  // One block a CU and rows by 256 where the blocks of an XCD stream far more
  // of the weights than its L2 holds, so that they are fetched again for every
  // 128 rows (dx at 4096 x 3584, I 2560, 64 experts top-8: 1.54 against 1.88
  // ms); elsewhere two blocks a CU, one's outputs beside the other's products
  // (Granite-shaped dx 135 against 157 us, gate and up 149 against 188).
  if (which == 3 && (int64_t)a.H * a.I >= (4 << 20) && P >= 256 * a.E) launch<8>(which, a, P, s);
  else launch<4>(which, a, P, s);
  return hipGetLastError();
}

}  // namespace moe
