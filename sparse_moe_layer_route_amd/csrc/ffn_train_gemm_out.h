  // (part of train_gemm_kernel) A wave's 16 MI x 16 NJ accumulators: lane (r16, kg)
  // holds of tile (i, j) outputs m = 16 i + 4 kg..+3 of row n = 16 j + r16.
  // bf16 outputs go through LDS in pieces of 16 rows x 64 m, 16-byte chunk c of
  // row r at c ^ (r % 8), and out as runs of 128 bytes of a row; fp32 ones out
  // as they are, runs of 64 bytes.
  float scales[EXTRA > 0 ? NJ : 1];   // DACT8: of rows 16 j + r16, matrix kg % 2, block kg / 2
  auto before_tile = [&](const Meta& m) __attribute__((always_inline)) {
    if constexpr (MODE == DACT8 && EXTRA > 0) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int64_t p = m.start + min(m.n0 + 16 * NJ * wn + 16 * j + r16, m.n - 1);
        const int b = min((m.m0 + 16 * MI * wm) / 64 + (kg >> 1), a.blocks - 1);
        scales[j] = a.scale[(2 * p + (kg & 1)) * a.blocks + b];
      }
    }
  };
  // The scales are ordinary loads: at their first use the compiler waits for all
  // that it knows to be in flight, and so for the stream's loads and the stores
  // behind them.  Used here, before the kept rows' stages, that happens once a tile
  // and the stages' counted waits hold (with two blocks a CU the time is the same:
  // 4096 tokens, H 3584, I 2560, 64 experts top-8, dact 975 us either way).
  auto settle_scales = [&]() __attribute__((always_inline)) {
    if constexpr (MODE == DACT8 && EXTRA > 0)
#pragma unroll
      for (int j = 0; j < NJ; ++j) asm volatile("" : "+v"(scales[j]));
  };
  // 16 rows x 64 outputs: take() the four of tile i, then store() them to
  // out[row * ld + m..] where rows and columns are left
  struct Piece { uint32_t v[8]; float f[SZ == 4 ? 16 : 1]; };
  auto take = [&](Piece& to, int i, const float (&v)[4]) __attribute__((always_inline)) {
    if constexpr (SZ == 4) {
#pragma unroll
      for (int q = 0; q < 4; ++q) to.f[4 * i + q] = v[q];
    } else {
      to.v[2 * i] = f2_to_bf16x2(v[0], v[1]);
      to.v[2 * i + 1] = f2_to_bf16x2(v[2], v[3]);
    }
  };
  auto store = [&](const Piece& from, T* out, int64_t ld, int rows_left, int cols_left) __attribute__((always_inline)) {
    const int l = fresh_lane(), r16 = l & 15, kg = l >> 4;
    if constexpr (SZ == 4) {
      if (r16 >= rows_left) return;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (16 * i < cols_left)
          *reinterpret_cast<float4*>(out + r16 * ld + 16 * i + 4 * kg) =
              float4{from.f[4 * i], from.f[4 * i + 1], from.f[4 * i + 2], from.f[4 * i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        write8(mine0 + r16 * 128 + (((2 * i + (kg >> 1)) ^ (r16 & 7)) << 4) + ((kg & 1) << 3), from.v[2 * i],
               from.v[2 * i + 1]);
      wait_lds();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 8 * h + (l >> 3), c = l & 7;
        const u32x4 w = read16(mine0 + r * 128 + ((c ^ (r & 7)) << 4));
        if (r < rows_left && 8 * c < cols_left) *reinterpret_cast<u32x4*>(out + r * ld + 8 * c) = w;
      }
      wait_lds();
    }
  };
  // DACT: dg, du and a of 16 rows x 64 channels, their kept g and u from LDS
  // (rows of 128 bytes at `at`, 2 KiB on for u) or from memory
  auto gradients16 = [&](const Meta& m, int j, int half, uint32_t at) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    const int l = fresh_lane(), r16 = l & 15, kg = l >> 4;
    const int row0 = m.n0 + 16 * NJ * wn + 16 * j, left = m.n - row0;
    const int c0 = m.m0 + 16 * MI * wm + 64 * half, cols = I - c0;
    const int64_t p0 = m.start + row0, p = m.start + min(row0 + r16, m.n - 1);
    float sg = 1.f, su = 1.f;
    if constexpr (MODE == DACT8) {
      if constexpr (EXTRA > 0) {
        sg = __shfl(scales[j], r16 + 32 * half);
        su = __shfl(scales[j], r16 + 32 * half + 16);
      } else {
        sg = a.scale[2 * p * a.blocks + c0 / 64];
        su = a.scale[(2 * p + 1) * a.blocks + c0 / 64];
      }
    }
    float g[4][4], u[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = c0 + min(16 * i, cols - 16) + 4 * kg;      // memory: columns that are there
      if constexpr (MODE == DACT8) {
        const uint32_t w = (((4 * half + i) ^ (r16 & 7)) << 4) + 4 * kg;
        const uint32_t gw = EXTRA > 0 ? read4(at + r16 * 128 + w)
                                      : *reinterpret_cast<const uint32_t*>((const int8_t*)a.kept + 2 * p * I + c);
        const uint32_t uw = EXTRA > 0 ? read4(at + 2048 + r16 * 128 + w)
                                      : *reinterpret_cast<const uint32_t*>((const int8_t*)a.kept + (2 * p + 1) * I + c);
        unpack8x4(gw, sg, g[i]);
        unpack8x4(uw, su, u[i]);
      } else if constexpr (EXTRA > 0) {
        const uint32_t w = at + r16 * 128 + (((2 * i + (kg >> 1)) ^ (r16 & 7)) << 4) + ((kg & 1) << 3);
        const u32x2 gw = read8(w), uw = read8(w + 2048);
        g[i][0] = bf16_lo(gw.x); g[i][1] = bf16_hi(gw.x); g[i][2] = bf16_lo(gw.y); g[i][3] = bf16_hi(gw.y);
        u[i][0] = bf16_lo(uw.x); u[i][1] = bf16_hi(uw.x); u[i][2] = bf16_lo(uw.y); u[i][3] = bf16_hi(uw.y);
      } else {
        load4((const T*)a.kept + 2 * p * I + c, g[i]);
        load4((const T*)a.kept + (2 * p + 1) * I + c, u[i]);
      }
    }
    Piece hv, gv, uv;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float d[4], h[4], dg[4], du[4];
      sum4((4 * half + i) % MI, j, d);
#pragma unroll
      for (int q = 0; q < 4; ++q) gated_grad(g[i][q], u[i][q], d[q], h[q], dg[q], du[q]);
      take(hv, i, h);
      take(gv, i, dg);
      take(uv, i, du);
    }
    store(hv, (T*)a.act + p0 * I + c0, I, left, cols);
    store(gv, (T*)a.dgu + 2 * p0 * I + c0, 2 * I, left, cols);
    store(uv, (T*)a.dgu + (2 * p0 + 1) * I + c0, 2 * I, left, cols);
  };
  // stage e of kept rows, lying in this wave's part of a slot
  auto gradients = [&](const Meta& m, int e, uint32_t at_slot) __attribute__((always_inline)) {
    const uint32_t at = ring0 + at_slot + 4096 * wv;
    if constexpr (MODE == DACT) {
      gradients16(m, e >> 1, e & 1, at);
    } else {
      gradients16(m, e, 0, at);
      gradients16(m, e, 1, at);
    }
  };
  auto outputs = [&](const Meta& m) __attribute__((always_inline)) {
    if constexpr (GU) {
      const int c0 = m.m0 + 64 * wm, cols = I - c0;
      if (cols <= 0) return;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        __builtin_amdgcn_sched_barrier(0);
        const int row0 = m.n0 + 16 * NJ * wn + 16 * j, left = m.n - row0;
        if (left <= 0) break;
        const int64_t p0 = m.start + row0;
        uint32_t code[2][4];
        if constexpr (MODE == GATE_UP8) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v[4];
              sum4(4 * w + i, j, v);
              if (16 * i < cols)
#pragma unroll
                for (int q = 0; q < 4; ++q) top = max(top, __float_as_uint(v[q]) & 0x7FFFFFFFu);
            }
            top = max(top, (uint32_t)__shfl_xor((int)top, 16));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            float scale;
            const float inv = pack8_inverse(__uint_as_float(top), scale);
            if (kg == w && r16 < left) a.scale[(2 * (p0 + r16) + w) * a.blocks + c0 / 64] = scale;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v[4];
              sum4(4 * w + i, j, v);
              code[w][i] = pack8x4(v, inv);
            }
          }
        }
        Piece hv, gv, uv;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float g[4], u[4], h[4];
          sum4(i, j, g);
          sum4(i + 4, j, u);
#pragma unroll
          for (int q = 0; q < 4; ++q) h[q] = silu_f(g[q]) * u[q];
          take(hv, i, h);
          if constexpr (MODE == GATE_UP) {
            take(gv, i, g);
            take(uv, i, u);
          }
        }
        store(hv, (T*)a.act + p0 * I + c0, I, left, cols);
        if constexpr (MODE == GATE_UP) {
          store(gv, (T*)a.kept + 2 * p0 * I + c0, 2 * I, left, cols);
          store(uv, (T*)a.kept + (2 * p0 + 1) * I + c0, 2 * I, left, cols);
        } else {   // codes: 64 bytes of g, then of u, of 16 rows
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *(lds4_t*)(uintptr_t)(mine0 + r16 * 128 + (((4 * w + i) ^ (r16 & 7)) << 4) + 4 * kg) = code[w][i];
          wait_lds();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = 8 * h + (lane >> 3), c = lane & 7;
            const u32x4 v = read16(mine0 + r * 128 + ((c ^ (r & 7)) << 4));
            if (r < left && 16 * (c & 3) < cols)
              *reinterpret_cast<u32x4*>((int8_t*)a.kept + (2 * (p0 + r) + (c >> 2)) * I + c0 + 16 * (c & 3)) = v;
          }
          wait_lds();
        }
      }
    } else if constexpr (MODE == DOWN || MODE == DX || MODE == DW) {
      const int M = MODE != DW ? H : m.which == 2 ? I : H, N = MODE != DW ? m.n : m.which == 2 ? H : I;
      T* out = MODE == DOWN ? (T*)a.y + (int64_t)m.start * H : MODE == DX ? (T*)a.dx + (int64_t)m.start * H
               : (T*)a.dw[m.which] + (int64_t)m.e * I * H;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int row0 = m.n0 + 16 * NJ * wn + 16 * j;
#pragma unroll
        for (int half = 0; half < MI / 4; ++half) {
          __builtin_amdgcn_sched_barrier(0);
          const int c0 = m.m0 + 16 * MI * wm + 64 * half;
          if (row0 >= N || c0 >= M) continue;
          Piece w;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v[4];
            sum4(4 * half + i, j, v);
            take(w, i, v);
          }
          store(w, out + (int64_t)row0 * M + c0, M, N - row0, M - c0);
        }
      }
    } else if constexpr (DA) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int half = 0; half < MI / 4; ++half)
          if (m.n0 + 16 * NJ * wn + 16 * j < m.n && m.m0 + 16 * MI * wm + 64 * half < I) gradients16(m, j, half, 0);
    } else {
      const int M = m.which == 2 ? I : H, N = m.which == 2 ? H : I;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        __builtin_amdgcn_sched_barrier(0);
        const int row = m.n0 + 16 * NJ * wn + 16 * j + r16;
        const int64_t at = (int64_t)m.e * I * H + (int64_t)row * M + m.m0 + 16 * MI * wm + 4 * kg;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          float v[4], was[4];
          sum4(i, j, v);
          if (row >= N || m.m0 + 16 * MI * wm + 16 * i >= M) continue;
          if (a.dw_f32) {
            float* to = (float*)a.dw[m.which] + at + 16 * i;
            if (a.accumulate) {
              load4(to, was);
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] += was[q];
            }
            store4(to, v);
          } else {
            bf16* to = (bf16*)a.dw[m.which] + at + 16 * i;
            load4(to, was);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += was[q];
            store4(to, v);
          }
        }
      }
    }
  };
