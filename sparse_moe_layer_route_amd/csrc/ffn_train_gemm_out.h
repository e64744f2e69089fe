  // (part of train_gemm_kernel) A wave's 128 x 16 NJ accumulators: lane (r16, kg)
  // holds of tile (i, j) outputs m = 16 i + 4 kg..+3 of row n = 16 j + r16.
  // They go through LDS in pieces of 16 rows x 64 m, 16-byte chunk c of row r at
  // c ^ (r % 8), and out as runs of 128 bytes of a row.
  float scales[NJ];   // DACT8: of rows 16 j + r16, matrix kg % 2, block kg / 2
  auto before_tile = [&](const Meta& m) __attribute__((always_inline)) {
    if constexpr (MODE == DACT8) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int64_t p = m.start + min(m.n0 + 16 * NJ * wn + 16 * j + r16, m.n - 1);
        const int b = min((m.m0 + 128 * wm) / 64 + (kg >> 1), a.blocks - 1);
        scales[j] = a.scale[(2 * p + (kg & 1)) * a.blocks + b];
      }
    }
  };
  // v: bf16 pairs of this lane's four m of tiles i; to out[row * ld + m..] where
  // rows and columns are left
  auto store_piece = [&](const uint32_t (&v)[8], bf16* out, int64_t ld, int rows_left, int cols_left) __attribute__((always_inline)) {
    const int l = fresh_lane(), r16 = l & 15, kg = l >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      write8(mine0 + r16 * 128 + (((2 * i + (kg >> 1)) ^ (r16 & 7)) << 4) + ((kg & 1) << 3), v[2 * i], v[2 * i + 1]);
    wait_lds();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 8 * h + (l >> 3), c = l & 7;
      const u32x4 w = read16(mine0 + r * 128 + ((c ^ (r & 7)) << 4));
      if (r < rows_left && 8 * c < cols_left) *reinterpret_cast<u32x4*>(out + r * ld + 8 * c) = w;
    }
    wait_lds();
  };
  auto pack = [&](uint32_t (&to)[8], int i, const float (&v)[4]) __attribute__((always_inline)) {
    to[2 * i] = f2_to_bf16x2(v[0], v[1]);
    to[2 * i + 1] = f2_to_bf16x2(v[2], v[3]);
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
        uint32_t top[2] = {0, 0};
        uint32_t code[2][4];
        if constexpr (MODE == GATE_UP8) {
          float inv[2];
#pragma unroll
          for (int w = 0; w < 2; ++w) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v[4];
              acc_read4(acc[4 * w + i][j], v);
              if (16 * i < cols)
#pragma unroll
                for (int q = 0; q < 4; ++q) top[w] = max(top[w], __float_as_uint(v[q]) & 0x7FFFFFFFu);
            }
            top[w] = max(top[w], (uint32_t)__shfl_xor((int)top[w], 16));
            top[w] = max(top[w], (uint32_t)__shfl_xor((int)top[w], 32));
            float scale;
            inv[w] = pack8_inverse(__uint_as_float(top[w]), scale);
            if (kg == w && r16 < left) a.scale[(2 * (p0 + r16) + w) * a.blocks + c0 / 64] = scale;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v[4];
              acc_read4(acc[4 * w + i][j], v);
              code[w][i] = pack8x4(v, inv[w]);
            }
          }
        }
        uint32_t hv[8], gv[8], uv[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float g[4], u[4], h[4];
          acc_read4(acc[i][j], g);
          acc_read4(acc[i + 4][j], u);
#pragma unroll
          for (int q = 0; q < 4; ++q) h[q] = silu_f(g[q]) * u[q];
          pack(hv, i, h);
          if constexpr (MODE == GATE_UP) {
            pack(gv, i, g);
            pack(uv, i, u);
          }
        }
        store_piece(hv, (bf16*)a.act + p0 * I + c0, I, left, cols);
        if constexpr (MODE == GATE_UP) {
          store_piece(gv, (bf16*)a.kept + 2 * p0 * I + c0, 2 * I, left, cols);
          store_piece(uv, (bf16*)a.kept + (2 * p0 + 1) * I + c0, 2 * I, left, cols);
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
      bf16* out = MODE == DOWN ? (bf16*)a.y + (int64_t)m.start * H : MODE == DX ? (bf16*)a.dx + (int64_t)m.start * H
                  : (bf16*)a.dw[m.which] + (int64_t)m.e * I * H;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int row0 = m.n0 + 16 * NJ * wn + 16 * j;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          __builtin_amdgcn_sched_barrier(0);
          const int c0 = m.m0 + 128 * wm + 64 * half;
          if (row0 >= N || c0 >= M) continue;
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v[4];
            acc_read4(acc[4 * half + i][j], v);
            pack(w, i, v);
          }
          store_piece(w, out + (int64_t)row0 * M + c0, M, N - row0, M - c0);
        }
      }
    } else if constexpr (DA) {
    } else {
      const int M = m.which == 2 ? I : H, N = m.which == 2 ? H : I;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        __builtin_amdgcn_sched_barrier(0);
        const int row = m.n0 + 16 * NJ * wn + 16 * j + r16;
        const int64_t at = (int64_t)m.e * I * H + (int64_t)row * M + m.m0 + 128 * wm + 4 * kg;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v[4];
          acc_read4(acc[i][j], v);
          if (row >= N || m.m0 + 128 * wm + 16 * i >= M) continue;
          if (a.dw_f32) {
            float4* to = reinterpret_cast<float4*>((float*)a.dw[m.which] + at + 16 * i);
            if (a.accumulate) {
              const float4 w = *to;
              v[0] += w.x; v[1] += w.y; v[2] += w.z; v[3] += w.w;
            }
            *to = float4{v[0], v[1], v[2], v[3]};
          } else {
            uint2* to = reinterpret_cast<uint2*>((bf16*)a.dw[m.which] + at + 16 * i);
            const uint2 w = *to;
            v[0] += bf16_lo(w.x); v[1] += bf16_hi(w.x); v[2] += bf16_lo(w.y); v[3] += bf16_hi(w.y);
            *to = make_uint2(f2_to_bf16x2(v[0], v[1]), f2_to_bf16x2(v[2], v[3]));
          }
        }
      }
    }
  };
  // DACT: stage e of kept rows, lying in this wave's part of a slot
  auto gradients = [&](const Meta& m, int e, uint32_t at_slot) __attribute__((always_inline)) {
    const int j = MODE == DACT ? e >> 1 : e, l = fresh_lane(), r16 = l & 15, kg = l >> 4;
    const int row0 = m.n0 + 16 * NJ * wn + 16 * j, left = m.n - row0;
    const uint32_t at = ring0 + at_slot + 4096 * wv + r16 * 128;
#pragma unroll
    for (int z = 0; z < (MODE == DACT ? 1 : 2); ++z) {
      __builtin_amdgcn_sched_barrier(0);
      const int half = MODE == DACT ? e & 1 : z;
      const int c0 = m.m0 + 128 * wm + 64 * half, cols = I - c0;
      float sg = 1.f, su = 1.f;
      if constexpr (MODE == DACT8) {
        sg = __shfl(scales[j], r16 + 32 * half);
        su = __shfl(scales[j], r16 + 32 * half + 16);
      }
      uint32_t hv[8], gv[8], uv[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float d[4], g[4], u[4], h[4], dg[4], du[4];
        acc_read4(acc[4 * half + i][j], d);
        if constexpr (MODE == DACT) {
          const uint32_t c = (((2 * i + (kg >> 1)) ^ (r16 & 7)) << 4) + ((kg & 1) << 3);
          const u32x2 gw = read8(at + c), uw = read8(at + 2048 + c);
          g[0] = bf16_lo(gw.x); g[1] = bf16_hi(gw.x); g[2] = bf16_lo(gw.y); g[3] = bf16_hi(gw.y);
          u[0] = bf16_lo(uw.x); u[1] = bf16_hi(uw.x); u[2] = bf16_lo(uw.y); u[3] = bf16_hi(uw.y);
        } else {
          const uint32_t c = (((4 * half + i) ^ (r16 & 7)) << 4) + 4 * kg;
          unpack8x4(*(const lds4_t*)(uintptr_t)(at + c), sg, g);
          unpack8x4(*(const lds4_t*)(uintptr_t)(at + 2048 + c), su, u);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) gated_grad(g[q], u[q], d[q], h[q], dg[q], du[q]);
        pack(hv, i, h);
        pack(gv, i, dg);
        pack(uv, i, du);
      }
      const int64_t p0 = m.start + row0;
      store_piece(hv, (bf16*)a.act + p0 * I + c0, I, left, cols);
      store_piece(gv, (bf16*)a.dgu + 2 * p0 * I + c0, 2 * I, left, cols);
      store_piece(uv, (bf16*)a.dgu + (2 * p0 + 1) * I + c0, 2 * I, left, cols);
    }
  };
