// Which block shape a launch of the experts' training takes: plain C++, no HIP.
#pragma once
#include <algorithm>
#include <cstdint>

namespace moe {

// The launches; outputs m x n of each: GATE_UP 2 I x rows, DOWN H x rows, DACT
// I x rows, DX H x rows, DW H x I (twice) and I x H of every expert.
enum train_launch { TRAIN_GATE_UP, TRAIN_DOWN, TRAIN_DACT, TRAIN_DX, TRAIN_DW };
enum train_shape { SHAPE_256x256, SHAPE_256x128, SHAPE_128x64, SHAPE_64x64 };

constexpr int kTrainCus = 256;

// Tiles of n rows by m of `width` outputs that P rows of E experts may need,
// however they are shared out: every expert may end in a part of a tile.
inline int64_t train_row_tiles(int P, int E, int width, int n, int m) {
  return ((int64_t)P / n + std::min(E, P)) * (((int64_t)width + m - 1) / m);
}

// The rule.  P counts a batch's T * k pairs, as the host knows no others: with
// many of them not computed a launch has fewer tiles than are counted here.
// Times in us of the launch within forward and backward at
//   few:    64 tokens, H 2048, I 1408, 64 experts top-6 (6 rows an expert)
//   batch:  4096 tokens, H 1536, I 512, 40 experts top-8 (819 rows)
//   shared: 2048 tokens, H 2048, I 1408, one expert
//   small:  1000 tokens, H 256, I 512, 8 experts top-2, fp32
//   256x128  two blocks a CU, one's outputs beside the other's products: where
//            its tiles fill the CUs.  batch: gate/up 160, down 85, dact 122, dx
//            149, dw 304 (128x64: 207, 109, 133, 201, 446); with 256x256, when
//            every launch had it, gate/up 188, down 92, dact 157 (149, 78, 120)
//   256x256  one block a CU, half of the weights' traffic: dx of matrices that
//            outgrow an XCD's L2, which are fetched again for every 128 rows
//            (4096 tokens, H 3584, I 2560, 64 experts top-8: 1535 against 1908).
//            Four rounds of its tiles, or CUs stand idle: below
//   128x64   few tiles: shared down 25, dact 32, dx 44 (256x128: 30, 53, 60);
//            few rows: few gate/up 212, dact 66 (215, 83), with 8 tokens
//            gate/up 131 (143)
//   64x64    fewer: few down 74, with 8 tokens 41 (128x64: 81, 43); small down
//            17, dx 32, dact 18, dw 35 (24, 48, 20, 43)
// Where 256x128 begins, time with it over that with 128x64 by its tiles (bf16,
// one expert or 8 top-2, H and I of 256 to 2048):
//   gate/up  82-99 tiles 1.4-1.6; 130-176 1.0-1.5; 187 0.80; 192-196 1.0-1.2; 260-288 0.8-1.1
//   down     72-98 1.4-1.8; 128-136 1.1-1.5; 160-196 0.9-1.1; 258-288 0.8-1.05
//   dact     72-102 1.7-2.1; 128-164 1.3-1.7; 192-240 1.15-1.4; 258-294 0.9-1.2; 386-528 0.7-1.0
//   dx       72-98 1.4-1.6; 128-164 1.1-1.4; 192-196 0.9-1.15; 258-288 0.7-1.0
//   dw       96 1.2; 192 1.1-1.2; 272 0.6-0.7; 384 0.7-0.8
//   dx of H I >= 2^22, 256x256 over the better of both, by its own tiles: 8-48 2.3-2.4; 64-144 1.25-2.0;
//            160-272 0.9-1.05; 288-384 1.05-1.5; 462-910 0.8-1.2; 1008-1280 0.8-1.05; 2688 0.8
//   dx of few rows  268-320 1.2; 416 1.1; 520-536 0.9; 832-1312 0.9-1.0
// and fp32's 128x64 over 64x64 by the tiles of the former:
//   down, dact, dx  130-320 1.0-1.5; 514-576 0.95-1.2; 1028-1152 0.9-1.15
//   dw (twice its tiles of 256x128)  192 1.1-1.3; 768 0.93
// fp32 is bound by its matrix instructions, a sixteenth as fast, and takes
// the smaller shapes throughout, whose sums can be put aside.  The largest
// batches lose by it: the backward pass of 4096 tokens, H 2048, I 512, 32 experts
// top-4, a fifth of the slots not computed, 2014, and 1691 with 256x128.
inline train_shape train_shape_of(train_launch which, bool is_bf16, int P, int E, int H, int I) {
  const bool rows = which != TRAIN_DW, few = P < 64 * E;
  const int width = which == TRAIN_GATE_UP ? 2 * I : which == TRAIN_DACT ? I : H;
  auto up = [](int64_t v, int64_t m) { return (v + m - 1) / m; };
  const int64_t tiles = rows ? train_row_tiles(P, E, width, 128, 256)
                             : E * (2 * up(H, 256) * up(I, 128) + up(I, 256) * up(H, 128));
  if (!is_bf16) {
    if (which == TRAIN_GATE_UP) return SHAPE_128x64;
    const bool fills = rows ? train_row_tiles(P, E, width, 64, 128) >= 3 * kTrainCus : 2 * tiles >= 2 * kTrainCus;
    return fills ? SHAPE_128x64 : SHAPE_64x64;
  }
  if (which == TRAIN_DX && (int64_t)H * I >= (4 << 20) && P >= 256 * E &&
      train_row_tiles(P, E, H, 256, 256) >= 4 * kTrainCus)
    return SHAPE_256x256;
  if (rows && few) {
    if (which == TRAIN_DX && tiles >= 2 * kTrainCus) return SHAPE_256x128;
    return which == TRAIN_DOWN ? SHAPE_64x64 : SHAPE_128x64;
  }
  return tiles > (which == TRAIN_GATE_UP ? 176 : 192) ? SHAPE_256x128 : SHAPE_128x64;
}

}  // namespace moe
