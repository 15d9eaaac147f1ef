// w4_plan.h -- sizes of packed 4-bit weights and how the few-token product
// spreads over waves (host code alone).
//
// Rows go in tiles of 16 and columns in tiles of 128, both rounded up:
//   codes [N / 16][K / 128][64 lanes][16 bytes]: lane l holds row l % 16 and, in
//         32-bit word s, columns 32 s + 8 (l / 16) .. + 7 of the tile, in nibbles
//         0 4 1 5 2 6 3 7 (columns 0, 1 are nibbles 0 and 4, ...);
//   scale [N / 16][K / 128][4][128 / group][4] bf16: rows 4 q + i (q, i the
//         first and last index); zero the same in bytes.
// Padding holds zeros (scale 0).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace hdq {

constexpr int kW4TileN = 16, kW4TileK = 128;

inline int64_t w4_tiles_n(int64_t N) { return (N + kW4TileN - 1) / kW4TileN; }
inline int64_t w4_tiles_k(int64_t K) { return (K + kW4TileK - 1) / kW4TileK; }
inline size_t w4_code_bytes(int64_t N, int64_t K) { return (size_t)(w4_tiles_n(N) * w4_tiles_k(K)) * 1024; }
inline size_t w4_scale_count(int64_t N, int64_t K, int group) {
  return (size_t)(w4_tiles_n(N) * w4_tiles_k(K)) * (size_t)(16 * (kW4TileK / group));
}

struct W4Plan {
  int mt, nt;       // tiles of 16 tokens, of 16 rows, that a wave multiplies
  int wn, wk;       // waves of a workgroup along the rows, and along K
  int64_t grid_x, grid_y;
};

// Waves wanted: eight for each CU.
constexpr int64_t kW4Waves = 2048;

inline W4Plan plan_w4(int64_t M, int64_t N, int64_t K) {
  W4Plan p;
  const int64_t tm = (M + 15) / 16, tn = w4_tiles_n(N), tk = w4_tiles_k(K);
  p.mt = tm == 1 ? 1 : tm == 2 ? 2 : 4;
  p.nt = p.mt == 1 ? 1 : 2;
  p.grid_y = (tm + p.mt - 1) / p.mt;
  const int64_t gn = (tn + p.nt - 1) / p.nt, want = (kW4Waves + gn * p.grid_y - 1) / (gn * p.grid_y);
  const int64_t most = p.mt == 4 ? 8 : 16;
  int64_t wk = want < tk ? want : tk;
  if (wk > most) wk = most;
  // the same number of tiles for each wave, as far as that goes
  const int64_t each = (tk + wk - 1) / wk;
  wk = (tk + each - 1) / each;
  p.wk = (int)wk;
  p.wn = wk >= 4 ? 1 : (int)(4 / wk);
  p.grid_x = (gn + p.wn - 1) / p.wn;
  return p;
}

}  // namespace hdq
