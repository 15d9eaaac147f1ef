// w4_plan.h -- sizes of packed 4-bit weights and how the few-token product
// spreads over waves (no HIP types).
//
// Rows go in tiles of 16 and columns in tiles of 128, both rounded up:
//   codes [N / 16][K / 128][64 lanes][16 bytes]: lane l holds row l % 16 and, in
//         32-bit word s, columns 32 s + 8 (l / 16) .. + 7 of the tile, in nibbles
//         0 4 1 5 2 6 3 7 (columns 0, 1 are nibbles 0 and 4, ...), the word
//         rotated left by 3 bits;
//   scale [N / 16][K / 512][16][512 / group] bf16 (four tiles of a row in one
//         load), zero the same in bytes.
// Padding holds zeros.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace hdq {

constexpr int kW4TileN = 16, kW4TileK = 128;

inline int64_t w4_tiles_n(int64_t N) { return (N + kW4TileN - 1) / kW4TileN; }
inline int64_t w4_tiles_k(int64_t K) { return (K + kW4TileK - 1) / kW4TileK; }
inline size_t w4_code_bytes(int64_t N, int64_t K) { return (size_t)(w4_tiles_n(N) * w4_tiles_k(K)) * 1024; }
inline size_t w4_scale_count(int64_t N, int64_t K, int group) {
  return (size_t)(w4_tiles_n(N) * ((w4_tiles_k(K) + 3) / 4)) * (size_t)(64 * (kW4TileK / group));
}
// Index of group kg of row n of row tile tn; groups: of a tile.
#ifdef __HIPCC__
__host__ __device__
#endif
inline int64_t w4_group_at(int64_t tn, int64_t n, int64_t kg, int64_t tiles_k, int groups) {
  return ((tn * ((tiles_k + 3) / 4) + kg / (4 * groups)) * 16 + n) * (4 * groups) + kg % (4 * groups);
}

// How a product runs.
//   k_w4_direct: up to 64 tokens and few rows.  A workgroup has one tile of
//     rows and a wave for every four tiles of K (two or one from 17 and 33 tokens
//     on; at most 16 waves), which loads all it needs at once, the tokens
//     straight from L2.
//   k_w4: up to 16 tokens that fit LDS.  A workgroup keeps them there and
//     streams weights.
//   k_w4_shared: else.  A workgroup of eight waves shares 64 tokens (16 or 32
//     where there are no more) a stage at a time among 128 rows, and K is split
//     over workgroups, whose sums a second launch adds, where there are too few.
struct W4Plan {
  bool direct;     // k_w4_direct
  int per;         // k_w4: tiles of rows of a wave; with neither k_w4_shared
  int wn, wk;      // waves of a workgroup along the rows, and along K
  int step, part;  // k_w4: wn * wk waves in whole tokens of a block of K each, and the rest
  size_t lds;
  int mt;          // k_w4_direct, k_w4_shared: tiles of 16 tokens of a workgroup
  int split;       // workgroups along K
  int64_t grid_x, grid_y;
};

// k_w4_direct: rows in tiles (three workgroups a CU), waves (as many as run at a
// time) and bytes of tokens that a CU's workgroups read.  Within these it is the
// faster one (us on the GPU; k_w4, or k_w4_shared and its second launch):
//   1 x 4096 -> 4096 4.3 (4.6), 16 x 1920 -> 1920 4.7 (6.8), -> 12288 9.1 (14.5),
//   13 x 4096 -> 4096 6.7 (5.0 + 2.4, and 7.2 for 11.1 a call), 32 x 1920 -> 1920
//   6.3 (6.2 + 2.2), 64 x 1024 -> 4096 7.2 (7.6 + 2.5).
// Past them it is not: 4 x 512 -> 65536 8.6 (6.7; 4096 tiles of rows), 16 x 4096
// -> 8192 11.6 (7.0 + 2.4; 256 KB), 32 x 4096 -> 4096 10.6 (7.3 + 3.0; 256 KB).
constexpr int64_t kW4DirectTiles = 768, kW4DirectWaves = 4096, kW4DirectBytes = 192 << 10;
constexpr int64_t kW4Waves = 4096;    // waves wanted of k_w4: 16 a CU, what its registers leave room for
constexpr size_t kW4Lds = 64 << 10;   // LDS its tokens may take: 13 x 4096 -> 1921 in 106 KB took 8.2 us (5.4 + 2.5 shared)
constexpr int64_t kW4Groups = 256;    // workgroups wanted of k_w4_shared, one a CU: with 512 its sums cost what it gains
constexpr int64_t kW4LeastTiles = 4;  // tiles of K that a split keeps at least: a stage is a tile, and two are loaded ahead

inline W4Plan plan_w4(int64_t M, int64_t N, int64_t K) {
  W4Plan p = {};
  const int64_t tm = (M + 15) / 16, tn = w4_tiles_n(N), tk = w4_tiles_k(K);
  p.split = 1;
  p.lds = (size_t)M * (size_t)(tk * 256 + 16);
  const int64_t blocks = (tk + 3) / 4;
  p.mt = tm <= 2 ? (int)tm : 4;
  const int64_t parts = (tk * p.mt + 3) / 4;  // waves of k_w4_direct
  if (tm <= 4 && parts <= 16 && tn <= kW4DirectTiles && tn * parts <= kW4DirectWaves &&
      (tn + 255) / 256 * M * K * 2 <= kW4DirectBytes) {
    p.direct = true;
    p.wn = 1;
    p.wk = (int)parts;
    p.lds = (size_t)(parts * p.mt) * 1024;
    p.grid_x = tn;
    p.grid_y = 1;
  } else if (tm == 1 && p.lds <= kW4Lds) {
    p.grid_y = 1;
    // waves of a tile of rows: as many as there are blocks of four tiles of K, and tiles of rows to go round
    int64_t wk = kW4Waves / tn < blocks ? kW4Waves / tn : blocks;
    wk = wk > 16 ? 16 : wk < 1 ? 1 : wk;
    const int64_t each = (blocks + wk - 1) / wk;  // the same number of blocks for each, as far as that goes
    wk = (blocks + each - 1) / each;
    p.wk = (int)wk;
    p.wn = wk >= 4 ? 1 : (int)(8 / wk);
    p.step = (int)(p.wn * p.wk / blocks);
    p.part = (int)(p.wn * p.wk % blocks);
    p.per = wk > 1 ? 1 : (int)((tn + kW4Waves - 1) / kW4Waves);
    p.grid_x = (tn + p.wn * p.per - 1) / (p.wn * p.per);
    if (wk > 1 && p.lds < (size_t)(p.wn * p.wk) * 1024) p.lds = (size_t)(p.wn * p.wk) * 1024;
  } else {
    p.wn = 8;
    p.wk = 1;
    p.grid_x = (tn + 7) / 8;
    p.grid_y = (tm + p.mt - 1) / p.mt;
    const int64_t most = tk / kW4LeastTiles;
    int64_t split = (kW4Groups + p.grid_x * p.grid_y - 1) / (p.grid_x * p.grid_y);
    if (split > most) split = most;
    if (split > 1) {
      const int64_t each = (tk + split - 1) / split;
      p.split = (int)((tk + each - 1) / each);
    }
  }
  return p;
}

// Scratch: the workgroups' float32 sums along K.
inline int64_t w4_slice(int64_t M, int64_t N) { return (M * N + 3) / 4 * 4; }
inline size_t w4_workspace(int64_t M, int64_t N, int64_t K) {
  const W4Plan p = plan_w4(M, N, K);
  return p.split > 1 ? (size_t)p.split * (size_t)w4_slice(M, N) * 4 : 0;
}

}  // namespace hdq
