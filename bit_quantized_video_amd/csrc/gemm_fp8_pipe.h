// gemm_fp8_pipe.h -- the pipelined FP8 block-128 GEMM body for large layers.
#pragma once

#include "gemm_fp8_tile.h"

namespace hdq {

// Tiles of BM x BN = 32 WM_T x 64 WN_T: the eight waves are 2 (tokens) x 4
// (features), each of 16 WM_T x 16 WN_T.  A persistent tile loop with
// the tile order of the other GEMMs.  A stage is one block of 128 k: the tile's
// X and W codes and its activation scales, brought into one of two LDS buffers
// by LDS-DMA while the other is computed.  Code rows are 128 bytes with 16-byte
// chunk c of row r at chunk c ^ (r & 7) (applied on the global side): a fragment
// read of 16 rows x 4 chunks then takes the 4 cycles that 1 KB needs (an
// in-bounds probe; 8 with the swizzle of the 32-row fragments, 16 without one).
// The weights' scale of the wave's features is a scalar.
//
// At no single limit: 256 x 256 tiles, 17776 x 3072 -> 12288, bf16 output, take
// 603 to 640 us (2.1 PFLOP/s), 1.24M cycles in which the matrix units are busy
// for 0.52 and 18 bytes per clock and CU come in, where k_fp8_deep takes in 24 and
// more.  A loop of products and scalings alone runs at 3.7 PFLOP/s (at 1.8 GHz),
// the kernel without its loads in 570 us.  What is lost: the stage barrier waits
// for every load in flight, and 3360 tiles are 14 rounds of 240 workgroups, with 16
// CUs idle.  The clock gives way, too: an order with 10% fewer cycles took as
// long (2.14 -> 1.98 GHz).  fp32 output, 17776 x 1920 -> 5760: 386 us, 1.0 PFLOP/s
// of twice the matrix work; 4050 x 1920 -> 5760: matrix units busy for 0.38, 9
// bytes per clock and CU: the conversions to bf16 and the LDS reads are not
// hidden behind the products.  A 128 x 256 tile
// takes 0.62 (fp32) to 0.74 of the time of a 256 x 256 one (1350 x 1920 -> 5760, one
// round of each: 19.9 and 27.1 us); a third stage buffer, which it leaves room
// for, changed nothing (20.8), and 128 x 128 tiles of four waves, two of them on a
// CU, were slower (21.2).
constexpr int kPipeWaves = 8, kPipeThreads = 64 * kPipeWaves;
template <int WM_T, int WN_T>
struct Fp8Tile {
  static constexpr int BM = 32 * WM_T, BN = 64 * WN_T;
  static constexpr int XB = BM * kFp8Block, WB = BN * kFp8Block;
  static constexpr int OUT_PITCH = BN * 2 + 16;                // bf16 output row staged in LDS
  static constexpr int kNeed = XB + WB + 4 * kPipeThreads;     // scales: one 4-byte slot per thread
  static constexpr int kOut = BM / 2 * OUT_PITCH;              // half an output tile
  static constexpr int STAGE = ((kNeed > kOut ? kNeed : kOut) + 1023) / 1024 * 1024;
  static constexpr int LDS = 2 * STAGE;
  static_assert(BM <= kPipeThreads / 2 && kFp8Block % (16 * WN_T) == 0 && LDS <= 160 * 1024, "tile shape");
};

template <int OUT, int WM_T, int WN_T>
__device__ __forceinline__ void gemm_fp8_pipe_body(const uint8_t* __restrict__ xc, const float* __restrict__ xs,
                                                   const uint8_t* __restrict__ wc, const float* __restrict__ ws,
                                                   void* __restrict__ Y, int64_t M, int N, int kb) {
  constexpr bool FAST = OUT == kOutBf16;
  using Tile = Fp8Tile<WM_T, WN_T>;
  constexpr int BM = Tile::BM, BN = Tile::BN, XB = Tile::XB, SB = Tile::STAGE, kOutPitch = Tile::OUT_PITCH;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % 2, wn = wave / 2;
  // The tile's loads are issued by LOADERS waves; a wave is held up while it
  // issues, so of the two waves on a SIMD one issues none.
  constexpr int LOADERS = kPipeWaves / 2;
  const bool loader = wave < LOADERS;
  const int tiles_m = (int)((M + BM - 1) / BM), tiles_n = (N + BN - 1) / BN;
  const TileSeq seq = tile_seq(tiles_m * tiles_n);
  const int G = seq.count * kb;
  if (G == 0) return;
  const int ld = kb * kFp8Block, nblocks = (N + kFp8Block - 1) / kFp8Block;

  // LDS-DMA: instruction p of wave w fills rows 8 LOADERS p + 8 w + (lane >> 3),
  // slot lane & 7
  constexpr int ROWS = 8 * LOADERS;
  const int drow = 8 * (wave % LOADERS) + (lane >> 3);
  const uint32_t dvoff = (uint32_t)(drow * ld + 16 * ((lane & 7) ^ (drow & 7)));

  int l_logical = seq.first, l_kt = 0;
  int64_t l_m0 = 0;
  __amdgpu_buffer_rsrc_t xres, wres;
  auto open_tile = [&]() {
    int tm, tn;
    grouped_tile(l_logical, tiles_m, tiles_n, tm, tn);
    l_m0 = (int64_t)tm * BM;
    const int n0 = tn * BN;
    // at most one tile's rows: offsets stay within 256 x 2^22
    xres = make_rsrc(xc + l_m0 * ld, (uint32_t)min((int64_t)BM, M - l_m0) * (uint32_t)ld);
    wres = make_rsrc(wc + (int64_t)n0 * ld, (uint32_t)min(BN, N - n0) * (uint32_t)ld);
  };
  open_tile();
  auto issue = [&](int buf) {
    if (loader) {
      uint8_t* base = smem + buf * SB + 1024 * wave;
#pragma unroll
      for (int p = 0; p < BM / ROWS; ++p)
        lds_dma16(xres, base + 128 * ROWS * p, dvoff, l_kt * kFp8Block + p * ROWS * ld);
#pragma unroll
      for (int p = 0; p < BN / ROWS; ++p)
        lds_dma16(wres, base + XB + 128 * ROWS * p, dvoff, l_kt * kFp8Block + p * ROWS * ld);
      const __amdgpu_buffer_rsrc_t sres =
          make_rsrc(xs + (int64_t)l_kt * M + l_m0, (uint32_t)min((int64_t)BM, M - l_m0) * 4u);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          sres, (__attribute__((address_space(3))) void*)(smem + buf * SB + XB + Tile::WB + 256 * wave), 4, 4 * tid, 0, 0,
          0);
    }
    if (++l_kt == kb) {
      l_kt = 0;
      l_logical += seq.stride;
      if (l_logical < tiles_m * tiles_n) open_tile();
    }
  };

  v4f acc[WN_T][WM_T];
  auto zero_acc = [&]() {
#pragma unroll
    for (int j = 0; j < WN_T; ++j)
#pragma unroll
      for (int i = 0; i < WM_T; ++i) acc[j][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  };
  zero_acc();
  const int r16 = lane & 15, q = lane >> 4;
  auto frag = [&](const uint8_t* rows, int r) {
    return load_frag(rows + r * 128 + 16 * (q ^ (r & 7)), rows + r * 128 + 16 * ((q + 4) ^ (r & 7)));
  };
  auto compute = [&](int buf, float sw) {
    const uint8_t* lx = smem + buf * SB;
    const uint8_t* lw = lx + XB;
    const float* ls = reinterpret_cast<const float*>(lw + Tile::WB) + wm * 16 * WM_T + r16;
    Fp8Operand<FAST> w[WN_T];
#pragma unroll
    for (int j = 0; j < WN_T; ++j) w[j].set(frag(lw, wn * 16 * WN_T + 16 * j + r16));
    // Software pipeline: product t of the wave's is issued together with
    // the scaling and adding of product t - LAG, so its readers are always LAG
    // matrix instructions behind it, and token fragment i + 2 is read when
    // fragment i's last product has been issued.
    constexpr int LAG = FAST ? 3 : 1;  // a product is one matrix instruction, or four in a chain
    Fp8Frag x[2];
    v4f p[LAG + 1];
    float sx[3];  // fragment i's activation scales in sx[i % 3]
    auto read = [&](int i) {
      x[i & 1] = frag(lx, wm * 16 * WM_T + 16 * i + r16);
      sx[i % 3] = ls[16 * i];
    };
    read(0);
    read(1);
    float s[2];
#pragma unroll
    for (int t = 0; t < WM_T * WN_T + LAG; ++t) {
      const int i = t / WN_T, j = t % WN_T;
      if (t < WM_T * WN_T) {
        Fp8Operand<FAST> xo;
        xo.set(x[i & 1]);
        if (j == 0) s[i & 1] = sx[i % 3] * sw;
        p[t % (LAG + 1)] = block_product(w[j], xo);
      }
      if (t >= LAG) {
        const int u = t - LAG;
        add_scaled(acc[u % WN_T][u / WN_T], p[u % (LAG + 1)], s[(u / WN_T) & 1]);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (j == WN_T - 1 && i + 2 < WM_T) read(i + 2);
    }
  };

  auto epilogue = [&](int logical, int buf) {
    // recomputed here: kept over the main loop, these addresses would spill,
    // and a reload waits for the loads in flight
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave % 2, wn = wave / 2;
    const int r16 = lane & 15, q = lane >> 4;
    int tm, tn;
    grouped_tile(logical, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * BM;
    const int n0 = tn * BN;
    if constexpr (OUT == kOutBf16) {
      // Half a tile at a time through buffer buf, which this stage has been
      // computed from: half hh holds fragments hh WM_T / 2 + 0 .. WM_T / 2 - 1 of
      // both wave rows, then whole rows are stored.  The barriers wait for LDS
      // only: the next stage's loads stay in flight.
      constexpr int HM = 8 * WM_T, PIECES = BN / 8;  // rows of a wave row's half, 16-byte pieces of a row
      uint8_t* const stage = smem + buf * SB;
      uint16_t* y16 = static_cast<uint16_t*>(Y);
      const int n = n0 + 8 * (tid % PIECES);
      const bool vec = n + 8 <= N;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        lds_only_barrier();
        uint8_t* const lrow = stage + (wm * HM + r16) * kOutPitch + 2 * (wn * 16 * WN_T + 4 * q);
#pragma unroll
        for (int ii = 0; ii < WM_T / 2; ++ii)
#pragma unroll
          for (int j = 0; j < WN_T; ++j) {
            const v4f& a = acc[j][WM_T / 2 * hh + ii];
            *reinterpret_cast<uint2*>(lrow + ii * 16 * kOutPitch + 32 * j) =
                make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
          }
        lds_only_barrier();
#pragma unroll 4
        for (int r = tid / PIECES; r < 2 * HM; r += kPipeThreads / PIECES) {
          const uint8_t* src = stage + r * kOutPitch + 16 * (tid % PIECES);
          const int64_t m = m0 + r / HM * (2 * HM) + hh * HM + r % HM;
          if (m < M) {
            uint16_t* dst = y16 + m * N + n;
            if (vec) {
              __builtin_nontemporal_store(*reinterpret_cast<const v4i*>(src), reinterpret_cast<i32x4_a2*>(dst));
            } else {
              for (int e = 0; e < 8 && n + e < N; ++e) dst[e] = reinterpret_cast<const uint16_t*>(src)[e];
            }
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < WM_T; ++i) {
        const int64_t m = m0 + wm * 16 * WM_T + 16 * i + r16;
        if (m >= M) continue;
#pragma unroll
        for (int j = 0; j < WN_T; ++j) store_out4<OUT>(Y, m, n0 + wn * 16 * WN_T + 16 * j + 4 * q, N, acc[j][i]);
      }
    }
  };

  // The weights' scales of the tile being computed: this wave's block row, read
  // through the constant address space (scalar loads: a vector load would wait
  // for the DMA loads issued before it).
  typedef const __attribute__((address_space(4))) float* ConstFloats;
  int ckt = 0, clogical = seq.first;
  ConstFloats wsp = (ConstFloats)(uintptr_t)ws;
  auto open_scales = [&]() {
    int tm, tn;
    grouped_tile(clogical, tiles_m, tiles_n, tm, tn);
    const int nb = min((tn * BN + wn * 16 * WN_T) / kFp8Block, nblocks - 1);
    wsp = (ConstFloats)(uintptr_t)ws + (int64_t)nb * kb;
  };
  open_scales();
  float sw = wsp[0];
  // Ends a stage; the next one's scale is on its way before the stage barrier.
  auto finish_stage = [&](int buf) {
    if (++ckt == kb) {
      epilogue(clogical, buf);
      zero_acc();
      ckt = 0;
      clogical += seq.stride;
      if (clogical < tiles_m * tiles_n) open_scales();
    }
    sw = wsp[ckt];
  };

  // Stage g lives in buffer g % 2; stage g + 1 is issued when stage g's compute
  // starts, into the buffer every wave finished reading before the last barrier.
  // Only the loaders wait for vector memory; the others' stores stay in flight.
  auto end_stage = [&]() {
    if (loader) wait_vmem<0>();
    lds_only_barrier();
  };
  issue(0);
  end_stage();
  for (int g0 = 0; g0 < G; g0 += 2) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (g0 + u < G) {
        if (g0 + u + 1 < G) issue(u ^ 1);
        compute(u, sw);
        finish_stage(u);
        end_stage();
      }
    }
  }
}

}  // namespace hdq
