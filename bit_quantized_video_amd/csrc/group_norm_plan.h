// group_norm_plan.h -- how a group norm runs, from its sizes alone: slabs, chunks,
// launches, workspace.  Host code without HIP types, so that a test without a GPU
// can look every launch over.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "launch_grid.h"

namespace hdq {

constexpr int kGnThreads = 512, kGnSlabThreads = 512;
constexpr int kGnMaxChunks = 512;   // of a sample's statistics
constexpr int kGnFinalThreads = 256, kGnFinalGroups = kGnFinalThreads / 64;  // of k_gn_final: a wave a group
constexpr int kGnCodeThreads = 256;  // of k_gn_apply_fp8
constexpr int kGnRows = 4;           // its row groups in flight

// Chunks of a sample's rows for a pass of about `total` workgroups that take
// `per` rows at least.  The statistics take 512, though bf16's registers leave one
// at a time per CU: with 256 some are shorter (1 x 691200 x 256 with SiLU 166 us
// a call, 512 of them 174) and some longer (100 x 6000 x 256, three chunks each,
// 166 and 154; 50000 x 301 39 and 35).  The normalization takes 8192 (175 us for
// the call above, 1024 of them 182).
inline void gn_chunks(int64_t total, int64_t n, int64_t length, int64_t per, int64_t& chunks, int64_t& rows_per) {
  int64_t want = (total + n - 1) / n;
  if (want > (length + per - 1) / per) want = (length + per - 1) / per;
  if (want < 1) want = 1;
  rows_per = (length + want - 1) / want;
  chunks = (length + rows_per - 1) / rows_per;
}

// 16-byte vectors where the channels allow, else 8 bytes of bf16, else one channel
inline int64_t gn_vec(int64_t C, bool f32) { return C % 8 == 0 && !f32 ? 8 : C % 4 == 0 ? 4 : 1; }
inline int64_t gn_rpar(int64_t C, int64_t vec) {
  const int64_t cv = C / vec;
  return cv >= kGnThreads ? 1 : kGnThreads / cv;
}

// How a call runs (a rule on its sizes alone; the workspace follows it).
constexpr int64_t kGnKeep = 16, kGnStream = 64;  // rows a thread keeps / streams at most
// k_gn_short_fp8: channels and elements of a sample at most, rows of a workgroup
constexpr int64_t kGnBriefChannels = 512, kGnBriefSample = 96 << 10, kGnBriefRows = 16;
// elements of x and pairs of a sample up to which the normalization joins the chunks
constexpr int64_t kGnJoinElements = 3 << 19, kGnJoinPairs = 1024;
struct GnPlan {
  int64_t vec;
  bool merge;            // a vector lies in one group
  int64_t width, slabs;  // channels of a slab, slabs per sample
  int64_t threads, rows; // of a slab: threads, and rows per thread
  bool keep;             // the slab is kept in registers (not for the FP8 form)
  bool slab;             // the statistics are a slab's
  bool brief;            // the FP8 form takes one launch
  bool join;             // the normalization joins the chunks
  int64_t chunks, rows_per;              // of the statistics' rows
  int64_t apply_chunks, apply_rows;      // of the normalization's
  int64_t code_chunks, code_rows;        // of its FP8 form's
  // The launches' workgroups: a slab each, or the chunks' statistics (both also
  // ahead of a normalization), their join, the normalization, its FP8 form, the
  // FP8 form in one launch.
  Grid slab_grid, partial_grid, final_grid, apply_grid, code_grid, brief_grid;
};

inline GnPlan gn_plan(int64_t n, int64_t length, int64_t C, int64_t groups, bool f32) {
  GnPlan p;
  p.vec = gn_vec(C, f32);
  const int64_t cg = C / groups;
  p.merge = cg % p.vec == 0;
  int64_t unit = cg;  // channels of the fewest whole groups that are whole vectors
  while (unit % p.vec != 0) unit += cg;
  // slabs of at least 64 channels, fewer where that leaves CUs without work
  int64_t k = 1;
  while (k * unit < 64 && n * (C / ((k + 1) * unit)) >= 256) ++k;
  p.width = k * unit < C ? k * unit : C;
  p.slabs = (C + p.width - 1) / p.width;
  const int64_t cv = p.width / p.vec;
  // the fewest threads whose registers hold the slab: fewer pairs to join
  p.threads = 0;
  p.rows = kGnStream + 1;
  for (const int64_t t : {(int64_t)256, (int64_t)kGnSlabThreads}) {
    if (cv > t) continue;
    p.threads = t;
    p.rows = (length + t / cv - 1) / (t / cv);
    if (p.rows <= kGnKeep) break;
  }
  // Kept in registers: up to 16 rows of 128 bytes or more; 8 of narrower ones,
  // whose lines several workgroups share (13 x 675 x 512, 6 rows of 32 bytes:
  // 10.8 us, with two launches 12.1; 13 x 4000 x 512, 16 rows of 512 threads: 53.9
  // and 40.1).
  p.keep = p.threads == 256 && p.rows <= (p.width * (f32 ? 4 : 2) >= 128 ? kGnKeep : kGnKeep / 2);
  // A larger slab is streamed by one workgroup only where there is one for every
  // CU: with few of them the chunks' three launches are faster (1 x 16384 x 128:
  // 12.4 us against 26.0).
  p.slab = p.keep || (p.threads == 256 && p.rows <= kGnKeep) || (p.rows <= kGnStream && n * p.slabs >= 256);
  // About as long on the GPU as two launches (225 x 320: 10.7 us and 9.5; 64 x 512:
  // 8.0 and 8.2; longer or wider samples lose: 225 x 1280 22.8 and 9.2), for one
  // launch's host time and no workspace.  A sample's workgroups read it again
  // each, so either it has one (1000 x 16 x 512: 26.2 and 50.8) or all run at a
  // time (13 x 225 x 320: 11.0 and 9.8; 64 x 225 x 320, 960 of them: 41.7 and 14.7).
  p.brief = C <= kGnBriefChannels && length * C <= kGnBriefSample &&
            (length <= kGnBriefRows || n * ((length + kGnBriefRows - 1) / kGnBriefRows) <= 256);
  gn_chunks(kGnMaxChunks, n, length, 8 * gn_rpar(C, p.vec), p.chunks, p.rows_per);
  // A launch less, and no longer on the GPU: 984 x 537, one group 13.5 us, joined
  // here 10.3; 6469 x 64 fp32 (832 pairs) 11.5 and 10.6; 2 x 3000 x 256 to FP8 14.1
  // and 13.6.  With more rows or pairs it is longer (16384 x 128, 256 pairs 12.4
  // and 13.8; 5000 x 256, 1280 pairs 12.7 and 14.7).
  p.join = !p.slab && n * length * C <= kGnJoinElements && p.chunks * groups <= kGnJoinPairs;
  gn_chunks(8192, n, length, 4 * gn_rpar(C, p.vec), p.apply_chunks, p.apply_rows);
  // One pass of a wave's loop: more rows a workgroup were slower (13 x 1350 x
  // 512 with its statistics: 21.3 us, 32 rows 22.5; 17776 x 1280: 41.0 and 43.2),
  // but for a grid past kWideRow workgroups.
  const int64_t kgroups = ((C + 127) / 128 + 3) / 4, passes = (length + 4 * kGnRows - 1) / (4 * kGnRows);
  const int64_t most = std::max<int64_t>(1, kWideRow / (n * kgroups));
  p.code_rows = 4 * kGnRows * ((passes + most - 1) / most);
  p.code_chunks = (length + p.code_rows - 1) / p.code_rows;
  p.slab_grid = Grid{n * p.slabs, 1};
  p.partial_grid = Grid{n * p.chunks, 1};
  p.final_grid = wide((n * groups + kGnFinalGroups - 1) / kGnFinalGroups);
  p.apply_grid = Grid{n * p.apply_chunks, 1};
  p.code_grid = Grid{n * p.code_chunks * kgroups, 1};
  p.brief_grid = Grid{n * ((length + kGnBriefRows - 1) / kGnBriefRows), 1};
  return p;
}

// Samples of a run: HIP takes fewer than 2^32 threads a row of a launch, so a
// call's samples go in runs of about equal number, whose slabs (at most ceil(C / 64)
// a sample) and chunks stay near kWideRow workgroups.  A sample may have a group
// per channel, so the join's workgroups are laid out in rows instead.  From 512
// samples on the plan does not depend on their number, so neither does the
// workspace's use.
inline int64_t gn_run_samples(int64_t n, int64_t C) {
  const int64_t most = kWideRow / ((C + 63) / 64), runs = (n + most - 1) / most;
  return (n + runs - 1) / runs;
}

inline size_t gn_align(size_t v) { return (v + 255) / 256 * 256; }
inline size_t gn_coef_bytes(int64_t n, int64_t C) { return gn_align((size_t)(n * C) * 3 * sizeof(float)); }

}  // namespace hdq
