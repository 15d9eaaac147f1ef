"""Every launch of the head kernels, the cache's reader and the 4-bit layer within
the documented sizes fits what HIP and the kernels take, and covers its work
once: the plans' host code, compiled alone and looked over on the CPU."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MAIN = """
#include <cstdio>
#include "heads_plan.h"
#include "w4_plan.h"
using namespace hdq;
int main() {
  char kind;
  long long a, b, c, d, e, f;
  while (std::scanf(" %c %lld %lld %lld %lld %lld %lld", &kind, &a, &b, &c, &d, &e, &f) == 7) {
    if (kind == 'h') {
      const HeadPlan p = plan_heads(a, b, c, d, (int)e, (int)f, kHeadWaves);
      std::printf("%d %d %d %d %d %d %d %d %lld\\n", p.lane_bits, p.slot_bits, p.step_end[0], p.step_end[1], p.step_end[2], p.steps,
                  p.slices[0], p.slices[1], (long long)p.groups);
    } else {
      const W4Plan p = plan_w4(a, b, c);
      std::printf("%d %d %d %d %d %d %lld %d %d %lld %lld %lld %lld\\n", (int)p.direct, p.step, p.part, p.per, p.wn, p.wk, (long long)p.lds, p.mt, p.split,
                  (long long)p.grid_x, (long long)p.grid_y, (long long)w4_workspace(a, b, c), (long long)w4_slice(a, b));
    }
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not found")
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "plan.cpp", d / "plan"
    src.write_text(MAIN)
    subprocess.check_call([cxx, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "bit_quantized_video_amd", "csrc"), str(src),
                           "-o", str(exe)])

    def run(kind, sizes):
        text = "".join(" ".join([kind, *(str(int(v)) for v in (*s, 0, 0, 0))][:7]) + "\n" for s in sizes)
        out = subprocess.check_output([str(exe)], input=text, text=True).splitlines()
        assert len(out) == len(sizes)
        return [tuple(map(int, line.split())) for line in out]
    return run


def up(a, b):
    return -(-a // b)


def log_size(g, low, high):
    return min(high, max(low, int(low * (high / low) ** g.random())))


def test_heads(plans):
    g, top, heads = random.Random(1), 0x7ffffc00, 1 << 20
    sizes = [(t, h, k, v, d, p) for t in (1, 2, 63, 4050, top) for h, k, v in ((1, 0, 0), (30, 30, 30), (0, 1, 1), (heads - 2, 1, 1),
             (0, heads // 2, heads // 2), (1, heads - 1, 0)) for d in (1, 8, 64, 72, 128, 500, 512) for p in (8, 16) if p == 8 or d % 16 == 0]
    for _ in range(3000):
        h, k = log_size(g, 1, heads // 4), log_size(g, 1, heads // 4)
        h, k, v = g.choice(((h, 0, 0), (h, k, 0), (h, k, k), (0, k, k)))
        d, p = g.choice(((g.randint(1, 512), 8), (16 * g.randint(1, 32), 16)))
        sizes.append((log_size(g, 1, top), h, k, v, d, p))
    for s, (ll, sl, e0, e1, e2, steps, qk, val, groups) in zip(sizes, plans("h", sizes)):
        tokens, h, dim, per_lane = s[0], s[1:4], s[4], s[5]
        assert 0 <= ll and 0 <= sl and ll + sl <= 6 and per_lane << ll >= dim, s
        per_wave = 1 << (6 - ll - sl)
        assert (groups - 1) * per_wave < tokens <= groups * per_wave
        ends = (e0, e1, e2)
        for t in range(3):           # a tensor's steps hold its heads, the last step one at least
            n = ends[t] - (ends[t - 1] if t else 0)
            assert (n - 1) << sl < h[t] <= n << sl, s
        # the queries' and keys' layers of the grid, and the values', end with their last step
        assert (qk - 1) * steps < e1 <= qk * steps and (val - 1) * steps < e2 - e1 <= val * steps
        assert 1 <= qk + val < 1 << 16
        # LDS: angles of a wave's tokens
        assert per_wave * (dim // 2) <= 256 if per_lane == 8 else per_wave * (8 << ll) <= 512 and dim <= 16 << ll, s


def test_reader_layers(plans):
    """The reader's plan is that of one tensor over twice the tokens: two layers for each slice."""
    for t in (1, 77, 0x7ffffc00):
        for heads in (1, 30, 1 << 19):
            (_, _, e0, e1, e2, steps, qk, val, _), = plans("h", [(2 * t, heads, 0, 0, 64, 16)])
            assert e0 == e1 == e2 and val == 0 and 2 * qk < 1 << 16 and (qk - 1) * steps < e0 <= qk * steps


def test_w4(plans):
    g = random.Random(2)
    top_m, top_n, top_k = 1 << 20, 1 << 27, 1 << 22
    sizes = [(m, n, k) for m in (1, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, top_m) for n in (1, 16, 17, 5760, 345600, top_n)
             for k in (32, 128, 512, 1920, 12288, 32640, 32672, top_k)]
    for _ in range(4000):
        sizes.append((log_size(g, 1, g.choice((16, 200, top_m))), log_size(g, 1, top_n), 32 * log_size(g, 1, g.choice((100, top_k // 32)))))
    forms = set()
    for (m, n, k), (direct, step, part, per, wn, wk, lds, mt, split, gx, gy, ws, piece) in zip(sizes, plans("w", sizes)):
        s = (m, n, k)
        tn, tk = up(n, 16), up(k, 128)
        blocks = up(tk, 4)
        assert 0 < gy < 1 << 16 and 0 < split < 1 << 16 and gx * 64 * wn * wk < 1 << 32, s
        assert m * n <= piece < m * n + 4
        if direct:
            forms.add(("direct", mt))
            tiles = 4 // mt                                                # of K, a wave's
            assert m <= 16 * mt and wn == 1 and (wk - 1) * tiles < tk <= wk * tiles and wk <= 16, s
            assert gx == tn and gy == split == 1 and ws == 0 and per == 0 and lds == wk * mt * 1024 <= 65536, s
        elif per:
            forms.add((per > 1, wk > 1, wn > 1))
            assert step * blocks + part == wn * wk and 0 <= part < blocks, s
            assert m <= 16 and gy == split == 1 and ws == 0
            assert 64 * wn * wk <= (1024 if m <= 8 else 512), s          # the kernels' launch bounds
            assert lds <= 65536 and lds >= m * (tk * 256 + 16), s
            rows = 1 if m <= 4 else 2 if m <= 8 else 4                     # results a lane
            assert wk == 1 or (per == 1 and lds >= wn * wk * rows * 256), s
            assert wk <= blocks
            assert (gx - 1) * wn * per < tn <= gx * wn * per, s
        else:
            forms.add((mt, split > 1))
            assert wn * wk == 8 and mt in (1, 2, 4)
            assert (gx - 1) * 8 < tn <= gx * 8 and (gy - 1) * 16 * mt < m <= gy * 16 * mt, s
            each = up(tk, split)
            assert (split - 1) * each < tk <= split * each, s              # no workgroup without tiles
            assert ws == (split * piece * 4 if split > 1 else 0)
            assert split == 1 or each >= 4
        if m <= 16 and m * k <= 24576:                                     # what the binding takes to need no scratch
            assert ws == 0, s
    assert {(1, True), (1, False), (2, True), (2, False), (4, True), (4, False)} <= forms
    assert {("direct", 1), ("direct", 2), ("direct", 4)} <= forms and {(False, True, False), (False, False, True), (True, False, True), (False, True, True)} <= forms
