"""Every launch of a group norm within the documented sizes fits what HIP takes:
the plan's host code, compiled alone and looked over on the CPU."""
import math
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MAIN = """
#include <cstdio>
#include "group_norm_plan.h"
using namespace hdq;
static void show(const char* name, const Grid& g, long long threads, long long need) {
  std::printf(" %s:%lld:%lld:%lld:%lld", name, (long long)g.x, (long long)g.y, threads, need);
}
int main() {
  long long n, length, C, groups;
  int f32, fp8;
  while (std::scanf("%lld %lld %lld %lld %d %d", &n, &length, &C, &groups, &f32, &fp8) == 6) {
    const long long run = gn_run_samples(n, C);
    std::printf("run:%lld:%lld:0:0", run, (n + run - 1) / run);
    for (long long r = run; r > 0; r = r == run && n % run ? n % run : 0) {  // a whole run, and the last
      const GnPlan p = gn_plan(r, length, C, groups, f32 != 0);
      if (fp8 ? p.brief : p.keep) {
        if (fp8) show("brief", p.brief_grid, kGnThreads, r * ((length + kGnBriefRows - 1) / kGnBriefRows));
        else show("keep", p.slab_grid, p.threads, r * p.slabs);
        continue;
      }
      if (p.slab) show("slab", p.slab_grid, p.threads, r * p.slabs);
      else show("partial", p.partial_grid, kGnThreads, r * p.chunks);
      if (!p.slab && !p.join) show("final", p.final_grid, kGnFinalThreads, (r * groups + kGnFinalGroups - 1) / kGnFinalGroups);
      if (fp8) show("code", p.code_grid, kGnCodeThreads, r * p.code_chunks * (((C + 127) / 128 + 3) / 4));
      else show("apply", p.apply_grid, kGnThreads, r * p.apply_chunks);
    }
    std::printf("\\n");
  }
}
"""


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not found")
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "plan.cpp", d / "plan"
    src.write_text(MAIN)
    subprocess.check_call([cxx, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "bit_quantized_video_amd", "csrc"), str(src),
                           "-o", str(exe)])

    def run(sizes):
        text = "".join(" ".join(str(int(v)) for v in s) + "\n" for s in sizes)
        out = subprocess.check_output([str(exe)], input=text, text=True).splitlines()
        assert len(out) == len(sizes)
        return [[(f[0], *map(int, f[1:])) for f in (w.split(":") for w in line.split())] for line in out]
    return run


def check(sizes, rows):
    kinds = set()
    for s, (head, *row) in zip(sizes, rows):
        run, runs = head[1:3]
        assert 0 < run <= s[0] and run * (runs - 1) < s[0] <= run * runs, s
        assert row, s
        for name, x, y, threads, need in row:
            assert 0 < x and x * threads < 1 << 32 and 0 < y < 1 << 16, (s, name, x, y, threads)
            assert need <= x * y < 1 << 31 and (y == 1 or x == 1 << 22), (s, name, x, y, need)
            assert (y == 1 and x == need) or name == "final", (s, name)   # only the join numbers its workgroups over rows
            kinds.add(name)
    return kinds


def test_a_group_per_channel_in_many_samples(launches):
    """The join's waves, one per sample and group, pass 2^26 (2^32 threads)."""
    sizes = [(427445, 513, 157, 157, 0, 0), (1 << 20, 600, 157, 157, 0, 0), (500000, 4000, 513, 513, 1, 0),
             (100000, 20000, 8191, 8191, 1, 0), (262144, 8191, 8192, 8192, 1, 0), (200000, 3000, 2048, 2048, 0, 1)]
    rows = launches(sizes)
    assert check(sizes, rows) >= {"partial", "final"}
    assert any(k[0] == "final" and k[2] > 1 for row in rows for k in row[1:])


def test_launches_of_documented_sizes(launches):
    rng = random.Random(3)
    top = 0x7ffffc00
    log = lambda hi: int(math.exp(rng.uniform(0, math.log(hi + 1))))
    sizes = []
    while len(sizes) < 20000:
        C = min(8192, log(8192))
        fp8 = rng.random() < 0.4
        if fp8:
            C = max(8, C // 8 * 8)
        groups = rng.choice([g for g in range(1, C + 1) if C % g == 0])
        n = min(top, log(top))
        length = min(top // n, log(top // n)) if rng.random() < 0.7 else top // n
        sizes.append((n, max(1, length), C, groups, rng.random() < 0.5, fp8))
    assert check(sizes, launches(sizes)) == {"keep", "slab", "partial", "final", "apply", "code", "brief"}
