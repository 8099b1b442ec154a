"""CPU test of the block-128 products' plan: a small host program built on the
library's own rules (csrc/block_plan.hpp) says what each size of _block_plans.py
takes on 256 compute units, and that no variant is left without a size."""
import os
import shutil
import subprocess

import pytest

from fp4_gemm_moe_amd import build
from tests import _block_plans as P

PROGRAM = r"""
#include <cstdio>
#include "block_plan.hpp"
int main() {
  static const char* tiles[] = {"256x256", "256x128", "128x256", "128x128", "64x128"};
  long long form, rows, groups, n, k, out, ws;
  hq::DeviceInfo dev{};
  dev.num_cus = 256;
  while (scanf("%lld %lld %lld %lld %lld %lld %lld", &form, &rows, &groups, &n, &k, &out, &ws) == 7) {
    hq::BlockGemmArgs p{};
    p.form = (int)form;
    p.groups = (int)groups;
    p.n = n;
    p.k = k;
    p.out_kind = (int)out;
    p.slices = 1;
    p.slot_rows = rows;
    p.rows = form == hq::kUniform || form == hq::kMasked ? rows * groups : rows;
    p.nkb = (int)((k + 127) / 128);
    p.nnb = (int)((n + 127) / 128);
    if (hq::direct_path(p)) {
      puts("direct");
      continue;
    }
    const bool fast = hq::fast_path(p);
    auto launch = [&](hq::BlockGemmArgs q, const hq::Plan& pl, long long columns) {
      q.n = columns;
      q.slices = pl.slices;
      if (pl.slices > 1) q.out_kind = hq::kOutF32;
      printf("%s %s s%d p%d", fast ? "fp8" : "fp16", tiles[pl.tile], pl.slices, hq::plan_policy(q));
    };
    hq::Plans pl;
    if (form == hq::kUniform) pl = hq::plan_all(p, dev, fast, (uint64_t)ws);
    else pl.all.tile = hq::plan_grouped(p, fast);
    launch(p, pl.all, pl.head ? pl.head : n);
    if (pl.head) {
      printf(" + ");
      launch(p, pl.rest, n - pl.head);
      printf(" head %lld", (long long)pl.head);
    }
    puts("");
  }
}
"""

KIND = {P.BF16: 0, P.F16: 1, P.F32: 2}
UNIFORM, CONTIGUOUS, MASKED, GROUP_K = range(4)


def _cases():
    """(numbers that the program reads, the plan expected)"""
    for m, n, k, t, ws, plan in P.DENSE:
        yield (UNIFORM, m, 1, n, k, KIND[t], ws), plan
    for b, m, n, k, t, ws, plan in P.BATCH:
        yield (UNIFORM, m, b, n, k, KIND[t], ws), plan
    for counts, spare, n, k, t, plan in P.CONTIGUOUS:
        yield (CONTIGUOUS, sum(counts) + spare, len(counts), n, k, KIND[t], 0), plan
    for counts, slot, n, k, t, plan in P.MASKED:
        yield (MASKED, slot, len(counts), n, k, KIND[t], 0), plan
    for blocks, m, n, t, plan in P.GROUP_K:
        yield (GROUP_K, m, len(blocks), n, 128 * sum(blocks), KIND[t], 0), plan


@pytest.fixture(scope="module")
def planned(tmp_path_factory):
    compiler = shutil.which("g++")
    if compiler is None:
        pytest.skip("no host compiler")
    where = tmp_path_factory.mktemp("plan")
    src, exe = str(where / "plan.cpp"), str(where / "plan")
    with open(src, "w") as f:
        f.write(PROGRAM)
    rocm = os.path.dirname(os.path.dirname(build.HIPCC))
    subprocess.run([compiler, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"), "-I",
                    build.INCLUDE, "-I", build.CSRC, "-o", exe, src], check=True)
    text = "".join(" ".join(map(str, c)) + "\n" for c, _ in _cases())
    return subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()


def test_each_size_takes_its_plan(planned):
    for (case, want), got in zip(_cases(), planned):
        assert got == want, case
    assert len(planned) == len(list(_cases()))


def test_every_variant_has_a_size(planned):
    launches = [p for plan in planned if plan != "direct" for p in plan.split(" + ")]
    seen = {(path, tile, slices != "s1") for path, tile, slices in (p.split()[:3] for p in launches)}
    for split in (False, True):
        assert {("fp8", t, split) for t in ("256x256", "128x256", "128x128", "64x128")} <= seen
        assert {("fp16", t, split) for t in ("256x128", "128x128", "64x128")} <= seen
    rest = {plan.split(" + ")[1].split()[1] for plan in planned if " + " in plan}
    assert rest == {"256x256", "128x256", "128x128", "64x128"}
    policies = {(path, policy) for path, _, _, policy in (p.split()[:4] for p in launches)}
    assert policies == {(path, policy) for path in ("fp8", "fp16") for policy in ("p0", "p1", "p2")}
