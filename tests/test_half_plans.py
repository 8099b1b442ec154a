"""CPU test of the 16-bit products' plan: a small host program built on the library's
own rules (csrc/half_plan.hpp) says what each size of _half_plans.py takes on 256
compute units, and that no kernel, result type or store policy is left without one."""
import os
import re
import shutil
import subprocess

import pytest

import fp4_gemm_moe_amd as hq
from fp4_gemm_moe_amd import build
from tests import _half_plans as P

PROGRAM = r"""
#include <cstdio>
#include "half_plan.hpp"
int main() {
  static const char* tiles[] = {"direct", "256x256", "128x256", "128x128", "64x128", "32x64"};
  long long form, rows, groups, n, k, out, transpose;
  hq::DeviceInfo dev{};
  dev.num_cus = 256;
  while (scanf("%lld %lld %lld %lld %lld %lld %lld", &form, &rows, &groups, &n, &k, &out, &transpose) == 7) {
    hq::HalfGemmArgs p{};
    p.form = (int)form;
    p.groups = (int)groups;
    p.slot_rows = rows;
    p.rows = form == hq::kMasked ? rows * groups : rows;
    p.n = n;
    p.k = k;
    p.out_kind = (int)out;
    p.b_t = transpose != 0;
    const int tile = hq::plan_half(p, dev);
    if (tile == hq::kDirect) puts("direct");
    else printf("%s p%d\n", tiles[tile + 1], (int)(out != hq::kOutF32Add && hq::plan_stream(p)));
  }
}
"""

CONTIGUOUS, MASKED, GROUP_K = 1, 2, 3
#: BlockOut's numbers.
KIND = {"bf16": 0, "fp16": 1, "f32": 2, "add": 3}


def _cases():
    """(numbers that the program reads, the plan expected)"""
    for counts, spare, n, k, t, out, transpose, plan in P.CONTIGUOUS:
        yield (CONTIGUOUS, sum(counts) + spare, len(counts), n, k, KIND[out or t], int(transpose)), plan
    for counts, slot, n, k, t, out, transpose, plan in P.MASKED:
        yield (MASKED, slot, len(counts), n, k, KIND[out or t], int(transpose)), plan
    for counts, spare, m, n, t, out, plan in P.GROUP_K:
        yield (GROUP_K, m, len(counts), n, sum(counts) + spare, KIND[out or t], 0), plan


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
    """Each tile of each form, weights' layout and operands' type with every result
    type, and with results that stay in the caches and that leave past them (those
    of 32x64 tiles with weights [k, n] are too few for that)."""
    sizes = ([(CONTIGUOUS, *c[-4:-1]) for c in P.CONTIGUOUS] + [(MASKED, *c[-4:-1]) for c in P.MASKED]
             + [(GROUP_K, *c[-3:-1], False) for c in P.GROUP_K])          # form, operands' type, results', layout
    seen = {(form, tr, t, out, plan) for (form, t, out, tr), plan in zip(sizes, planned)}
    want = set()
    for t, out in P.KINDS:
        for policy in ("p0",) if out == "add" else ("p0", "p1"):
            for form in (CONTIGUOUS, MASKED):
                want |= {(form, tr, t, out, f"{tile} {policy}") for tr in (False, True)
                         for tile in ("256x256", "128x256", "128x128", "64x128", "32x64")
                         if (tile, tr, policy) != ("32x64", True, "p1")}
                want.add((form, False, t, out, "direct"))
            want |= {(GROUP_K, False, t, out, f"{tile} {policy}") for tile in ("256x256", "128x128")}
    assert seen == want


def test_every_kernel_that_is_built_has_a_size(planned):
    """The tiled kernels in the library are those that the plans take."""
    if shutil.which("nm") is None:
        pytest.skip("no symbol reader")
    if not os.path.exists(hq.library_path()):
        build.build(verbose=False)
    names = subprocess.run(["nm", "-C", hq.library_path()], capture_output=True, text=True, check=True).stdout
    built = {(f"{m[1]}x{m[2]}", m[3] == "true", m[4] == "true", m[5] == "true") for m in re.finditer(
        r"__device_stub__half_gemm_tiled<hq::half::Cfg<(\d+), (\d+)[^>]*>, (\w+), (\w+), (\w+)>", names)}
    sizes = ([(False, c[-2], c[-4]) for c in P.CONTIGUOUS + P.MASKED] + [(True, True, c[-3]) for c in P.GROUP_K])
    taken = {(plan.split()[0], at, bt, t == "fp16") for (at, bt, t), plan in zip(sizes, planned) if plan != "direct"}
    assert built == taken
