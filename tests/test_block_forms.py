"""CPU test that the sizes of block_cases take the forms that they are there for, by the library's own rules
(csrc/linear_plan.h and csrc/seq_plan.h, compiled here)."""

import os
import shutil
import subprocess

import pytest

from block_cases import BACKWARD, CONV, CONV_NARROW, E, FORWARD, SCAN, scan_lens

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "recurrent_sequence_models_amd", "csrc")

ASK = r"""
#include <cstdio>
#include "linear_plan.h"
#include "seq_plan.h"
using namespace falcon;
static void show(const Plan &p) {
  const char *name[] = {"few", "small", "deep", "medium", "large"};
  printf(p.splits > 1 ? "%s/%d " : "%s ", name[(int)p.form], p.splits);
}
int main() {
  char what;
  long a, b, c;
  int e, n, T, D, N, mark = 0;
  while (scanf(" %c", &what) == 1) {
    if (what == 'f' && scanf("%ld %ld %ld %d", &a, &b, &c, &e) == 4) {          // tokens, in, out
      show(plan_of(c, a, b, e));
      printf("%d", tokens_apart(c, a, b, e));
    } else if (what == 'b' && scanf("%ld %ld %ld %d", &a, &b, &c, &e) == 4) {
      show(tiles_of(b, a, c, e));
      show(tiles_of(b, c, a, e));
    } else if (what == 's' && scanf("%d %d %d %d %d", &n, &T, &D, &N, &e) == 5) {
      const SeqMap q{e ? &mark : nullptr, n, T};
      const int seg = ssm_segment_fwd(q, D, N);
      printf("%s %d", ssm_few_fwd(q, seg, D) ? "few" : "many", ssm_segmented(q, seg) ? seg : 0);
    } else if (what == 'c' && scanf("%d %d %d %d", &n, &T, &D, &e) == 4) {
      const SeqMap q{&mark, n, T};
      const ConvPlan f = conv_plan(q, D, e == 2, false), b = conv_plan(q, D, e == 2, true);
      printf("%d %d %d %d", f.lanes, f.run, b.lanes, b.run);
    } else return 1;
    printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    d = tmp_path_factory.mktemp("ask")
    (d / "ask.cpp").write_text(ASK)
    gxx = shutil.which("g++") or pytest.skip("no host compiler")
    r = subprocess.run([gxx, "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", CSRC, "-o", str(d / "ask"),
                        str(d / "ask.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(*words):
        r = subprocess.run([str(d / "ask")], input=" ".join(map(str, words)), capture_output=True, text=True)
        assert r.returncode == 0, words
        return r.stdout.split()
    return ask


def test_products(ask):
    seen = {dtype: set() for dtype in E}
    for size, forms in FORWARD:
        for dtype, form in forms.items():
            assert ask("f", *size, E[dtype]) == [form, "0"], (size, dtype)
            seen[dtype].add(form.split("/")[0])
    for dtype, forms in seen.items():
        assert forms == {"few", "small", "deep", "medium"} | ({"large"} if dtype != "fp32" else set()), dtype
    back = {dtype: (set(), set()) for dtype in ("bf16", "fp32")}
    for size, forms in BACKWARD:
        for dtype, want in forms.items():
            assert ask("b", *size, E[dtype]) == list(want), (size, dtype)
            for s, form in zip(back[dtype], want):
                s.add(form.split("/")[0])
    assert back["bf16"][0] == {"small", "deep", "medium", "large"} and back["bf16"][1] >= {"small", "deep", "large"}
    assert back["fp32"][0] >= {"small", "deep", "medium"} and back["fp32"][1] >= {"small", "deep", "medium"}


@pytest.mark.parametrize("name", SCAN)
@pytest.mark.parametrize("N", [16, 32, 64])
def test_scans(ask, name, N):
    _, D, packed, cut = SCAN[name]
    lens = scan_lens(name, N)
    form, seg = ask("s", len(lens), sum(lens) if packed else lens[0], D, N, int(packed))
    assert form == "many" and (int(seg) > 0) == cut
    if cut:
        assert max(lens) > int(seg)
    if packed:
        assert 0 in lens


@pytest.mark.parametrize("dtype,taps,act,D,lens", CONV)
def test_convolution_runs(ask, dtype, taps, act, D, lens):
    assert ask("c", len(lens), sum(lens), D, E[dtype]) == ["64", "16", "64", "32"]


@pytest.mark.parametrize("dtype,taps,act,D,lens", CONV_NARROW)
def test_narrow_convolution(ask, dtype, taps, act, D, lens):
    assert ask("c", len(lens), sum(lens), D, E[dtype])[:2] == ["16", "8"]
