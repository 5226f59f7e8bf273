"""Which kernel a product takes: the rules of csrc/ffn_plan.h, compiled for the host."""
import os
import shutil
import subprocess
import tempfile

from conftest import ROOT

KINDS = ("256x256", "256x128", "128x128", "32x128", "few rows")
available = shutil.which("g++") is not None

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include "ffn_plan.h"
int main() {
  char op[16];
  long long M, N, K, groups;
  int grouped;
  while (scanf("%15s %lld %lld %lld %lld %d", op, &M, &N, &K, &groups, &grouped) == 6) {
    const bool g = grouped != 0;
    glu::ProductPlan p{};
    if (!strcmp(op, "linear")) p = glu::plan_product(glu::FWD, M, N, K, groups, g);
    if (!strcmp(op, "dx")) p = glu::plan_product(glu::DGRAD, M, K, N, groups, g);
    if (!strcmp(op, "dw")) p = glu::plan_product(glu::WGRAD, N, K, M, groups, g);
    if (!strcmp(op, "gated")) p = glu::plan_gated(false, M, N, K, groups, g);
    if (!strcmp(op, "gated8")) p = glu::plan_gated(true, M, N, K, groups, g);
    if (!strcmp(op, "fp8")) p = glu::plan_fp8(M, N, K, groups, g);
    if (!strcmp(op, "both")) p.kind = glu::plan_gradients(M, N, K), p.splits = 1;
    printf("%d %lld\n", p.kind, (long long)p.splits);
  }
}
"""


def plans(queries):
    """[(kernel, parts of the sum)] of [(op, M, N, K, groups)], groups 0 without offsets.  op is "linear", "dx", "dw" (of
    x [M, K], W [N, K]), "gated", "gated8" (with codes), "fp8" or "both" (one launch for both gradients; no kernel: None)."""
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "plans.cpp"), os.path.join(d, "plans")
        with open(src, "w") as f:
            f.write(PROGRAM)
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.join(ROOT, "glu_activation_microscaling_amd", "csrc"), src, "-o", exe], check=True)
        text = "\n".join(f"{op} {M} {N} {K} {max(g, 1)} {int(g > 0)}" for op, M, N, K, g in queries)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
    pairs = [(int(a), int(b)) for a, b in zip(out[::2], out[1::2])]
    assert len(pairs) == len(queries)
    return [(KINDS[k] if k >= 0 else None, s) for k, s in pairs]
