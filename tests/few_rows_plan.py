"""The plans of the products of few tokens (csrc/few_rows_plan.h), evaluated on the host: which kernel form a size runs on."""
import functools
import os
import shutil
import subprocess
import tempfile

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_transformer_mlp_gb300", "csrc")
FIELDS = ("takes", "nt", "token_tiles", "col_tiles", "splits", "ranks", "shard", "unit", "num_kb", "stages", "stage_bytes")

SOURCE = r"""
#include <cstdio>
#include "few_rows_plan.h"
using namespace tpmlp::few_rows;
int main() {
  long long n, cols, k, m, t;  // FC1 of the gated block: m > 0 and cols = m; a plain product: m = 0
  while (std::scanf("%lld %lld %lld %lld %lld", &n, &cols, &k, &m, &t) == 5) {
    const Plan p = make_plan(n, cols, k, m, static_cast<int>(t), m > 0);
    const bool takes = m > 0 ? gated_fc1_pays(n, k, m, static_cast<int>(t)) : gemm_pays(n, cols, k);
    std::printf("%d %d %d %d %d %d %d %d %d %d %d\n", takes, p.nt, p.token_tiles, p.col_tiles, p.splits, p.ranks, p.shard, p.unit,
                p.num_kb, p.stages, plan_stage_bytes(p));
  }
}
"""


@functools.lru_cache(maxsize=None)
def _program():
    cxx = shutil.which("g++") or shutil.which("c++")
    assert cxx, "no C++ compiler"
    folder = tempfile.mkdtemp()
    with open(os.path.join(folder, "plan.cpp"), "w") as f:
        f.write(SOURCE)
    exe = os.path.join(folder, "plan")
    subprocess.run([cxx, "-std=c++17", "-O2", "-I", CSRC, f.name, "-o", exe], check=True, capture_output=True, text=True)
    return exe


def _run(lines):
    text = "".join(" ".join(map(str, line)) + "\n" for line in lines)
    out = subprocess.run([_program()], input=text, check=True, capture_output=True, text=True).stdout.split("\n")[:-1]
    assert len(out) == len(lines)
    return [dict(zip(FIELDS, map(int, line.split()))) for line in out]


def fc1(shapes):
    """Plans of the gated block's FC1 for [(n, d, m, t)]; "takes": whether it runs on them."""
    return _run([(n, m, d, m, t) for n, d, m, t in shapes])


def plain(shapes):
    """Plans of plain products [n, k] x [k, cols] for [(n, cols, k)]."""
    return _run([(n, cols, k, 0, 1) for n, cols, k in shapes])
