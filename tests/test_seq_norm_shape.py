"""The norm kernels' shared memory: the size rule over every width and number of column sums (on the host), and
the calls at its border, each as the first one of a process."""
import os
import subprocess
import sys

import pytest

import linear_spatial_propagation_gspn_b200 as g

WALK = r"""
#include <cstdio>
#include "norm_shape.h"
using namespace gspn::seq;
int main() {
    for (int C = 1; C <= 16384; ++C)
        for (int slots = 0; slots <= 5; ++slots) {
            const size_t n = smem_for(shape_for(C), slots);
            // what a block has without asking: 48 KB, its own arrays included
            if (n + kStaticSmem > 49152 && !over_48k(n)) { std::printf("%d columns, %d sums: %zu bytes\n", C, slots, n); return 1; }
        }
    return 0;
}
"""


def test_every_width_asks_for_what_it_needs(tmp_path):
    (tmp_path / "walk.cpp").write_text(WALK)
    subprocess.check_call([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-I", g._build_mod.CSRC, str(tmp_path / "walk.cpp"),
                           "-o", str(tmp_path / "walk")])
    r = subprocess.run([str(tmp_path / "walk")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


# The calls whose column sums and parameters come to 48 KB by themselves. What a kernel was allowed by an earlier
# call stays allowed in a process, so each of these starts one.
FIRST = r"""
import sys
import torch
import _seq_ref as R
import linear_spatial_propagation_gspn_b200 as g
from test_seq_norm import NAMES, make, reach

C, parts, center = int(sys.argv[1]), sys.argv[2].split(","), sys.argv[3] == "1"
for types in (("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")):
    t = make(3, C, *types, seed=1)
    kw = {k: t[k] for k in parts}
    do = t["do"] if "w_pre" in kw else None
    got = g.norm_backward(t["y"], t["r"], t["dr"], do, center=center, **kw)
    ref = R.norm(t["y"], None, *(kw.get(k) for k in ("gate", "w_post", "b_post", "scale", "w_pre", "b_pre")), 1e-5, center,
                 t["r"], t["dr"], do)
    for name, a in zip(NAMES, got):                # the bounds of test_seq_norm.test_backward
        if a is None:
            continue
        r = ref[name]
        mag = r.abs() + r.abs().max(-1, keepdim=True).values if r.dim() == 2 else ref[name + "_m"] + ref[name + "_m"].max()
        R.check(a, r, mag, 8 * 96.0 * reach(t, kw, center) + (0 if r.dim() == 2 else 3), f"{types} {name}")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("C,parts,center", [
    (2048, "w_pre", 0), (1800, "w_pre", 0), (1789, "w_post", 0), (1536, "gate,w_post,scale,w_pre", 0), (1281, "scale,w_pre,b_pre", 1),
    (6144, "w_post,w_pre", 0), (12288, "w_pre", 0), (4093, "w_post,scale,w_pre", 0)])
def test_first_call_of_a_process(C, parts, center):
    here = os.path.dirname(os.path.abspath(__file__))
    env = {**os.environ, "PYTHONPATH": os.pathsep.join([here, os.path.dirname(here)])}
    r = subprocess.run([sys.executable, "-c", FIRST, str(C), parts, str(center)], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
