"""Which tokens a run of the convolution takes, and which rows of the states before the sequences its index rule
can name: csrc/conv_runs.h compiled for the host and walked as the kernels walk it (no GPU needed)."""
import os
import subprocess

import pytest

import linear_spatial_propagation_gspn_b200 as g

WALK = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "conv_runs.h"
using namespace gspn::seq;

// All runs of one row: every token of a sequence once and no other, each with its own sequence.
static int walk(const Tokens& p, int run, bool sorted) {
    std::vector<int> seen(p.L, 0);
    for (int at = 0; at < p.L; at += run) {
        const Run r = run_at(p, at, run);
        if (r.first >= r.end) continue;
        if (r.first < 0 || r.end > p.L || (p.cu && (r.first < border(p, 0) || r.end > border(p, p.S)))) return 1;
        Seq s = find(p, 0, r.first);
        for (int t = r.first; t < r.end; ++t) {
            if (p.cu && t >= s.end) enter(p, s, t);
            if (s.q < 0 || s.q >= p.S) return 2;              // no such row of the states
            if (s.start < 0 || s.start > t || s.end <= t || s.end > p.L) return 3;
            if (p.cu && sorted && (s.start != border(p, s.q) || s.end != border(p, s.q + 1))) return 4;
            ++seen[t];
        }
    }
    for (int t = 0; t < p.L; ++t) {
        const bool in = !p.cu || (t >= border(p, 0) && t < border(p, p.S));
        if (seen[t] != (in ? 1 : 0)) return 5;
    }
    return 0;
}

int main() {
    std::mt19937 g(1);
    auto upto = [&](int n) { return (int)(g() % (unsigned)(n + 1)); };
    for (int trial = 0; trial < 40000; ++trial) {
        const int kind = trial % 4, S = 1 + upto(6), L = upto(60), run = 4 << upto(3);
        std::vector<int> cu(S + 1);
        for (int& v : cu) v = kind == 3 ? upto(4 * L + 8) - 2 * L - 4 : upto(L);   // 3: any values, in any order
        if (kind != 3) {
            for (int i = 1; i <= S; ++i)
                for (int j = i; j > 0 && cu[j] < cu[j - 1]; --j) std::swap(cu[j], cu[j - 1]);
            if (kind == 1) cu[0] = 0;
            if (kind == 2) cu[S] = L;
        }
        const int rc = walk(Tokens{kind == 0 && trial % 8 == 0 ? nullptr : cu.data(), S, L}, run, kind != 3);
        if (rc) {
            std::printf("rule %d broken: L %d, run %d, borders", rc, L, run);
            for (int v : cu) std::printf(" %d", v);
            std::printf("\n");
            return rc;
        }
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def walker(tmp_path_factory):
    d = tmp_path_factory.mktemp("runs")
    (d / "walk.cpp").write_text(WALK)
    subprocess.check_call([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-I", g._build_mod.CSRC, str(d / "walk.cpp"), "-o", str(d / "walk")])
    return str(d / "walk")


def test_runs_name_states_of_the_sequences_only(walker):
    """Tokens before the first border and from the last one on are in no run, so none of them can name a sequence
    behind the last one, whose states are not there."""
    r = subprocess.run([walker], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
