"""The losses' tiling and passes (csrc/row_loss_plan.h), compiled for the host: which calls go without a
workspace, and that none of those has a use for one."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <stdio.h>
#include <initializer_list>
#include "row_loss_plan.h"
using namespace dg;

static int bad = 0;
static void check(bool ok, const char *what, long V, int size, int K, int sms) {
    if (!ok && bad++ < 20) printf("%s: V = %ld, %d bytes an entry, K = %d, %d SMs\n", what, V, size, K, sms);
}

static void plan(long V, int size, int K) {
    const Tiling t = tile_row(V, size, K);
    const long vecs = V * size / 16;
    check((long)t.tile_vecs * t.tiles >= vecs && (long)t.tile_vecs * (t.tiles - 1) <= vecs, "tiles", V, size, K, 0);
    check((t.tiles == 1) == (tile_row(V, size, 0).tiles == 1), "one tile whatever K", V, size, K, 0);
    const int few = tile_row(V, size, kFewEntries).tiles, many = tile_row(V, size, kMaxTopK).tiles;
    check(t.tiles <= (few > many ? few : many), "more sums than the workspace holds", V, size, K, 0);
    const int stages = ring_stages(t, K);
    check(stages >= 2 && stages * stage_bytes(t, K) <= kRingBytes, "stages", V, size, K, 0);
    for (int sms : {1, 2, 76, 152})
        for (long R : {1L, 2L, 1000L})
            if (reads_twice(t, K, R, sms))
                for (RowLossHead head : {kHeadToken, kHeadDistill})
                    check(takes_workspace(V, size, head, kPassStep), "two passes without a workspace", V, size, K, sms);
    check(!reads_twice(t, K, 1000, 152) || vecs * 16 > (12l << 20), "two passes over a row the chip holds", V, size, K, 152);
}

int main() {
    for (int size : {2, 4}) {
        for (long V = 1; V <= 40000; ++V)
            for (int K = 0; K <= kMaxTopK && K <= V; ++K) plan(V, size, K);
        for (long V = 40001; V < 40000000; V += V / 50)
            for (int K = 0; K <= kMaxTopK; K += 31) plan(V, size, K);
    }
    check(takes_workspace(100, 4, kHeadDistill, kPassBackward), "distillation backward", 100, 4, 5, 0);
    return bad ? 1 : 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    csrc = os.path.join(ROOT, "denoising_sampler_step_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-I", csrc, str(d / "plan.cpp"), "-o",
                    str(d / "plan")], check=True)
    return str(d / "plan")


def test_no_call_without_a_workspace_takes_two_passes(program):
    """Every row of up to 40,000 entries with every list of a teacher's entries, and longer ones; a step whose
    rows are read twice writes to the workspace between its passes."""
    r = subprocess.run([program], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
