"""The calls of tests/kv_division.py take the number of teams that they are there for (csrc/kv_rules.h compiled as plain C++); CPU
only."""
import os
import subprocess

from tests.kv_division import CALLS, width
from tests.test_kv_rules import CSRC

SOURCE = r"""
#include <stdio.h>
#include "kv_rules.h"
using namespace ftmoe::kv;

// D, bytes of an element, items of a request, steps of the widest request, requests, their lengths -> teams, launched
int main() {
    int D, e, per, most, n;
    while (scanf("%d %d %d %d %d", &D, &e, &per, &most, &n) == 5) {
        uint32_t total = 0, busy = 0;
        for (int i = 0; i < n; ++i) {
            int len;
            if (scanf("%d", &len) != 1) return 1;
            total += item_length((len + kStep - 1) / kStep);
            busy += len > 0;
        }
        const int grid = grid_of((int64_t)n * per, (int64_t)n * per * most, D, e);
        const Division d = divide(busy * per, total * per, team_steps(D), grid, many_items(D * e));
        printf("%d %d\n", d.teams, grid);
    }
    return 0;
}
"""


def test_teams_of_the_calls(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(SOURCE)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)])
    lines, want = [], []
    for fmt, D, heads, g, P, lens, teams in CALLS.values():
        steps = -(-width(P, lens) * P // 32)
        lines.append(" ".join(map(str, [D, 2 if fmt == "bf16" else 1, heads * -(-g // 16), steps, len(lens)] + lens)))
        want.append(teams)
    out = subprocess.run([str(exe)], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True).stdout.split()
    got, grid = [int(v) for v in out[::2]], [int(v) for v in out[1::2]]
    assert dict(zip(CALLS, got)) == dict(zip(CALLS, want))
    # calls with room for more teams than they take are among them
    assert any(g > t for g, t in zip(grid, got)) and all(g >= t for g, t in zip(grid, got))


def test_the_widest_calls_pass_what_the_first_tests_reach():
    """Team indexes of 256 and more, that is parts and counters behind the first half's."""
    assert sum(teams == 512 for *_, teams in CALLS.values()) >= 5
    assert {(f, D) for f, D, *_, teams in CALLS.values() if teams == 512} == {("bf16", 64), ("e4m3", 64), ("e4m3", 128)}
