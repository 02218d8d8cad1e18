"""How attention's work is divided (csrc/kv_rules.h): the teams' ranges cover every step once, team_of finds the team of
a step, parts of one item have slots of their own, and the join counts each of them.  Compiled as plain C++; CPU only."""
import os
import subprocess

import pytest

from tests.kv_util import place

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_execution_amd", "csrc")

SOURCE = r"""
#include <stdio.h>
#include <stdlib.h>
#include <map>
#include <set>
#include <vector>
#include "kv_rules.h"
using namespace ftmoe::kv;
#define CHECK(c) do { if (!(c)) { printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)

int division(const std::vector<int>& items, int grid) {
    std::vector<long long> first{0};
    for (int n : items) first.push_back(first.back() + n);
    const long long total = first.back();
    const int teams = teams_of(total, grid);
    CHECK(teams >= 1 && teams <= grid && teams <= total && teams <= kMaxTeams);
    CHECK(team_begin(total, teams, 0) == 0 && team_begin(total, teams, teams) == total);
    std::map<int, int> arrived;                       // by counter
    std::map<int, int> expected;
    std::set<int> slots;
    for (int t = 0; t < teams; ++t) {
        const long long b = team_begin(total, teams, t), e = team_begin(total, teams, t + 1);
        CHECK(b < e);
        for (long long s = b; s < e; ++s) CHECK(team_of(total, teams, s) == t);
        int open = 0;                                 // items that go on in the next team
        for (size_t i = 0; i < items.size(); ++i) {
            if (items[i] == 0 || first[i] >= e || first[i + 1] <= b) continue;
            const int tf = team_of(total, teams, first[i]), tl = team_of(total, teams, first[i + 1] - 1);
            if (tf == tl) continue;
            const int slot = 2 * t + (first[i] < b ? 0 : 1);
            CHECK(slots.insert(slot).second);         // no two parts in one place
            CHECK(slot == 2 * t + (t == tf ? 1 : 0)); // where the join looks for it
            if (t == tf) ++open;
            ++arrived[tf];
            expected[tf] = tl - tf + 1;
        }
        CHECK(open <= 1);                             // so a team's counter serves one item
    }
    CHECK(arrived == expected);
    return 0;
}

int main() {
    srand(5);
    const int grids[] = {1, 2, 3, 7, 64, 511, kMaxTeams};
    for (int g : grids)
        for (int r = 0; r < 60; ++r) {
            std::vector<int> items;
            const int n = 1 + rand() % 40, big = r % 3 == 0 ? 3000 : r % 3 == 1 ? 40 : 3;
            for (int i = 0; i < n; ++i) items.push_back(rand() % 4 ? 1 + rand() % big : 0);
            items.push_back(1);
            if (division(items, g)) return 1;
        }
    // totals beyond 32 bits
    for (long long total : {1ll << 31, (1ll << 38) + 12345, (1ll << 41) - 1})
        for (int t = 0; t < kMaxTeams; ++t) {
            const long long b = team_begin(total, kMaxTeams, t), e = team_begin(total, kMaxTeams, t + 1);
            CHECK(b < e && team_of(total, kMaxTeams, b) == t && team_of(total, kMaxTeams, e - 1) == t);
        }
    for (int g : {1, 8, 9, 16, 17, 32, 33, 128}) {
        int n = 0;
        for (int i = 0; i < head_blocks(g); ++i) n += g - i * kCols < kCols ? g - i * kCols : kCols;
        CHECK(n == g && item_heads(g) <= kCols);
    }
    CHECK(grid_of(0) == 1 && grid_of(1ll << 40) == kMaxTeams);
    printf("ok\n");
    return 0;
}
"""


def test_division_of_attention(tmp_path):
    src, exe = tmp_path / "r.cpp", tmp_path / "r"
    src.write_text(SOURCE)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC,
                           str(src), "-o", str(exe)])
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout == "ok\n"


@pytest.mark.parametrize("fmt,D", [(f, d) for f in ("bf16", "e4m3") for d in (64, 128, 256)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_layout_is_a_permutation(fmt, D, which):
    size = {"bf16": 2, "e4m3": 1}[fmt]
    seen = sorted(place(fmt, D, which, t, e) for t in range(16) for e in range(D))
    assert seen == list(range(0, 16 * D * size, size))
