"""How attention's work is divided (csrc/kv_rules.h): every step of every item belongs to one team, parts of one item have slots of their own, and the join counts each of them.  Compiled as plain C++; CPU only."""
import os
import subprocess

import pytest

from tests.kv_util import place

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_execution_amd", "csrc")

SOURCE = r"""
#include <stdio.h>
#include <stdlib.h>
#include <algorithm>
#include <map>
#include <set>
#include <vector>
#include "kv_rules.h"
using namespace ftmoe::kv;
#define CHECK(c) do { if (!(c)) { printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)

int division(const std::vector<int>& items, int steps, int grid, uint32_t many) {
    std::vector<uint32_t> first{0};
    long long busy = 0;
    for (int n : items) {
        first.push_back(first.back() + item_length(n));
        busy += n > 0;
    }
    const uint32_t total = first.back();
    const Division d = divide(busy, total, steps, grid, many);
    CHECK(d.teams >= 1 && d.teams <= grid && (uint32_t)d.teams <= total && d.teams <= kMaxTeams);
    CHECK(cut(d, 0) == 0 && cut(d, d.teams) == total && d.slack >= 0 && 2 * d.slack < (int)(total / d.teams + 1));
    std::vector<int> load(d.teams, 0), length(d.teams, 0);
    std::map<int, int> expected;                      // arrivals by counter
    std::set<int> slots;
    for (size_t i = 0; i < items.size(); ++i) {
        const int n = items[i];
        if (n == 0) continue;
        const Teams who = teams_of(d, first[i], n);
        CHECK(0 <= who.first && who.first <= who.last && who.last < d.teams);
        int next = 0;
        for (int t = who.first; t <= who.last; ++t) {
            const Segment s = segment(d, who, first[i], n, t);
            CHECK(s.from == next && s.to > s.from);   // every step once, in order
            next = s.to;
            load[t] += s.to - s.from;
            length[t] += s.to - s.from + (t == who.first ? kItemCost : 0);
            if (who.first == who.last) continue;
            CHECK(part_slot(who, t) < 2 * kMaxTeams && slots.insert(part_slot(who, t)).second);
        }
        CHECK(next == n);
        // the join: every team arrives once at its run's counter or is its run; every run at the item's
        const int run = join_run(who), parts = who.last - who.first + 1, runs = (parts - 1) / run + 1;
        if (parts == 1) continue;
        CHECK(run <= 2 * kJoin && (runs == 1 || run == kJoin) && runs <= kMaxTeams / kJoin);
        int joined = 0;
        for (int r0 = who.first; r0 <= who.last; r0 += run) {
            const int n = std::min(run, who.last - r0 + 1);
            joined += n;
            if (runs > 1 && n > 1) CHECK(expected.emplace(r0, n).second);     // (a counter serves one run)
        }
        CHECK(joined == parts);
        CHECK(expected.emplace(kMaxTeams + who.first, runs > 1 ? runs : parts).second);
    }
    for (int t = 0; t < d.teams; ++t) CHECK(length[t] <= (int)(total / d.teams) + 1 + 2 * d.slack + kItemCost);
    // how a team finds its items: from the one that its cut falls into, on while they are its own
    for (int t = 0; t < d.teams; ++t) {
        size_t i = 0;
        while (!(first[i] <= cut(d, t) && cut(d, t) < first[i + 1])) ++i;
        for (int mine = 0;; ++i) {
            while (i < items.size() && items[i] == 0) ++i;
            if (i == items.size()) { CHECK(mine == load[t]); break; }
            const Teams who = teams_of(d, first[i], items[i]);
            if (t > who.last) { CHECK(mine == 0); continue; }
            if (t < who.first) { CHECK(mine == load[t]); break; }
            const Segment s = segment(d, who, first[i], items[i], t);
            mine += s.to - s.from;
        }
    }
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
            if (division(items, r % 6 < 2 ? 3 : r % 2 ? 6 : 8, g, r % 4 ? 16 : UINT32_MAX)) return 1;
        }
    // equal short items are not cut
    for (int n = 1; n <= 40; ++n)
        for (int items : {1, 3, 64, 100, 500}) {
            const Division d = divide(items, items * item_length(n), 4, kMaxTeams, 192);
            for (int i = 0; i < items && n <= 4; ++i) {
                const Teams who = teams_of(d, i * item_length(n), n);
                CHECK(who.first == who.last);
            }
        }
    // the largest calls
    for (long long total : {(1ll << 24) + 1, (1ll << 30) + 12345, (1ll << 30) + (4096ll * 1024 * kItemCost)}) {
        const Division d = divide(1 << 20, (uint32_t)total, 8, kMaxTeams, 16);
        CHECK(cut(d, 0) == 0 && cut(d, d.teams) == total);
        for (int t = 0; t < d.teams; ++t) {
            const uint32_t b = cut(d, t), e = cut(d, t + 1);
            CHECK(b < e && team_at(d, b) == t && team_at(d, e - 1) == t);
        }
    }
    for (int g : {1, 8, 9, 16, 17, 32, 33, 128}) {
        int n = 0;
        for (int i = 0; i < head_blocks(g); ++i) n += g - i * kCols < kCols ? g - i * kCols : kCols;
        CHECK(n == g && item_heads(g) <= kCols);
    }
    for (int D : {64, 128, 256})
        for (int e : {1, 2})
            CHECK(grid_of(1, 1, D, e) == 1 && grid_of(4096 * 1024, kMaxSteps, D, e) == (D * e < 256 ? 512 : 256) && most_teams(D) <= kMaxTeams);
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
