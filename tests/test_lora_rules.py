"""The adapters' host rules (csrc/lora_rules.h): the sizes of the tests that are there for one launch form take that
form.  CPU only."""
import os
import subprocess

import pytest

from tests.test_gpu_lora_slots import EXPERTS, PROJECTS, T

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_expert_execution_amd", "csrc")

HARNESS = r"""
#include <stdio.h>
#include <stdlib.h>
#include "lora_rules.h"
using namespace ftmoe::rs;
int main(int argc, char** argv) {     // project n K T slots | expert d f T slots
    const bool project = argv[1][0] == 'p';
    const int a = atoi(argv[2]), b = atoi(argv[3]), T = atoi(argv[4]), slots = atoi(argv[5]);
    const Shrink s = shrink_of(T, project ? b : a, slots, 1, true);
    printf("%d %d %d", project ? project_tiles(a, b, T) : expert_tiles(a, b, T), s.per, s.span);
    return 0;
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("rules")
    src, exe = tmp / "rules.cpp", tmp / "rules"
    src.write_text(HARNESS)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, str(src), "-o", str(exe)])
    return lambda *args: subprocess.check_output([str(exe), *map(str, args)], text=True).split()


def test_two_slot_sizes_take_two_slots(rules):
    """They go through the GEMM tiles, behind a shrink launch of two slots to a workgroup over 32 tokens."""
    for n, K, count, R in PROJECTS:
        assert rules("project", n, K, T, R // 16) == ["1", "2", "32"], (n, K, R)
    for d, f, gate, up, _ in EXPERTS:
        pools = [p for p in (gate, up) if p]
        slots = len(pools) * max(p[1] for p in pools) // 16
        assert rules("expert", d, f, T, slots) == ["1", "2", "32"], (d, f, gate, up)
    assert {R // 16 % 2 for _, _, _, R in PROJECTS} == {0, 1}, "an odd and an even number of slots"
