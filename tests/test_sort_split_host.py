"""How ns_moe_sort deals slots to workgroups, over its whole range: csrc/sort_split.h compiled with g++ and run
(tests/c/sort_split.cpp). No GPU is needed."""

import os
import random
import shutil
import subprocess

import pytest

import newton_schulz_quintic_amd as nsq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")
def test_every_slot_has_a_workgroup(tmp_path):
    exe = str(tmp_path / "sort_split")
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror",
                        "-I", os.path.join(ROOT, "newton_schulz_quintic_amd", "csrc"),
                        os.path.join(ROOT, "tests", "c", "sort_split.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    top = 2 ** 31 - 1
    rng = random.Random(0)
    slots = [0, 1, 511, 512, 513, 2047, 2048, 2049, 131072, 131073, 2 ** 28, 2 ** 30, top - 512, top - 511, top - 510,
             top - 8, top - 1, top] + [int(2 ** rng.uniform(0, 31)) for _ in range(500)]
    r = subprocess.run([exe] + [str(s) for s in slots], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    got = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    assert len(got) == len(slots)
    for n, (per, blocks) in zip(slots, got):
        assert per > 0 and per % 512 == 0 and 1 <= blocks <= 256, n
        assert per * blocks >= n and (blocks == 1 or per * (blocks - 1) < n), n   # all dealt, no workgroup without slots
        assert (blocks == 1) == (n <= 2048), n                                     # a single launch for few


@pytest.mark.parametrize("top_k", [1, 2, 3, 5, 7, 8, 1000, 2 ** 30])
def test_every_count_of_slots_below_two_to_the_31_is_taken(top_k):
    most = (2 ** 31 - 1) // top_k
    assert nsq.ns_moe_sort_workspace_bytes(most, top_k, 8) > 0
    with pytest.raises(nsq.NSError) as e:
        nsq.ns_moe_sort_workspace_bytes(most + 1, top_k, 8)
    assert e.value.name == "NS_ERR_OVERFLOW"


def test_choices_past_30_bits_are_refused():
    assert nsq.ns_moe_sort_workspace_bytes(0, 2 ** 31 - 1, 8) > 0
    with pytest.raises(nsq.NSError) as e:
        nsq.ns_moe_sort_workspace_bytes(1, 2 ** 30 + 1, 8)
    assert e.value.name == "NS_ERR_OVERFLOW"
