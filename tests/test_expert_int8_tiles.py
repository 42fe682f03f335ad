"""The tiles that each case of int8_tile_cases.py takes, by the library's own rule
(expert_plan.h, compiled for the host with g++; no GPU needed), and that its
live tiles are more than the kernel has workgroups."""

import os
import shutil
import subprocess

import pytest

from tests.int8_tile_cases import CASES, CHANGING, TILES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kinds(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = tmp_path_factory.mktemp("kind") / "expert_int8_kind"
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "combine_get_dispatch_layout_amd", "csrc"),
                    os.path.join(ROOT, "tests", "expert_int8_kind.cpp"), "-o", str(exe)], check=True)

    def ask(products):
        """The kind of each (experts, cap, rows, outs)."""
        args = []
        for E, cap, rows, outs in products:
            args += ["counts" if cap else "offsets", str(E), str(cap or rows), str(outs)]
        out = subprocess.run([str(exe), *args], capture_output=True, text=True, check=True, timeout=60)
        return out.stdout.split()

    return ask


def test_cases_take_their_kernel(kinds):
    got = kinds([(c.E, c.cap, c.rows, c.outs) for c in CASES])
    assert got == [c.kind for c in CASES]
    assert {c.kind for c in CASES} == set(TILES)


def test_changing_rows_take_their_kernel(kinds):
    got = kinds([(len(counts[0]), cap, M, outs) for _, cap, outs, M, counts in CHANGING])
    assert got == [c[0] for c in CHANGING]
    assert set(got) == set(TILES)


@pytest.mark.parametrize("case", CASES, ids=repr)
def test_workgroups_take_several_tiles(case):
    assert case.live_tiles() > TILES[case.kind][2]
    assert all(0 <= n <= (case.cap or case.rows) for n in case.counts)


@pytest.mark.parametrize("case", CHANGING, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}")
def test_workgroups_take_several_tiles_of_changing_rows(case):
    kind, cap, outs, M, counts = case
    rows, cols, most = TILES[kind]
    live = [sum(-(-c // rows) for c in v) * -(-outs // cols) for v in counts]
    assert live[0] > most and 0 in live
    for v in counts:
        assert sum(v) <= M and all(0 <= c <= (cap or M) for c in v)
