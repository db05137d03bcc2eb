"""The ring of key tiles in the 4-bit cache's attention, without a GPU: a model of its barriers, in
which copies land in any order, and the rule that picks the number of stages (the header the
kernels use, compiled for the host)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "accelerator_decode_gb300", "csrc")


def early_waits(stages, sets, tiles):
    """Tiles whose wait can pass before their copy has landed, over every order of events.

    Set s takes tiles s, s + sets, ..; tile t is fill t // stages of stage t % stages, and is filled
    in order, once the tile before in its stage has been left.  full[stage] completes a phase per
    landed copy; a wait for parity p passes when the phase that is not complete yet has another."""
    early, seen = set(), set()
    todo = [(0, frozenset(), (0,) * stages, tuple(range(sets)))]    # fills begun, copies under way, phases, next tiles
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        begun, flying, phases, at = state
        if begun < tiles and (begun < stages or at[(begun - stages) % sets] > begun - stages):
            todo.append((begun + 1, flying | {begun}, phases, at))
        for t in flying:                                            # any copy under way may land next
            p = list(phases)
            p[t % stages] += 1
            todo.append((begun, flying - {t}, tuple(p), at))
        for s in range(sets):
            t = at[s]
            if t < tiles and (phases[t % stages] & 1) != (t // stages & 1):
                if phases[t % stages] < t // stages + 1:
                    early.add(t)
                    continue
                nxt = list(at)
                nxt[s] += sets
                todo.append((begun, flying, phases, tuple(nxt)))
    return early


@pytest.mark.parametrize("sets,stages,sound", [(1, 2, True), (1, 3, True), (1, 4, True), (2, 2, True), (2, 3, False),
                                               (2, 4, True)])
def test_which_rings_are_sound(sets, stages, sound):
    assert (not early_waits(stages, sets, 2 * stages + 3)) == sound


RULE = r"""
#include "kv4_layout.h"
#include <cstdio>
int main() {
  for (int sets = 1; sets <= 2; ++sets)
    for (int tile = 18432; tile <= 36864; tile *= 2)
      for (long room = 36864; room <= 240000; room += 1000)
        printf("%d %d %ld %d\n", sets, tile, room, g4::kv4_ring_stages(room, tile, sets));
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_ring_rule_is_sound(tmp_path):
    """Every number of stages that the rule gives is sound and, where two tiles fit, fits."""
    src = tmp_path / "rule.cpp"
    src.write_text(RULE)
    exe = tmp_path / "rule"
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    pairs = set()
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        sets, tile, room, stages = map(int, line.split())
        assert 2 <= stages <= 4 and (stages * tile <= room or room < 2 * tile)
        pairs.add((stages, sets))
    assert len(pairs) == 5
    for stages, sets in pairs:
        assert not early_waits(stages, sets, 2 * stages + 3)
    with open(os.path.join(CSRC, "kv4.cu")) as f:
        launches = [x for x in f if "stages =" in x]
    assert len(launches) == 1 and "kv4_ring_stages(room, C::kTile, C::kSets)" in launches[0]


def test_waits_answer_for_whole_warps():
    """A wait whose result decides what a warp does is voted on: lanes that left it with different
    answers (one at its limit, one on the abort flag) would miss each other at the next vote.  In the
    block kernel only the single issuing lane goes by the answer."""
    lines = open(os.path.join(CSRC, "kv4_attend.cuh")).read().splitlines()
    for x in lines:
        if "mbar_wait(" in x or "mbar_try(" in x:
            assert "__all_sync(0xFFFFFFFFu, mbar_" in x, x
    assert not any("!*sh.abort_flag" in x or "*sh.abort_flag ?" in x for x in lines)
    for x in open(os.path.join(CSRC, "kv4_block.cuh")).read().splitlines():
        if "kv4_wait(" in x and "__device__" not in x:
            before = x.split("kv4_wait(")[0].strip()
            assert before == "" or before.startswith("if (n >= ") or before.startswith("if (y >= ") or \
                before.startswith("if (runs >= ") or before in ("ok =", "bool ok ="), x
            if before.startswith("if"):
                after = before[before.index(")") + 1:].strip()
                assert after in ("", "ok ="), x
