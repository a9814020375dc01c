"""The few tokens' kernels wait for columns on their way to LDS by counting the loads behind them.  What they count
on is checked in the assembly of the built source: a step's columns come first, then its weight, nothing between
the two and nothing of the next step before them."""
import os
import re
import subprocess

import pytest

from combine_get_dispatch_04_amd import build as B

SOURCE = os.path.join(B.CSRC, "ep_expert_few.hip")
COLUMN, WEIGHT, OTHER, BARRIER, MEET, LABEL = "column", "weight", "other", "barrier", "wait and barrier", "label"


def assembly(path):
    flags = [f for f in B.FLAGS if f not in ("-shared", "-Wall")]
    r = subprocess.run([B.HIPCC, *flags, f"-I{B.INCLUDE}", f"-I{B.CSRC}", "--cuda-device-only", "-S", SOURCE, "-o", path],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    with open(path) as f:
        return f.read()


def events(text):
    """kernel -> its vector memory loads and barriers (with how many loads the instruction in front of one leaves in
    flight, if it is a wait for all but some), in the order of the text."""
    out, cur, left = {}, None, 0
    for line in text.splitlines():
        m = re.match(r"^(_ZN\S*few_(?:up|down)_kernelILb([01])ELb([01])E\S*):", line)
        if m:
            cur = out.setdefault((m.group(1), m.group(2) == "1", m.group(3) == "1"), [])
        elif line.startswith("_ZN"):
            cur = None
        if cur is None:
            continue
        s = line.strip()
        if s.startswith("buffer_load"):
            cur.append((COLUMN if re.search(r"\blds\b", s) else OTHER, 0))
        elif s.startswith("global_load"):
            cur.append((WEIGHT if s.startswith("global_load_dwordx4") and s.endswith(" nt") else OTHER, 0))
        elif s.startswith(("flat_load", "scratch_load")):
            cur.append((OTHER, 0))
        elif s.startswith("s_barrier"):
            cur.append((MEET if left else BARRIER, left))
        elif re.match(r"^\.LBB\S+:", s):
            cur.append((LABEL, 0))
        if s and not s.startswith(";"):
            m = re.match(r"s_waitcnt.*vmcnt\((\d+)\)", s)
            left = int(m.group(1)) if m else 0
    return out


def shared_faults(ev, per_step):
    """Behind each run of columns' loads come per_step of the weight, before anything else is loaded."""
    faults, steps, i = [], 0, 0
    loads = [(n, k) for n, (k, _) in enumerate(ev) if k != LABEL]
    while i < len(loads):
        if loads[i][1] == WEIGHT:
            faults.append((loads[i][0], "a weight without columns in front of it"))
            i += 1
        elif loads[i][1] == COLUMN:
            at, run = loads[i][0], 0
            while i < len(loads) and loads[i][1] == COLUMN:
                run, i = run + 1, i + 1
            weights = 0
            while i < len(loads) and loads[i][1] == WEIGHT and weights < per_step:
                weights, i = weights + 1, i + 1
            if run not in (1, 2, 4) or weights != per_step:
                faults.append((at, f"{run} columns' loads, {weights} of the weight"))
            steps += 1
        else:
            i += 1
    return steps, faults


def staged_faults(ev):
    """In front of a barrier that leaves loads in flight stand as many of the weight, in its own basic block."""
    faults, waits = [], 0
    for i, (k, n) in enumerate(ev):
        if k == MEET:
            waits += 1
            before = [e[0] for e in ev[max(0, i - n):i]]
            if before != [WEIGHT] * n:
                faults.append((i, before))
    return waits, faults


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc is not available")
    ev = events(assembly(str(tmp_path_factory.mktemp("asm") / "few.s")))
    assert len(ev) == 8
    return ev


def test_columns_come_before_their_weight(kernels):
    for (name, fp4, wide), ev in kernels.items():
        if wide:
            steps, faults = shared_faults(ev, 2 if fp4 else 8)
            # three forms (8, 16 or 32 columns and more), each with the steps in front of and in the loop
            assert steps >= 3 * (3 + 4) and not faults, (name, steps, faults[:5])


def test_staged_columns_come_before_the_first_weight(kernels):
    for (name, fp4, wide), ev in kernels.items():
        if fp4 and not wide:
            waits, faults = staged_faults(ev)
            assert waits == 1 and not faults, (name, faults[:5])


def test_the_checks_see_loads_out_of_order():
    step = [(COLUMN, 0)] * 2 + [(WEIGHT, 0)] * 2
    assert shared_faults(step * 3, 2) == (3, [])
    assert shared_faults([(OTHER, 0)] + step + [(MEET, 4)] + step, 2) == (2, [])
    for bad in ([(WEIGHT, 0)] + step, [(COLUMN, 0)] * 2 + [(WEIGHT, 0)], step + step[:3] + [(BARRIER, 0), (WEIGHT, 0)],
                [(COLUMN, 0), (WEIGHT, 0), (COLUMN, 0), (WEIGHT, 0)], [(COLUMN, 0), (OTHER, 0), (WEIGHT, 0), (WEIGHT, 0)],
                [(COLUMN, 0)] * 3 + [(WEIGHT, 0)] * 2):
        assert shared_faults(bad, 2)[1]
    good = [(WEIGHT, 0)] * 4 + [(MEET, 4)]
    assert staged_faults(good) == (1, [])
    assert staged_faults(good[1:])[1] and staged_faults(good[:2] + [(OTHER, 0)] + good[2:])[1]
    assert staged_faults(good[:2] + [(LABEL, 0)] + good[2:])[1]
