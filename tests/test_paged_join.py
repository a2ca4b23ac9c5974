"""How the few-row kernel of the paged cache deals its units' key tiles to CTAs and joins the parts: no ticket counter
and no workspace slot may belong to two units, and every unit is joined once, whoever comes last.  The numbering is the
kernel's own (csrc/paged_join.h, compiled here for the host); the deal is restated from csrc/paged_few.cu (Walk)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "video_diffusion_transformer_sage_gb300", "csrc")
NAMES = {"join_groups": 1, "join_first": 3, "join_group_of": 3, "join_counter": 3, "join_unit_counter": 3,
         "join_group_slot": 3, "join_part_slot": 4}


@pytest.fixture(scope="module")
def J(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    tmp = tmp_path_factory.mktemp("join")
    src = '#include "paged_join.h"\nextern "C" {\n'
    for name, n in NAMES.items():
        args = ", ".join(f"int a{i}" for i in range(n))
        src += f"int c_{name}({args}) {{ return sage::{name}({', '.join(f'a{i}' for i in range(n))}); }}\n"
    src += "int c_max_ctas() { return sage::kFewMaxCtas; }\nint c_slots() { return sage::kPagedSlots; }\n"
    src += "int c_region() { return sage::kPagedMaxCtas; }\n}\n"
    (tmp / "j.cpp").write_text(src)
    lib = str(tmp / "j.so")
    subprocess.run([gxx, "-O1", "-shared", "-fPIC", "-I", CSRC, str(tmp / "j.cpp"), "-o", lib], check=True)
    return ctypes.CDLL(lib)


def deal(seqs, rows):
    """seqs: [(units, key tiles per unit)]; rows: rows of CTAs.  [(unit, first row, parts)] of the units that more than one
    part makes up, and whether units have rows of their own."""
    total = sum(u * n for u, n in seqs)
    even = -(-total // rows)
    if sum(u for u, _ in seqs) <= rows:
        for q in range(max(even, 4), even + 5):
            if sum(u * -(-n // q) for u, n in seqs) <= rows:
                out, row, unit = [], 0, 0
                for u, n in seqs:
                    for _ in range(u):
                        parts = -(-n // q)
                        if parts > 1:
                            out.append((unit, row, parts))
                        row += parts
                        unit += 1
                return out, True
    out, at, unit = [], 0, 0
    for u, n in seqs:
        for _ in range(u):
            first, last = at // even, (at + n - 1) // even
            if last > first:
                out.append((unit, first, last - first + 1))
            at += n
            unit += 1
    return out, False


def replay(J, seqs, rows, lock, rng):
    """Asserts that counters and slots have one owner each and that tickets drawn in a random order join every unit."""
    split, aligned = deal(seqs, rows)
    assert rows * lock <= J.c_max_ctas()
    most = 0
    for col in range(lock):
        counter_of, slot_of = {}, {}

        def own(table, key, who):
            assert table.setdefault(key, who) == who, (key, table[key], who)

        ctas = {}     # row -> [(is it the unit's first part, group counter, count, unit counter, groups, unit)]
        for unit, cf, parts in split:
            groups = J.c_join_groups(parts)
            assert 1 <= groups <= 16
            most = max(most, parts)
            firsts = [J.c_join_first(parts, groups, g) for g in range(groups + 1)]
            assert firsts[0] == 0 and firsts[-1] == parts and all(a < b for a, b in zip(firsts, firsts[1:]))
            for i in range(parts):
                g = J.c_join_group_of(parts, groups, i)
                assert firsts[g] <= i < firsts[g + 1]
                counter = J.c_join_counter(cf + firsts[g], lock, col)
                assert 0 <= counter < J.c_region()
                own(counter_of, counter, (unit, g))
                own(slot_of, J.c_join_part_slot(cf + i, lock, col, i == 0), (unit, "part", i))
                up = J.c_join_unit_counter(cf, lock, col)
                assert J.c_region() <= up < 2 * J.c_region()
                if groups > 1:
                    own(counter_of, up, (unit, "groups"))
                    own(slot_of, J.c_join_group_slot(cf + firsts[g], lock, col), (unit, "group", g))
                ctas.setdefault(cf + i, []).append((i == 0, counter, firsts[g + 1] - firsts[g], up, groups, unit))
        assert all(0 <= s < J.c_slots() for s in slot_of)
        # A CTA draws for the unit that it ends, then for the one that it begins; then it joins in that order.
        todo = {}
        for row, parts in ctas.items():
            parts.sort()
            assert len(parts) <= 2
            todo[row] = [("draw", x) for x in parts] + [("join", x) for x in parts]
        value, last, joined = {}, set(), []
        live = list(todo)
        while live:
            row = rng.choice(live)
            what, part = todo[row].pop(0)
            if not todo[row]:
                live.remove(row)
            begins, counter, count, up, groups, unit = part
            if what == "draw":
                value[counter] = value.get(counter, 0) + 1
                if value[counter] == count:
                    value[counter] = 0
                    last.add((row, begins))
            elif (row, begins) in last:
                if groups > 1:
                    value[up] = value.get(up, 0) + 1
                    if value[up] != groups:
                        continue
                    value[up] = 0
                joined.append(unit)
        assert sorted(joined) == [unit for unit, _, _ in split]
        assert not any(value.values())
    return most, aligned


def test_groups_of_every_number_of_parts(J):
    for parts in range(2, J.c_max_ctas() + 1):
        groups = J.c_join_groups(parts)
        firsts = [J.c_join_first(parts, groups, g) for g in range(groups + 1)]
        sizes = [b - a for a, b in zip(firsts, firsts[1:])]
        assert sum(sizes) == parts and max(sizes) - min(sizes) <= 1
        # none but the first group begins in the unit's last row, which the next unit may share
        assert min(sizes) >= 2 and all(f < parts - 1 for f in firsts[1:-1])


# (key tiles of each sequence's units, units of a sequence for a CTA row, rows, lock)
KNOWN = [
    ([16] * 20 + [1094] + [16] * 43, 1, 38, 4),       # 21 parts, the next unit but two begins in the 21st's row
    ([501] + [16] * 200, 1, 152, 1),
    ([521] + [16] * 200, 1, 148, 1),
    ([16] * 30 + [1900] + [40] * 3 + [1700] + [16] * 120, 1, 152, 1),
]


@pytest.mark.parametrize("case", KNOWN, ids=lambda c: f"{len(c[0])}seqs-max{max(c[0])}-{c[2]}x{c[3]}")
def test_one_long_sequence_among_short_ones(J, case):
    tiles, units, rows, lock = case
    for seed in range(20):
        most, aligned = replay(J, [(units, n) for n in tiles], rows, lock, random.Random(seed))
        assert most > 16 and not aligned


def test_random_batches(J):
    """Every number of parts above 16 that occurs, among them those that leave a remainder of one to the old square root."""
    rng = random.Random(5)
    seen, evens = set(), 0
    for _ in range(1500):
        lock = rng.choice((1, 1, 2, 4, 8))
        rows = rng.choice((148, 152, 160, 213)) // lock
        n = int(rng.choice((3, 40, 160, 300)) * (0.5 + rng.random()))
        short = rng.choice((2, 16, 60))
        seqs = [(rng.choice((1, 1, 2, 3)), 1 + int(rng.random() * short)) for _ in range(n)]
        for _ in range(rng.choice((0, 1, 1, 2, 3))):
            seqs.insert(rng.randrange(len(seqs) + 1), (1, rng.randrange(200, 3000)))
        most, aligned = replay(J, seqs, rows, lock, rng)
        evens += not aligned
        seen.add(most)
    assert evens > 500 and {21, 31, 43} <= seen
