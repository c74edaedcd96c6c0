"""Host checks of the grouped products' loop that begins with two steps of another product (G16_GROUPED_RR2, for adapters of
more than 32 ranks), and of tiles carried on from ones with such steps, on the simulator of test_grouped_schedule.py.

There the simulator knows one leading step; here it also takes a second, loaded into the other stage from %[rsa1], and a
masked first step of the contraction whose offsets are made load by load.
"""
import inspect
import re
import textwrap

import pytest

from tests import test_grouped_schedule as one

GEN = one.GEN


def _simulator():
    src = textwrap.dedent(inspect.getsource(one.Sim))
    changes = [
        # whether there are such steps, and how many, is the tile's own; a carried tile has none
        ("out.append(self.tile(tile, kt, par, int(not carried)))", "self.ext = self.exts[tile]\nout.append(self.tile(tile, kt, par, int(not carried)))"),
        ("carried = tile > 0 and self.carry", "carried = tile > 0 and self.carry and self.exts[tile] == 0"),
        ("on = self.carry and tile + 1 < len(self.kts)", "on = self.carry and tile + 1 < len(self.kts) and self.exts[tile + 1] == 0"),
        # leading step n lies in stage n and comes from %[rsan]; both from %[rsb0]
        (r"%\[rs([ab])0\], %\[kh", r"%\[rs(a[01]|b0)\], %\[kh"),
        ("assert op == m.group(3) == m.group(4) and m0", "assert op == m.group(3)[0] == m.group(4) and m0"),
        ("assert rest == 0 and 0 <= q < 8 and q % 2 == odd", "lead, q = divmod(q, 32)\nassert rest == 0 and 0 <= q < 8 and q % 2 == odd and lead < self.ext and m.group(3) in (f'a{lead}', 'b0')"),
        ("assert (tile, op, 0, q) not in loaded", "assert (tile, op, lead, q) not in loaded"),
        ("loaded.add((tile, op, 0, q))", "loaded.add((tile, op, lead, q))"),
        ("content[op, 0, q] = ((tile, 0), \"flight\")", "content[op, lead, q] = ((tile, lead), \"flight\")"),
        ("vm.append((\"load\", (op, 0, q)))", "vm.append((\"load\", (op, lead, q)))"),
        ("s[\"far\"] = int(m.group(1))", "s[\"far\"] = s[\"kha\"] = int(m.group(1))"),
        # the contraction's first step, masked in the loop
        ("else head[reg[1:]]", "else ht if reg == '%[ht]' else head[reg[1:]]"),
        ("elif ln.startswith(\"s_cbranch_scc1 \"):", "elif ln == \"s_mov_b32 %[khb], 0\":\n    s[\"khb\"] = 0\nelif ln.startswith(\"s_cbranch_scc1 \"):"),
    ]
    for old, new in changes:
        assert src.count(old) == 1, old
        at = src.index(old)
        pad = re.search(r"[ ]*$", src[:at]).group(0)
        src = src.replace(old, new.replace("\n", "\n" + pad))
    space = dict(vars(one))
    exec(compile(src, "leads", "exec"), space)
    return space["Sim"]


SIM = _simulator()


def run(name, kts, exts, carry, wide):
    la, lb, p = GEN.LOOPS[name]
    sim = SIM(GEN.generate(la, lb, p), la, lb, wide, kts, carry)
    sim.exts = exts
    runs = sim.run()
    assert sim.loaded == {(t, op, s, q) for t, kt in enumerate(kts) for op in "ab" for s in range(kt) for q in range(8)}
    for r, kt in zip(runs, kts):
        assert r["done"] == {b: 2 * kt for b in range(64)}
        assert r["read"] == set(range(256))
        assert r["stores"] == (64 if wide else 32)
        assert r["barriers"] == 2 * kt - 1


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kt", [4, 5, 6, 7, 12, 33])
def test_two_leading_steps(kt, wide):
    run("G16_GROUPED_RR2", (kt,), (2,), False, wide)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("name,leads", [("G16_GROUPED_RR", 1), ("G16_GROUPED_RR2", 2)])
@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("kts", [(4, 4, 4), (5, 4, 6), (6, 2, 5), (4, 5, 2), (7, 3, 4)])
def test_tiles_with_and_without(kts, first, name, leads, wide):
    # a tile carried on from one with leading steps, and one with them behind one without
    exts = tuple(leads if (t + first) % 2 and kt >= 4 else 0 for t, kt in enumerate(kts))
    run(name, kts, exts, True, wide)
