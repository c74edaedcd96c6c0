"""Host checks of the generated k loops of the grouped products' large tiles (csrc/grouped_sched.inc).

A simulator runs each loop's control flow for a range of step counts and checks what keeps its waves together:

* every step of both sides is loaded once, to the stage step % 2, at the step's own offset, and none behind the last;
* a load goes into a stage only after a barrier that follows the completion of all reads of the stage's contents;
* a fragment read sees a stage whose loads of one step were all waited for (vmcnt) and then published by a barrier;
* every product takes the fragments of its own step, sub-step and block, whose reads were waited for (lgkmcnt; LDS reads
  complete in order), and a block's products follow each other from zero on;
* the last step loads the next tile's steps 0 and 1, the first into the stage that it does not read, and the next tile
  begins there;
* the epilogue reads each accumulator once, long enough after its last product, and stores each row group at its own offset;
* the committed include is what the generator writes.

All four waves run the same stream, so a barrier is the point where all waves' waited-for loads become visible.
"""
import importlib.util
import os
import re
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_fp16_gemm_nt_amd", "csrc")


def _gen():
    sys.path.insert(0, CSRC)
    try:
        spec = importlib.util.spec_from_file_location("gen_grouped_sched", os.path.join(CSRC, "gen_grouped_sched.py"))
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
    finally:
        sys.path.remove(CSRC)
    return mod


GEN = _gen()
NB = 8
LOAD = re.compile(r"buffer_load_dwordx4 (\S+), %\[rs([ab])\], %\[(ko|kh)([ab])\] offen(?: offset:(\d+))? lds$")
READ_R = re.compile(r"ds_read_b128 v\[(\d+):\d+\], %\[r([ab])([01])\] offset:(\d+)$")
READ_C = re.compile(r"ds_read_b64_tr_b16 v\[(\d+):(\d+)\], %\[r([ab])([0-7])\] offset:(\d+)$")
MFMA = re.compile(r"v_mfma_f32_16x16x32_@T@ a\[(\d+):\d+\], v\[(\d+):\d+\], v\[(\d+):\d+\], (0|a\[\d+:\d+\])$")


class Sim:
    """Runs the loop for tiles of kts[0], kts[1], ... steps, each carried on from the one before where `carry` says so."""

    def __init__(self, text, la, lb, wide, kts, carry, ext=0):
        self.lines, self.kts, self.wide, self.carry, self.ext = text.split("\n"), kts, wide, carry, ext
        self.layout = {"a": la, "b": lb}
        self.labels = {}
        for i, ln in enumerate(self.lines):
            if re.match(r"^\d+:$", ln):
                self.labels.setdefault(ln[:-1], []).append(i)

    def target(self, ref, pc):
        c = self.labels[ref[:-1]]
        return min(x for x in c if x > pc) if ref[-1] == "f" else max(x for x in c if x < pc)

    def run(self):
        self.vm = []                        # loads and stores in issue order
        self.content = {}                   # (side, stage, load) -> ((tile, step), "flight" | "landed" | "visible")
        self.unread = {}                    # (side, stage) -> "open" | "done" (reads since the last barrier, completed or not)
        self.loaded = set()
        par, out = 0, []
        for tile, kt in enumerate(self.kts):
            carried = tile > 0 and self.carry
            if not carried:
                par = 0
            out.append(self.tile(tile, kt, par, int(not carried)))
            par = (par + kt) % 2
            for k, (step, state) in list(self.content.items()):   # the barrier behind a tile
                if state == "landed":
                    self.content[k] = (step, "visible")
            assert all(v == "done" for v in self.unread.values())
            self.unread.clear()
        return out

    def tile(self, tile, kt, par, own):
        vm, content, unread, loaded = self.vm, self.content, self.unread, self.loaded
        s = {"koa": 0, "kob": 0}            # offsets in steps
        rem, scc, m0, sdo = kt, 0, None, None
        lgkm = []                           # LDS operations in issue order
        frag, half = {}, {}                 # first VGPR -> (side, step, sub-step, block) once complete
        head, ht = {}, None
        done = {}                           # accumulator block -> products so far
        final, read_acc, stores, barriers = {}, set(), 0, 0
        clock, pc, steps = 0, 0, 0

        def complete(n):
            while len(lgkm) > n:
                op = lgkm.pop(0)
                if op[0] == "read":
                    _, reg, what, part = op
                    if part is None:
                        frag[reg] = what
                    elif part == 0:
                        half[reg] = what
                    else:
                        assert half.pop(reg) == what
                        frag[reg] = what
            if not lgkm:
                for k in unread:
                    unread[k] = "done"

        while pc < len(self.lines):
            ln = self.lines[pc]
            steps += 1
            assert steps < 100000
            nop = re.match(r"s_nop (\d+)$", ln)
            clock += int(nop.group(1)) + 1 if nop else 4 if ln.startswith("v_mfma") else 1
            if m := re.match(r"s_cmp_eq_u32 %\[rem\], (\d+)$", ln):
                scc = int(rem == int(m.group(1)))
            elif ln == "s_cmp_eq_u32 %[wide], 0":
                scc = int(not self.wide)
            elif m := re.match(r"s_cmp_eq_u32 %\[(first|par)\], 0$", ln):
                scc = int((own if m.group(1) == "first" else par) == 0)
            elif ln.startswith("s_cbranch_scc0 "):
                if not scc:
                    pc = self.target(ln.split()[1], pc)
                    continue
            elif m := re.match(r"v_or_b32 %\[ht\], %\[([ab])x(\d)\], %\[hm([01])\]$", ln):
                assert self.layout[m.group(1)] == "r" and int(m.group(3)) == int(m.group(2)) % 2
                ht = (m.group(1), int(m.group(2)))
            elif ln == "v_mov_b32 %[ht], 0x80000000":
                ht = "beyond"
            elif ln == "v_cmp_le_i32 vcc, %[khb], %[kr]":
                pass
            elif m := re.match(r"v_cndmask_b32 %\[ht\], %\[ht\], %\[bx(\d)\], vcc$", ln):
                assert masked == 2 * int(m.group(1)) and self.layout["b"] == "c" and ht == "beyond"
                ht = ("b", int(m.group(1)))
            elif m := re.match(r"s_mov_b32 %\[kh([ab])\], (128|%\[st([ab])\])$", ln):
                assert m.group(2) == ("128" if self.layout[m.group(1)] == "r" else f"%[st{m.group(1)}]")
                s["kh" + m.group(1)] = 1
            elif m := re.match(r"buffer_load_dwordx4 (\S+), %\[rs([ab])n\], (?:0|%\[kh([ab])\]) offen(?: offset:(\d+))? lds$", ln):
                op, imm = m.group(2), int(m.group(4) or 0)
                nstep = 0 if m.group(3) is None else s["kh" + m.group(3)]
                assert m.group(3) in (None, op) and nstep in (0, 1)
                r = re.match(r"%\[([ab])x(\d)\]$", m.group(1))
                side, q = (r.group(1), int(r.group(2))) if r else ht
                assert side == op and imm == 1024 * (q % 4) and m0 is not None and pc - m0[1] > 1
                assert (r is None) == (self.layout["a"] == "r" and nstep == 0), "masked where a first step can be partial"
                stage, at = divmod(m0[0] + imm - (65536 if op == "b" else 0), 32768)
                assert at == 1024 * q and stage == (par + kt + nstep) % 2, "step 0 goes to the stage that the last step does not read"
                assert (op, stage) not in unread and content[op, stage, q][1] != "flight"
                on = self.carry and tile + 1 < len(self.kts)
                if on:
                    assert (tile + 1, op, nstep, q) not in loaded
                    loaded.add((tile + 1, op, nstep, q))
                content[op, stage, q] = ((tile + 1, nstep) if on else ("empty", 0), "flight")
                vm.append(("load", (op, stage, q)))
            elif ln == "s_cmp_eq_u32 %[ext], 0":
                scc = int(not self.ext)
            elif m := re.match(r"s_mov_b32 %\[kha\], (\d+)$", ln):
                s["far"] = int(m.group(1))
            elif m := re.match(r"s_mul_i32 %\[khb\], %\[sb8\], (\d)$", ln):
                s["rows8"] = int(m.group(1))
            elif m := re.match(r"buffer_load_dwordx4 %\[h([ab])([01])\], %\[rs([ab])0\], %\[kh([ab])\] offen(?: offset:(\d+))? lds$", ln):
                op, odd, imm = m.group(1), int(m.group(2)), int(m.group(5) or 0)
                assert op == m.group(3) == m.group(4) and m0 is not None and pc - m0[1] > 1
                q, rest = divmod(m0[0] + imm - (65536 if op == "b" else 0), 1024)
                assert rest == 0 and 0 <= q < 8 and q % 2 == odd
                assert s["far"] + imm == 1024 * q if op == "a" else s["rows8"] == q and imm == 0   # rows 8 q further on
                assert (tile, op, 0, q) not in loaded
                loaded.add((tile, op, 0, q))
                content[op, 0, q] = ((tile, 0), "flight")
                vm.append(("load", (op, 0, q)))
            elif ln.startswith("s_cbranch_scc1 "):
                if scc:
                    pc = self.target(ln.split()[1], pc)
                    continue
            elif ln.startswith("s_branch "):
                pc = self.target(ln.split()[1], pc)
                continue
            elif ln == "s_sub_u32 %[rem], %[rem], 1":
                rem -= 1
            elif m := re.match(r"s_add_u32 m0, %\[lb\], (\d+)$", ln):
                m0 = (int(m.group(1)), pc)
            elif m := re.match(r"s_add_u32 %\[(k[oh])([ab])\], %\[(k[oh])([ab])\], (\S+)$", ln):
                assert m.group(2) == m.group(4)
                assert m.group(5) == ("128" if self.layout[m.group(2)] == "r" else f"%[st{m.group(2)}]")
                s[m.group(1) + m.group(2)] = s[m.group(3) + m.group(4)] + 1
            elif ln == "s_mov_b32 %[sdo], 0":
                sdo = 0
            elif ln == "s_add_u32 %[sdo], %[sdo], %[gstr]":
                sdo += 1
            elif m := re.match(r"v_or_b32 v(\d+), %\[([ab])x(\d)\], %\[hm([01])\]$", ln):
                assert self.layout[m.group(2)] == "r" and int(m.group(4)) == int(m.group(3)) % 2
                head[m.group(1)] = (m.group(2), int(m.group(3)))
            elif m := re.match(r"s_sub_i32 %\[khb\], %\[hk\], (\d+)$", ln):
                masked = int(m.group(1))
            elif ln in ("v_cmp_gt_i32 vcc, %[khb], %[kr]", "v_bfrev_b32 v80, 1"):
                pass
            elif m := re.match(r"v_cndmask_b32 v(\d+), %\[bx(\d)\], v80, vcc$", ln):
                assert masked == 2 * int(m.group(2)) and self.layout["b"] == "c"
                head[m.group(1)] = ("b", int(m.group(2)))
            elif m := LOAD.match(ln):
                reg, op, kreg, kop, imm = m.groups()
                assert op == kop and m0 is not None and pc - m0[1] > 1
                r = re.match(r"%\[([ab])x(\d)\]$", reg)
                side, q = (r.group(1), int(r.group(2))) if r else head[reg[1:]]
                at, imm = m0[0], int(imm or 0)
                assert side == op and imm == 1024 * (q % 4)
                at -= 65536 if op == "b" else 0
                stage, at = divmod(at + imm, 32768)
                assert stage in (0, 1) and at == 1024 * q
                first = s[kreg + op] == 0
                step = s[kreg + op] + self.ext
                assert step < kt and (step + par) % 2 == stage, "a step behind the last, or in the wrong stage"
                assert (r is None) == (first and self.layout["a"] == "r"), "the first step alone goes by masked offsets"
                assert (tile, op, step, q) not in loaded
                loaded.add((tile, op, step, q))
                assert (op, stage) not in unread, "a load into a stage that is still read"
                assert content.get((op, stage, q), (0, ""))[1] != "flight", "two loads to one place"
                content[op, stage, q] = ((tile, step), "flight")
                vm.append(("load", (op, stage, q)))
            elif m := re.match(r"s_waitcnt (?:vmcnt\((\d+)\))?\s*(?:lgkmcnt\((\d+)\))?$", ln):
                if m.group(1) is not None:
                    while len(vm) > int(m.group(1)):
                        kind, key = vm.pop(0)
                        if kind == "load":
                            content[key] = (content[key][0], "landed")
                if m.group(2) is not None:
                    complete(int(m.group(2)))
            elif ln == "s_barrier":
                barriers += 1
                assert not lgkm, "LDS operations in flight across a barrier"
                for key, (step, state) in list(content.items()):
                    if state == "landed":
                        content[key] = (step, "visible")
                for k in [k for k, v in unread.items() if v == "done"]:
                    del unread[k]
            elif (m := READ_R.match(ln)) or READ_C.match(ln):
                if m:
                    reg, op, h, off = int(m.group(1)), m.group(2), int(m.group(3)), int(m.group(4))
                    assert self.layout[op] == "r"
                    stage, off = divmod(off, 32768)
                    idx, odd = divmod(off, 2048)
                    part = None
                    assert odd == 0 and idx < NB
                else:
                    m = READ_C.match(ln)
                    reg, op, idx, off = int(m.group(1)), m.group(3), int(m.group(4)), int(m.group(5))
                    assert self.layout[op] == "c" and int(m.group(2)) == reg + 1
                    stage, off = divmod(off, 32768)
                    h, off = divmod(off, 32 * 512)
                    part = {0: 0, 4 * 512: 1}[off]
                    reg -= 2 * part
                held = {content[op, stage, q] for q in range(8)}
                assert len(held) == 1, "a stage of two steps"
                (whose, step), state = held.pop()
                assert state == "visible" and whose == tile
                frag.pop(reg, None)
                lgkm.append(("read", reg, (op, step, h, idx), part))
                unread[op, stage] = "open"
            elif m := MFMA.match(ln):
                acc, b, a = int(m.group(1)), int(m.group(2)), int(m.group(3))
                block, n = acc // 4, done.get(acc // 4, 0)
                i, j = divmod(block, NB)
                assert frag.get(a) == ("a", n // 2, n % 2, i), (pc, frag.get(a), n, i)
                assert frag.get(b) == ("b", n // 2, n % 2, j)
                assert (m.group(4) == "0") == (n == 0) and (n == 0 or m.group(4) == f"a[{acc}:{acc + 3}]")
                done[block] = n + 1
                if n + 1 == 2 * kt:
                    final[block] = clock - 4   # its own issue is 4 wait states at least
            elif m := re.match(r"v_accvgpr_read_b32 v(\d+), a(\d+)$", ln):
                acc = int(m.group(2))
                assert acc not in read_acc and clock - final[acc // 4] >= 11, "an accumulator read too early or twice"
                read_acc.add(acc)
                for base in [x for x in frag if x <= int(m.group(1)) < x + 4]:
                    del frag[base]
            elif ln.startswith("v_cvt_pk_@T@_f32 "):
                pass
            elif ln.startswith("ds_write_b64 "):
                lgkm.append(("write",))
            elif ln.startswith("ds_read_b128 ") and "%[er" in ln:
                assert not any(x[0] == "write" for x in lgkm)
                lgkm.append(("staged",))
            elif ln.startswith("buffer_store_dwordx4 "):
                assert sdo is not None and sdo == stores // (8 if self.wide else 4)
                assert self.wide or not lgkm
                assert ("%[sw]" in ln) == self.wide
                vm.append(("store", None))
                stores += 1
            elif nop or re.match(r"^\d+:$", ln):
                pass
            else:
                raise AssertionError(f"unknown instruction {ln}")
            pc += 1
        complete(0)
        return dict(done=done, read=read_acc, stores=stores, barriers=barriers, rem=rem)


@pytest.mark.parametrize("name", sorted(GEN.LOOPS))
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("ext", [0, 1])
@pytest.mark.parametrize("kts,carry", [((2,), False), ((3,), False), ((4,), False), ((5,), False), ((6,), False), ((12,), False), ((33,), False),
                                       ((4, 3), False), ((2, 2, 2), True), ((3, 3, 3), True), ((4, 5, 2, 3, 7, 6, 2), True), ((12, 13, 12), True)])
def test_loop(name, kts, carry, ext, wide):
    if ext and (name != "G16_GROUPED_RR" or carry):
        pytest.skip("this loop has no such step, and tiles with one are not carried on to")
    la, lb, p = GEN.LOOPS[name]
    sim = Sim(GEN.generate(la, lb, p), la, lb, wide, kts, carry, ext)
    runs = sim.run()
    want = {(t, op, s, q) for t, kt in enumerate(kts) for op in "ab" for s in range(kt) for q in range(8)}
    assert sim.loaded == want
    for r, kt in zip(runs, kts):
        assert r["done"] == {b: 2 * kt for b in range(64)}
        assert r["read"] == set(range(256))
        assert r["stores"] == (64 if wide else 32)
        # one for step 0, a release for each step that loads and the last, a publish for each but the last
        assert r["barriers"] == 2 * kt - 1


def test_committed_include():
    want = "// Generated by gen_grouped_sched.py.  Do not edit.\n"
    for name, (la, lb, p) in GEN.LOOPS.items():
        want += f"// {name}: {GEN.ring4.params_line(p)}.\n" + GEN.as_macro(name, GEN.generate(la, lb, p))
    assert open(os.path.join(CSRC, "grouped_sched.inc")).read() == want
