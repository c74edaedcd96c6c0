"""Generate the instruction schedules of the grouped products' large tiles (grouped_ring.hpp).

The k loops are inline assembly, as those of the four-wave ring are, and for
the same reason: with one wave to a SIMD nothing hides a stalled instruction
stream, so the order of matrix-core instructions, LDS reads, loads to LDS and
waits is fixed here.  Run it after changing a schedule:

    python gen_grouped_sched.py            # writes grouped_sched.inc

Output tile 256 x 256, 64-wide steps of the contraction, 4 waves of 128 x 128
(8 x 8 blocks of v_mfma_f32_16x16x32, each block's two 32-wide sub-steps back
to back), two LDS stages.  The A side (rows of the output) and the B side
(columns) are each in one of two layouts:

  r   by rows: the contraction is contiguous.  LDS rows of 128 bytes, one for
      each row of the side; a fragment is one ds_read_b128;
  c   by columns: the side's own index is contiguous.  LDS rows of 512 bytes,
      one for each element of the contraction; a fragment is two
      ds_read_b64_tr_b16, each 4 elements of the contraction for 16 columns
      and 4 groups of lanes.

The loops that are generated are RR, RC and CC, for the grouped products NT, NN
and TN, and RR2, for adapters.  Each is a macro with the operands' type, "f16"
or "bf16", as its argument, and ends with one of two epilogues: outputs rounded
to that type, or, where %[wide] is not 0, in 32 bits.

LDS: the A side's stages at 0 and 32 KiB, the B side's at 64 and 96 KiB, so
that one address and an instruction offset reach both stages, then 8 KiB for
each wave's epilogue.  Registers are those of the four-wave ring's fourth form:
accumulators a0..a255, A fragments v64..v127, two sets of B fragments
v128..v255, whose idle set serves the epilogue.

A step j of the contraction: the late rows' A fragments of this step; a
release barrier (this wave's and all others' reads of the stage are done); the
16 loads of step j + 2 into it, spread out; a publish barrier (the loads of
step j + 1 have landed everywhere); the fragment reads of step j + 1: B blocks
into the other set, A rows as their rows of this step are done.

The contraction need not be a multiple of 64.  A side by rows then begins
before its first element, by as much as is missing, and step 0's chunks that
lie before it get offsets past the buffer's end (%[hm0], %[hm1]), which load
zeros; a side by columns beside it begins that many rows early, and those
rows' offsets are masked likewise.  With both sides by columns the rows behind
the last load zeros by themselves: the buffers end there.

From tile to tile: the last step also loads steps 0 and 1 of the workgroup's
next tile, from %[rsan] and %[rsbn], the first into the stage that it does not
read, the second behind a release barrier into its own, so that the next tile's
block begins with both on the way (%[first] is 0 then, and %[par] the stage of
step 0; otherwise a tile loads them itself, step 0 into stage 0).  Where there
is no such tile these buffers are empty.

RR can begin with a step of another product, whose operands have rows of their
own (the second product of a low-rank adapter, up to 64 elements of its
contraction): where %[ext] is not 0, step 0 is loaded from %[rsa0] (rows of 128
bytes, lane offsets %[ha0], %[ha1] for even and odd loads) and %[rsb0] (lane
offsets %[hb0], %[hb1], %[sb8] bytes for 8 rows), and the contraction's first
step, with its masks, is step 1.  RR2 is RR with two such steps, the second from
%[rsa1] and again %[rsb0]; a step 0 of its own then loads the contraction's
first, masked, as step 2.  It needs four steps in all where it has these.

Operands: load offsets %[axQ], %[bxQ] (less 1024 * (Q mod 4), the instruction
offset of the load); fragment addresses %[raN], %[rbN] (N: sub-step by rows,
block by columns); resources %[rsa], %[rsb], %[rsd]; the wave's LDS load base
%[lb]; the steps' byte offsets %[koa], %[kha], %[kob], %[khb] (next step and
the one after; the first of each is 0 on entry), advanced by 128 by rows and
by %[sta], %[stb] by columns;
the count %[rem] of steps, at least 2; epilogue
%[ewJ], %[erQ], %[soQ], or %[sw] with %[wide], %[gstr], scratch %[sdo]; RC:
%[hk] masked rows and %[kr], the lane's row of its first load.
"""
from __future__ import annotations

import os
import sys

import gen_ring4_sched as ring4
from gen_ring4_sched import KSUB, LOAD3, NB, NLOAD, NQ, a4, areg, b4, epi_set4, head_reg, late_rows4, mfma_block

STAGE_BYTES = 32768     # of one side
SIDE_B = 65536
HALF_C = 32 * 512       # bytes of 32 LDS rows by columns


def side_steps(op: str, layout: str) -> str:
    return "128" if layout == "r" else f"%[st{op}]"


class Emitter(ring4.Emitter):
    def __init__(self, la: str, lb: str) -> None:
        super().__init__()
        self.layout = {"a": la, "b": lb}
        self.wide = False
        self.behind: list[tuple] = []   # loads and stores behind the next tile's step 0, and its step 1, for each last step

    @staticmethod
    def m0(op: str, q: int, stage: int) -> str:
        return f"s_add_u32 m0, %[lb], {stage * STAGE_BYTES + (SIDE_B if op == 'b' else 0) + 4096 * (q // 4)}"

    @staticmethod
    def load(op: str, q: int, koff: str, reg: str | None = None) -> str:
        imm = 1024 * (q % 4)
        off = f" offset:{imm}" if imm else ""
        return f"buffer_load_dwordx4 {reg or f'%[{op}x{q}]'}, %[rs{op}], %[{koff}{op}] offen{off} lds"

    def parts(self, op: str) -> tuple:
        """The instructions of a fragment read."""
        return (None,) if self.layout[op] == "r" else (0, 1)

    def read(self, op: str, h: int, idx: int, stage: int, p: int, part) -> None:
        reg = a4(h, idx) if op == "a" else b4(p, h, idx)
        key = (op, h, idx, p if op == "b" else None)
        if part is None:
            off = stage * STAGE_BYTES + 2048 * idx
            self.op(f"ds_read_b128 {reg}, %[r{op}{h}] offset:{off}")
            self.lgkm.append(key)
            return
        first = int(reg[2:].split(":")[0]) + 2 * part
        off = stage * STAGE_BYTES + h * HALF_C + 2048 * part
        self.op(f"ds_read_b64_tr_b16 v[{first}:{first + 1}], %[r{op}{idx}] offset:{off}")
        self.lgkm.append(key if part == 1 else ("first half", *key))

    def mfma(self, p: int, h: int, i: int, j: int, first: bool) -> None:
        self.wait_frag(("a", h, i, None), ("b", h, j, p))
        c = areg(i, j)
        self.op(f"v_mfma_f32_16x16x32_@T@ {c}, {b4(p, h, j)}, {a4(h, i)}, {'0' if first else c}")

    # --- epilogue: rows of 16, as soon as their last products are done -------
    def group(self, i: int, t: int) -> list[tuple[str, bool]]:
        if not self.wide:
            return [(text.replace("v_cvt_pk_f16_f32", "v_cvt_pk_@T@_f32"), lds) for text, lds in ring4.epilogue_group(i, t, t + 32)]
        # 32-bit outputs: four columns of a row from each lane, 64 bytes of 16
        # rows to a store; ordinary stores, so that L2 joins the halves of lines
        out: list[tuple[str, bool]] = []
        base = t + 32 * (i % 2)
        for j in range(NB):
            v, b = base + 4 * j, NB * i + j
            out += [(f"v_accvgpr_read_b32 v{v + r}, a{4 * b + r}", False) for r in range(4)]
            off = f" offset:{64 * j}" if j else ""
            out.append((f"buffer_store_dwordx4 v[{v}:{v + 3}], %[sw], %[rsd], %[sdo] offen{off}", False))
        out.append(("s_add_u32 %[sdo], %[sdo], %[gstr]", False))
        return out

    def next_load(self, op: str, q: int, step: int) -> list[str]:
        """Load q of the next tile's step 0 or 1, with what masks its offset."""
        layout = self.layout
        imm = 1024 * (q % 4)
        off = f" offset:{imm}" if imm else ""
        if step == 1:
            return [f"buffer_load_dwordx4 %[{op}x{q}], %[rs{op}n], %[kh{op}] offen{off} lds"]
        load = f"buffer_load_dwordx4 %[ht], %[rs{op}n], 0 offen{off} lds"
        if layout["a"] == "c":
            return [load.replace("%[ht]", f"%[{op}x{q}]")]
        if layout[op] == "r":
            return [f"v_or_b32 %[ht], %[{op}x{q}], %[hm{q % 2}]", load]
        return [f"s_sub_i32 %[khb], %[hk], {2 * q}", "v_mov_b32 %[ht], 0x80000000", "v_cmp_le_i32 vcc, %[khb], %[kr]",
                f"v_cndmask_b32 %[ht], %[ht], %[bx{q}], vcc", load]

    def epi_after(self, g: int, per_slot: int, delay: int, t: int) -> None:
        while self.epi_next < NB and g >= 2 * NB * self.epi_next + 2 * NB - 1 + delay:
            self.epi_q += self.group(self.epi_next, t)
            self.epi_next += 1
        for _ in range(min(per_slot, len(self.epi_q))):
            self.epi_emit(*self.epi_q.pop(0))

    def epi_rest(self, t: int) -> None:
        for _ in range(3):
            self.op("s_nop 7")
        while self.epi_next < NB:
            self.epi_q += self.group(self.epi_next, t)
            self.epi_next += 1
        while self.epi_q:
            self.epi_emit(*self.epi_q.pop(0))


def emit_step(e: Emitter, stage: int, first: bool, ahead: bool, has_next: bool, last: bool, tail: list[str], p: dict, masked: bool = False) -> None:
    """One step reading `stage`.  ahead: it loads step j + 2 (masked: which is the contraction's first); has_next: step j + 1
    exists; last: with the epilogue."""
    ng = KSUB * NQ
    gaps: list[list[tuple]] = [[] for _ in range(ng)]
    late = late_rows4(p)
    rel, pub, every, limit = p["rel"], p["pub"], p["load_every"], p["read_limit"]

    def first_free(g: int) -> int:
        while gaps[g]:
            g += 1
        return g

    if not last:
        br = [t for t in tail if t.startswith(("s_cbranch", "s_branch"))]
        rest = [t for t in tail if t not in br]
        assert tail == rest + br, "branches close the tail"
        for k, t in enumerate(rest):
            gaps[ng - 1 - len(rest) + k].append(("text", t))
        for t in br:
            gaps[ng - 1].append(("text", t))
    if not first:
        g = 0
        for i in late:
            for h in range(KSUB):
                for part in e.parts("a"):
                    gaps[g].append(("read", ("a", h, i, stage, stage, part)))
                    g += 1
        assert g < rel - 1, "late reads after the release"
    if ahead:
        gaps[rel - 1].append(("text", "s_waitcnt lgkmcnt(0)", "clear"))
        gaps[rel].append(("text", "s_barrier"))
    if has_next:
        gaps[pub - 1].append(("wait",))
        gaps[pub].append(("text", "s_barrier"))
    loads = []
    if ahead:
        prev, group = -1, None
        for k, (op, q) in enumerate(LOAD3):
            g = first_free(max(rel + 1 + every * k, prev + 1))
            if (op, q // 4) != group:
                m = next((x for x in range(g - 1, max(prev, rel), -1) if not gaps[x]), None)
                if m is None:
                    m = first_free(max(prev, rel) + 1)
                    g = first_free(m + 1)
                gaps[m].append(("text", Emitter.m0(op, q, stage)))
                group = (op, q // 4)
            if masked:
                gaps[g].append(("text", f"v_or_b32 %[ht], %[{op}x{q}], %[hm{q % 2}]"))
            gaps[g].append(("text", Emitter.load(op, q, "kh", "%[ht]" if masked else None)))
            loads.append(g)
            prev = g
        assert prev < ng - 8, "loads run into the tail"
    if has_next:
        young = sum(1 for g in loads if g < pub - 1)   # loads of step j + 2 need not have landed
        gaps[pub - 1] = [("text", f"s_waitcnt vmcnt({young}) lgkmcnt(0)", "clear")]
        reads = [(pub + 1, ("a", h, 0, part)) for h in range(KSUB) if 0 not in late for part in e.parts("a")]
        reads += [(pub + 1, ("b", h, j, part)) for j in range(NB) for h in range(KSUB) for part in e.parts("b")]
        reads += [(max(pub + 1, 2 * NB * i + 2 * NB + p["a_delay"]), ("a", h, i, part)) for i in range(1, NB) if i not in late
                  for h in range(KSUB) for part in e.parts("a")]
        reads.sort(key=lambda r: r[0])
        g = at = pub + 1
        for n, (earliest, (op, h, idx, part)) in enumerate(reads):
            at = max(at, earliest)
            open_gaps = [x for x in range(at, limit) if not gaps[x]]
            crowded = len(reads) - n > len(open_gaps)   # two to a gap where one each does not fit
            g = next((x for x in range(at, limit) if len(gaps[x]) < (2 if crowded else 1) and all(it[0] == "read" for it in gaps[x])), None)
            assert g is not None, "next-step reads beyond the read limit"
            gaps[g].append(("read", (op, h, idx, stage ^ 1, stage ^ 1, part)))
            at = g
        gaps[first_free(g + p["f0_lat"])].append(("text", "s_waitcnt lgkmcnt(0)", "clear"))
    if last:
        # the late reads are the stage's last: behind this barrier it is free
        gaps[rel - 1].append(("text", "s_waitcnt lgkmcnt(0)", "clear"))
        gaps[rel].append(("text", "s_barrier"))
        lines = []
        for op, q in LOAD3:
            lines += ([Emitter.m0(op, q, stage ^ 1)] if q % 4 == 0 else []) + e.next_load(op, q, 0)
        for op in "ab":
            lines.append(f"s_mov_b32 %[kh{op}], {side_steps(op, e.layout[op])}")
        for op, q in LOAD3:
            lines += ([Emitter.m0(op, q, stage)] if q % 4 == 0 else []) + e.next_load(op, q, 1)
        # one to a gap, or two where one each does not fit; those of this stage behind the barrier
        from_gap, at = rel + 1, p["nxt_start"]
        own = next(n for n, text in enumerate(lines) if text == Emitter.m0("a", 0, stage))
        for n, text in enumerate(lines):
            if n == own:
                at = max(at, from_gap)
            gaps[at].append(("text", text))
            if sum(it[0] == "text" and it[1] in lines for it in gaps[at]) > (len(lines) - n) // max(1, ng - 2 - at):
                at += 1
        assert at < ng, "next-tile loads beyond the step"
    texts = [(g, it[1]) for g in range(ng) for it in gaps[g] if it[0] == "text"]
    writers = [g for g, t in texts if t.startswith(("s_add_u32", "s_sub_u32"))]
    compares = [g for g, t in texts if t.startswith("s_cmp")]
    assert last or not compares or max(writers, default=-1) < min(compares), "SCC clobbered before the branch"

    t_base = epi_set4(stage)
    start = len(e.lines)
    for g in range(ng):
        pq, h = divmod(g, 2)
        i, j = mfma_block(pq, "snake")
        if last and g == 0:
            e.epi_start("snake")
        e.mfma(stage, h, i, j, first and h == 0)
        if last:
            e.epi_after(g, p["epi_slot"], p["epi_delay"], t_base)
        for it in gaps[g]:
            if it[0] == "read":
                e.read(*it[1])
            else:
                e.op(it[1])
                if len(it) > 2:
                    e.lgkm.clear()
    if last:
        e.epi_rest(t_base)
        vm = [ln for ln in e.lines[start:] if ln.startswith("buffer_")]
        at = [n for n, ln in enumerate(vm) if ln.startswith("buffer_load")]
        e.behind.append((len(vm) - 1 - at[NLOAD - 1], len(vm) - 1 - at[2 * NLOAD - 1]))
        for t in tail:
            e.op(t)


def generate(la: str, lb: str, p: dict) -> str:
    e = Emitter(la, lb)
    layout = e.layout
    head = {op: "none" if la == "c" else layout[op] for op in "ab"}

    def loads(step: int, masked: bool, stage: int) -> None:
        for op, q in LOAD3:
            if q % 4 == 0:
                e.op(Emitter.m0(op, q, stage))
                e.op("s_nop 0")   # M0 write -> LDS-DMA read of M0
            e.op(Emitter.load(op, q, "ko", f"v{head_reg(op, q)}" if masked and head[op] != "none" else None))

    def rest(stage: int, wait: str) -> None:
        for op in "ab":
            e.op(f"s_add_u32 %[kh{op}], %[ko{op}], {side_steps(op, layout[op])}")
        e.op(f"s_waitcnt vmcnt({wait})")
        e.op("s_barrier")
        e.lgkm = []
        order = [("a", h, 0) for h in range(KSUB)] + [("b", h, j) for j in range(NB) for h in range(KSUB)]
        order += [("a", h, i) for i in range(1, NB) for h in range(KSUB)]
        for op, h, idx in order:
            for part in e.parts(op):
                e.read(op, h, idx, stage, stage, part)

    def advance() -> None:
        for op in "ab":
            e.op(f"s_add_u32 %[ko{op}], %[ko{op}], {side_steps(op, layout[op])}")

    adv = [f"s_add_u32 %[kh{op}], %[kh{op}], {side_steps(op, layout[op])}" for op in "ab"]
    sub, cmp2 = "s_sub_u32 %[rem], %[rem], 1", "s_cmp_eq_u32 %[rem], 2"

    def step(stage, first, ahead, has_next, last, tail, masked=False):
        pending = list(e.lgkm) if first else []
        e.lgkm = pending
        emit_step(e, stage, first, ahead, has_next, last, tail, p, masked)

    e.op("s_cmp_eq_u32 %[first], 0")
    e.op("s_cbranch_scc1 15f")
    # this tile's own first steps, behind what the tile before loaded from empty buffers
    e.op("s_waitcnt vmcnt(@BEHIND@)")
    for op, q in LOAD3:
        if head[op] == "r":
            e.op(f"v_or_b32 v{head_reg(op, q)}, %[{op}x{q}], %[hm{q % 2}]")
    if head["b"] == "c":   # rows 2 q further on for load q
        e.op("v_bfrev_b32 v80, 1")   # 0x80000000
        for q in range(8):
            e.op(f"s_sub_i32 %[khb], %[hk], {2 * q}")
            e.op("v_cmp_gt_i32 vcc, %[khb], %[kr]")
            e.op(f"v_cndmask_b32 v{head_reg('b', q)}, %[bx{q}], v80, vcc")
    if layout == {"a": "r", "b": "r"}:
        e.op("s_cmp_eq_u32 %[ext], 0")
        e.op("s_cbranch_scc1 11f")
        for term in range(p.get("leads", 1)):
            for q in range(8):
                if q % 4 == 0:
                    e.op(f"s_mov_b32 %[kha], {4096 * (q // 4)}")
                    e.op(Emitter.m0("a", q, term))
                    e.op("s_nop 0")
                off = f" offset:{1024 * (q % 4)}" if q % 4 else ""
                e.op(f"buffer_load_dwordx4 %[ha{q % 2}], %[rsa{term}], %[kha] offen{off} lds")
            for q in range(8):
                e.op(f"s_mul_i32 %[khb], %[sb8], {q}")
                e.op(f"s_add_u32 m0, %[lb], {SIDE_B + STAGE_BYTES * term + 1024 * q}")
                e.op("s_nop 0")
                e.op(f"buffer_load_dwordx4 %[hb{q % 2}], %[rsb0], %[khb] offen lds")
        if p.get("leads", 1) == 1:
            loads(1, True, 1)
            e.op("s_branch 12f")
        else:   # a step 0 of its own, which loads the contraction's first
            rest(0, str(NLOAD))
            for op in "ab":
                e.op(f"s_mov_b32 %[kh{op}], 0")
            step(0, True, True, True, False, adv + [sub, cmp2, "s_cbranch_scc1 6f", "s_branch 1f"], True)
        e.label("11")
    loads(0, True, 0)
    advance()
    loads(1, False, 1)
    if layout == {"a": "r", "b": "r"} and p.get("leads", 1) == 1:
        e.label("12")
    rest(0, str(NLOAD))
    zero = list(e.lgkm)   # the reads under way at label 20, from either side
    e.op("s_branch 20f")
    # carried from the tile before: step 0 has to be there, what came behind it not
    e.label("15")
    advance()
    e.op("s_cmp_eq_u32 %[par], 0")
    e.op("s_cbranch_scc0 16f")
    rest(0, "@WAIT@")
    e.op("s_branch 20f")
    e.label("16")
    rest(1, "@WAIT@")
    entry = list(e.lgkm)
    e.op(cmp2)
    e.op("s_cbranch_scc1 25f")
    step(1, True, True, True, False, adv + [sub, cmp2, "s_cbranch_scc1 8f", "s_branch 17f"])
    e.label("25")
    e.lgkm = list(entry)
    step(1, True, False, True, False, [sub, "s_branch 3f"])     # two steps in all

    e.label("20")
    e.lgkm = list(zero)
    e.op(cmp2)
    e.op("s_cbranch_scc1 5f")
    step(0, True, True, True, False, adv + [sub, cmp2, "s_cbranch_scc1 6f"])
    e.label("1")
    step(1, False, True, True, False, adv + [sub, cmp2, "s_cbranch_scc1 8f"])
    e.label("17")
    step(0, False, True, True, False, adv + [sub, cmp2, "s_cbranch_scc1 6f", "s_branch 1b"])
    e.label("5")
    e.lgkm = list(zero)
    step(0, True, False, True, False, [sub, "s_branch 2f"])     # two steps in all
    e.label("6")
    step(1, False, False, True, False, [sub, "s_branch 3f"])    # the step before the last, in stage 1
    e.label("8")
    step(0, False, False, True, False, [sub])                   # the same in stage 0
    for name, stage, narrow in (("2", 1, "9"), ("3", 0, "10")):  # the last step
        e.label(name)
        e.op("s_cmp_eq_u32 %[wide], 0")
        e.op(f"s_cbranch_scc1 {narrow}f")
        e.wide = True
        step(stage, False, False, False, True, ["s_branch 4f"])
        e.label(narrow)
        e.wide = False
        step(stage, False, False, False, True, ["s_branch 4f"] if stage else [])
    e.label("4")
    return "\n".join(e.lines).replace("@WAIT@", str(min(63, *(w for w, _ in e.behind)))).replace("@BEHIND@", str(min(w for _, w in e.behind)))


# Loads of step j + 2 all go out in step j, so that they have the rest of it
# and the next step up to the publish barrier to land.
ROWS = {"rel": 12, "load_every": 6, "pub": 64, "a_delay": 1, "read_limit": 112, "f0_lat": 8, "epi_slot": 8, "epi_delay": 2, "nxt_start": 2}
MIXED = {**ROWS, "pub": 56}
COLS = {**ROWS, "rel": 14, "pub": 48}

LOOPS = {   # macro: A side, B side, schedule
    "G16_GROUPED_RR": ("r", "r", ROWS),
    "G16_GROUPED_RR2": ("r", "r", {**ROWS, "leads": 2}),
    "G16_GROUPED_RC": ("r", "c", MIXED),
    "G16_GROUPED_CC": ("c", "c", COLS),
}


def as_macro(name: str, text: str) -> str:
    body = []
    for ln in text.split("\n"):
        body.append('    "' + ln.replace("@T@", '" TYPE "') + '\\n"')
    return f"#define {name}(TYPE) \\\n" + " \\\n".join(body) + "\n"


def main() -> int:
    out = os.path.join(os.path.dirname(os.path.abspath(__file__)), "grouped_sched.inc")
    lines = 0
    with open(out, "w") as f:
        f.write("// Generated by gen_grouped_sched.py.  Do not edit.\n")
        for name, (la, lb, p) in LOOPS.items():
            text = generate(la, lb, p)
            lines += len(text.split("\n"))
            f.write(f"// {name}: {ring4.params_line(p)}.\n")
            f.write(as_macro(name, text))
    print(out, lines, "lines")
    return 0


if __name__ == "__main__":
    sys.exit(main())
