"""Static check of the gfx950 assembly the compiler emits for the kernels.

An MFMA that takes its accumulator (srcC) from the result of a recently
issued MFMA of a *different* opcode (for example a 16x16x16 accumulating onto a
16x16x32 result) reads stale data on gfx950 unless enough independent work
separates the two, and the compiler inserts no wait states for that case.
The kernels therefore never chain accumulators across MFMA shapes; this check
scans the emitted assembly and reports every place where such a chain appears
within `window` wait states, so the build fails instead of the numerics.

The compiler may also place a copy of a vector register, made where registers
run short, between the masked half of a lane-dependent branch and the
instruction that turns to the other lanes.  Lanes of the other half then miss
the copy and read what was in the register before.  No vector register is
written at that place in a right program of these kernels, so the check
reports every one that is.
"""
from __future__ import annotations

import re

_RANGE = re.compile(r"^([va])\[(\d+):(\d+)\]$")
_SINGLE = re.compile(r"^([va])(\d+)$")
_FUNC = re.compile(r"^([A-Za-z_][\w.$]*):\s*(;.*)?$")


def _regs(tok: str) -> frozenset:
    tok = tok.strip().split()[0] if tok.strip() else ""
    m = _RANGE.match(tok)
    if m:
        base = 0 if m.group(1) == "v" else 1 << 16
        return frozenset(range(base + int(m.group(2)), base + int(m.group(3)) + 1))
    m = _SINGLE.match(tok)
    if m:
        base = 0 if m.group(1) == "v" else 1 << 16
        return frozenset([base + int(m.group(2))])
    return frozenset()


_NO_VDST = ("ds_write", "ds_store", "global_store", "buffer_store", "flat_store",
            "scratch_store", "s_", "v_cmp", "v_readlane", "v_readfirstlane")


def mixed_mfma_chains(asm: str, window: int = 32):
    """Returns [(function, line_no, producer_text, consumer_text, distance)].

    `window` is in wait states (instruction issues, s_nop N counting N+1); an
    accumulator written by another instruction in between no longer counts."""
    hits = []
    func = "?"
    recent = []          # (wait_states_at_issue, opcode, dst regs, text, line)
    ws = 0
    for no, raw in enumerate(asm.split("\n"), 1):
        t = raw.strip()
        if not t or t.startswith(";") or t.startswith("."):
            continue
        fm = _FUNC.match(t)
        if fm:
            if not t.startswith(".L") and not t.startswith("$"):
                func, recent, ws = fm.group(1), [], 0
            continue
        parts = t.split(None, 1)
        op = parts[0]
        if op == "s_nop":
            try:
                ws += int(parts[1].split()[0], 0) + 1
            except (IndexError, ValueError):
                ws += 1
            continue
        if op.startswith("v_mfma"):
            ops = [x.strip() for x in parts[1].split(",")] if len(parts) > 1 else []
            dst = _regs(ops[0]) if ops else frozenset()
            srcc = _regs(ops[3]) if len(ops) > 3 else frozenset()
            for (w0, op0, d0, txt0, _) in recent:
                if ws - w0 < window and op0 != op and (srcc & d0):
                    hits.append((func, no, txt0, t, ws - w0))
            recent = [(r[0], r[1], r[2] - dst, r[3], r[4]) for r in recent
                      if ws - r[0] < window and r[2] - dst]
            recent.append((ws, op, dst, t, no))
        elif recent and len(parts) > 1 and not op.startswith(_NO_VDST):
            w = _regs(parts[1].split(",")[0])
            if w:
                recent = [(r[0], r[1], r[2] - w, r[3], r[4]) for r in recent if r[2] - w]
        ws += 1
    return hits


_BLOCK = re.compile(r"^(\.LBB\d+_\d+:|; %bb\.\d+:)")


def masked_copies(asm: str):
    """Vector registers written in a block before the s_andn2_saveexec or s_or_saveexec that turns to a branch's other
    lanes: [(function, line_no, text)].  Writes of single lanes take no notice of the mask and pass."""
    hits, func, block = [], "?", []
    for no, raw in enumerate(asm.split("\n"), 1):
        t = raw.strip()
        fm = _FUNC.match(t)
        if fm and not t.startswith((".L", "$")):
            func, block = fm.group(1), []
        elif _BLOCK.match(t):
            block = []
        elif t.startswith(("s_andn2_saveexec", "s_or_saveexec")):
            hits += block
            block = []
        elif t.startswith(("v_", "ds_read", "scratch_load", "global_load", "buffer_load")) and \
                not t.startswith(("v_writelane", "v_readlane", "v_readfirstlane", "v_cmp")):
            block.append((func, no, t))
    return hits


def check_file(path: str, window: int = 32):
    with open(path) as f:
        return mixed_mfma_chains(f.read(), window)
