"""In-flight load registers: a check of the compiled kernels' gfx9 assembly.

The kernels issue most of their global loads as inline assembly and wait for
them with explicit `s_waitcnt vmcnt(N)`, so the compiler does not know a load
is still in flight.  If it copies, moves or reuses a destination register of
such a load before the wait that completes it (a live-range split into an
AGPR, a spill, a register reused for a temporary), the copy holds stale data
and the load later overwrites whatever the register holds then.  Neither is
visible in the compiler's resource-usage remarks: an AGPR copy is not a spill.

This module models the vector-memory counter over each kernel's control-flow
graph.  The pending loads are a queue, oldest first.  Every vector-memory
instruction (load, store, buffer-to-LDS copy) enters it; `s_waitcnt vmcnt(N)`
keeps only the newest N.  Where control flow merges, the queues are aligned at
their newest end and only what both hold is kept: the analysis finds what is
pending on every path (it reports no hazard that a path-insensitive merge
would invent, and may miss one that exists on some paths only).  An
instruction that names a register of a load still pending is reported, the
next load into that register included.

What lies between inline loads and the first explicit wait for them (an adapter
extension's loops, with loads of the compiler's own) is walked path by path as
well: check_kernel_paths.

It also checks the wait states of gfx9 that inline assembly has to keep by
itself: a vector-memory instruction that reads a scalar register (a buffer
descriptor, a scalar offset) must come at least five wait states after a vector
instruction wrote that register.  The compiler keeps them for its own
instructions and does not look into inline assembly, so a scalar register
reloaded from a lane of a vector register (v_readlane_b32) right before an
inline buffer load gives the load its old value: a wrong descriptor, and a
memory fault.  The same holds for a matrix instruction that reads a vector
register two wait states after the vector instruction that wrote it, where one
of the two is inline.
"""
from __future__ import annotations

import re
import subprocess
from typing import Dict, FrozenSet, List, Optional, Sequence, Tuple

_REG_RANGE = re.compile(r"^([va])\[(\d+):(\d+)\]")
_REG_ONE = re.compile(r"^([va])(\d+)\b")
_VMCNT = re.compile(r"vmcnt\((\d+)\)")
_LABEL = re.compile(r"^(\.?[\w.$]+):")
_FUNC = re.compile(r"^(_Z\w+):")
_MAX_PENDING = 63

Reg = Tuple[str, int]
Queue = Tuple[FrozenSet[Reg], ...]


def _regs(tok: str) -> FrozenSet[Reg]:
    tok = tok.strip()
    m = _REG_RANGE.match(tok)
    if m:
        return frozenset((m.group(1), k) for k in range(int(m.group(2)), int(m.group(3)) + 1))
    m = _REG_ONE.match(tok)
    if m:
        return frozenset({(m.group(1), int(m.group(2)))})
    return frozenset()


def _strip(line: str) -> str:
    for c in (";", "//"):
        k = line.find(c)
        if k >= 0:
            line = line[:k]
    return line.strip()


def _operands(text: str) -> List[FrozenSet[Reg]]:
    """Register sets of the comma-separated operands, in order (modifiers
    after an operand, such as `offen` or `op_sel:[...]`, name none)."""
    return [_regs(p.strip().split(" ")[0]) if p.strip() else frozenset() for p in text.split(",")]


class _Instr:
    __slots__ = ("text", "op", "ops", "line")

    def __init__(self, text: str, line: int):
        self.text = text
        self.line = line
        parts = text.split(None, 1)
        self.op = parts[0]
        self.ops = _operands(parts[1]) if len(parts) > 1 else []


def _is_vmem(op: str) -> bool:
    return op.startswith(("buffer_", "global_", "flat_", "scratch_")) and not op.startswith(
        ("buffer_wbl2", "buffer_inv", "buffer_wbinvl1", "buffer_gl"))


def _is_load(ins: _Instr) -> bool:
    return "_load" in ins.op and " lds" not in ins.text and not ins.text.rstrip().endswith("lds")


def _blocks(body: Sequence[Tuple[int, str]]):
    """Basic blocks: (label or None, [instr], successor labels, falls through)."""
    blocks = []
    cur_label, cur = None, []

    def close(succ, falls):
        blocks.append([cur_label, cur, succ, falls])

    for line_no, raw in body:
        s = _strip(raw)
        if not s or s.startswith("."):
            m = _LABEL.match(s) if s else None
            if m and s.endswith(":"):
                if cur or cur_label is not None:
                    close([], True)
                cur_label, cur = m.group(1), []
            continue
        m = _LABEL.match(s)
        if m and s.endswith(":"):
            if cur or cur_label is not None:
                close([], True)
            cur_label, cur = m.group(1), []
            continue
        ins = _Instr(s, line_no)
        cur.append(ins)
        if ins.op == "s_branch":
            close([s.split()[1]], False)
            cur_label, cur = None, []
        elif ins.op.startswith("s_cbranch_"):
            close([s.split()[1]], True)
            cur_label, cur = None, []
        elif ins.op in ("s_endpgm", "s_setpc_b64"):
            close([], False)
            cur_label, cur = None, []
    if cur or cur_label is not None:
        close([], False)
    return blocks


def _join(a: Optional[Queue], b: Queue) -> Queue:
    # what is pending on every path into the block: the queues aligned at
    # their newest end, the common length, the registers common to both
    if a is None:
        return b
    n = min(len(a), len(b))
    return tuple(a[len(a) - k] & b[len(b) - k] for k in range(n, 0, -1))


def _step(q: Queue, ins: _Instr, report) -> Queue:
    if ins.op == "s_waitcnt":
        m = _VMCNT.search(ins.text)
        if m:
            keep = int(m.group(1))
            q = q[len(q) - keep:] if keep and len(q) > keep else (q if keep else ())
        return q
    live = frozenset().union(*q) if q else frozenset()
    used = frozenset().union(*ins.ops) if ins.ops else frozenset()
    if used & live and report is not None:
        report(ins, sorted(used & live))
    if _is_vmem(ins.op):
        dst = ins.ops[0] if (_is_load(ins) and ins.ops) else frozenset()
        q = (q + (dst,))[-_MAX_PENDING:]
    return q


def _graph(body: Sequence[Tuple[int, str]]):
    """The kernel's basic blocks and each one's successors."""
    blocks = _blocks(body)
    index = {b[0]: i for i, b in enumerate(blocks) if b[0] is not None}
    succs = []
    for i, (_, _, targets, falls) in enumerate(blocks):
        s = [index[t] for t in targets if t in index]
        if falls and i + 1 < len(blocks):
            s.append(i + 1)
        succs.append(s)
    return blocks, succs


def check_kernel(body: Sequence[Tuple[int, str]]) -> List[Tuple[int, str, List[Reg]]]:
    """[(line, instruction, pending registers it names)] for one kernel."""
    blocks, succs = _graph(body)
    entry: List[Optional[Queue]] = [None] * len(blocks)
    if blocks:
        entry[0] = ()
    work = [0] if blocks else []
    while work:
        i = work.pop()
        q = entry[i]
        for ins in blocks[i][1]:
            q = _step(q, ins, None)
        for j in succs[i]:
            nq = _join(entry[j], q)
            if nq != entry[j]:
                entry[j] = nq
                work.append(j)
    found = []
    for i, blk in enumerate(blocks):
        q = entry[i]
        if q is None:
            continue
        for ins in blk[1]:
            q = _step(q, ins, lambda ins, regs: found.append((ins.line, ins.text, regs)))
    return found


# ---------------------------------------------------------------------------
# From an inline load to its first explicit wait, over every path.
#
# State: register -> the fewest vector-memory instructions issued after its
# inline load on any path (an implicit wait vmcnt(N), the compiler's, completes
# the load where that is at least N), or _WAITED once an inline wait or a
# barrier has been passed.  From then on the kernel's own counting rules, which
# check_kernel follows; where paths merge and one of them has waited, the merge
# counts as waited (the paths around a ring's loop that its trip count rules
# out would be reported otherwise).
#
# Two walks, and what both report is reported.  One merges at every block.  The
# other keeps paths apart by what they tell of the compiler's branch flags
# (scalar pairs set to 0 or -1, tested through vcc), which rule out most pairs
# of branches, and takes exec for nonzero where nothing narrowed it.
# ---------------------------------------------------------------------------
_WAITED = -1
PathState = Dict[Reg, int]
Facts = Dict[str, object]


def _inline_lines(body: Sequence[Tuple[int, str]]) -> FrozenSet[int]:
    """Numbers of the lines that inline assembly wrote."""
    lines, inside = set(), False
    for n, text in body:
        if "#ASMSTART" in text:
            inside = True
        elif "#ASMEND" in text:
            inside = False
        elif inside:
            lines.add(n)
    return frozenset(lines)


def _path_step(st: PathState, ins: _Instr, inline: FrozenSet[int], report) -> PathState:
    if ins.op == "s_barrier":
        return dict.fromkeys(st, _WAITED)
    if ins.op == "s_waitcnt":
        m = _VMCNT.search(ins.text)
        if m is None:
            return st
        if ins.line in inline:
            return dict.fromkeys(st, _WAITED)
        return {r: _WAITED if c >= int(m.group(1)) else c for r, c in st.items()}
    load = _is_vmem(ins.op) and _is_load(ins)
    own = load and ins.line in inline
    if report is not None:
        # (a ring's next inline load into a register is check_kernel's)
        named = [r for ops in (ins.ops[1:] if own else ins.ops) for r in ops if st.get(r, _WAITED) != _WAITED]
        if named:
            report(ins, sorted(set(named)))
    if _is_vmem(ins.op):
        st = {r: c if c == _WAITED else min(c + 1, _MAX_PENDING) for r, c in st.items()}
        for r in ins.ops[0] if load and ins.ops else ():
            if own:
                st[r] = 0
            else:
                st.pop(r, None)
    return st


def _path_join(old: Optional[PathState], new: PathState) -> PathState:
    if old is None:
        return dict(new)
    out = dict(old)
    for r, c in new.items():
        o = old.get(r)
        out[r] = c if o is None else _WAITED if _WAITED in (o, c) else min(o, c)
    return out


def _writes_exec(ins: _Instr) -> bool:
    return "saveexec" in ins.op or (ins.op.startswith(("s_", "v_cmpx")) and bool(_tokens(ins)[:1])
                                    and _tokens(ins)[0].startswith("exec"))


def _fact_step(facts: Facts, ins: _Instr) -> Facts:
    """facts: "s[a:b]" -> whether that pair is nonzero; "vcc" -> (True, value)
    or (False, pair, negated); "exec" -> True where it is nonzero for sure."""
    op, tok = ins.op, _tokens(ins)
    if _writes_exec(ins):
        facts = dict(facts)
        facts.pop("exec", None)
        if op in ("s_or_b64", "s_mov_b64"):    # (restored after a narrowed region)
            facts["exec"] = True
        if "saveexec" not in op:
            return facts
    scalar = op.startswith("s_") and not op.startswith(
        ("s_cbranch", "s_branch", "s_waitcnt", "s_barrier", "s_nop", "s_cmp", "s_bitcmp", "s_sleep", "s_setprio"))
    written = [tok[0]] if scalar and tok else []
    if op.startswith(("v_cmp", "v_readlane", "v_readfirstlane")) and tok:
        written = [tok[0]]
    elif op.startswith("v_") and ("_co_" in op or op.startswith(("v_div_scale", "v_mad_u64", "v_mad_i64"))):
        written = tok[1:2]
    if not written:
        return facts
    new = dict(facts)
    dst, regs = written[0], _sregs(written[0])
    value = None
    if scalar and op == "s_mov_b64" and len(tok) == 2:
        value = (True, tok[1] == "-1") if tok[1] in ("0", "-1") else (
            (True, new[tok[1]]) if tok[1] in new and tok[1] != "exec" else (False, tok[1], False))
    elif scalar and op in ("s_and_b64", "s_andn2_b64") and len(tok) == 3 and tok[1] == "exec" and _sregs(tok[2]):
        neg = op == "s_andn2_b64"
        value = (True, new[tok[2]] != neg) if tok[2] in new else (False, tok[2], neg)
    if dst.startswith("vcc"):
        new.pop("vcc", None)
        if value is not None and (value[0] or _sregs(value[1])):
            new["vcc"] = value
        return new
    for k in [k for k in new if _sregs(k) & regs]:
        del new[k]
    v = new.get("vcc")
    if v and not v[0] and _sregs(v[1]) & regs:
        del new["vcc"]
    if value is not None and value[0] and op == "s_mov_b64" and dst.startswith("s["):
        new[dst] = value[1]
    return new


def _live_scalars(blocks, succs):
    """Scalar registers and vcc read before they are written, at each block's
    start: what is worth keeping paths apart for."""
    def keys(tok):
        return {"vcc"} if tok.startswith("vcc") else set(_sregs(tok))

    use, kill = [], []
    for _, instrs, _, _ in blocks:
        u, d = set(), set()
        for ins in instrs:
            tok = _tokens(ins)
            reads_all = ins.op.startswith(("s_cmp", "s_bitcmp", "buffer_store", "global_store", "s_cbranch", "s_branch"))
            r = set().union(*[keys(t) for t in (tok if reads_all else tok[1:])]) if tok else set()
            if ins.op.startswith(("s_cbranch_vcc", "v_cndmask", "v_addc", "v_subb")):
                r.add("vcc")
            u |= r - d
            if tok and not reads_all:
                d |= keys(tok[0])
        use.append(u)
        kill.append(d)
    live = [set() for _ in blocks]
    changed = True
    while changed:
        changed = False
        for i in range(len(blocks) - 1, -1, -1):
            new = use[i] | (set().union(*[live[j] for j in succs[i]]) - kill[i] if succs[i] else set())
            if new != live[i]:
                live[i], changed = new, True
    return live


def _branches(blocks, index, i: int, facts: Facts):
    """(successor, facts on that edge) of block i for the facts at its end."""
    _, instrs, targets, falls = blocks[i]
    taken = [index[t] for t in targets if t in index]
    nxt = [i + 1] if falls and i + 1 < len(blocks) else []
    op = instrs[-1].op if instrs else ""
    if op in ("s_cbranch_vccnz", "s_cbranch_vccz") and "vcc" in facts:
        v, nz = facts["vcc"], op.endswith("nz")
        if v[0]:
            return [(j, facts) for j in (taken if v[1] == nz else nxt)]
        out = []
        for edge, value in ((taken, nz), (nxt, not nz)):
            f = dict(facts)
            f[v[1]], f["vcc"] = value != v[2], (True, value)
            out += [(j, f) for j in edge]
        return out
    if op in ("s_cbranch_execz", "s_cbranch_execnz"):
        zero, sure = op.endswith("execz"), bool(facts.get("exec"))
        nonzero = dict(facts, exec=True)
        none = {k: x for k, x in facts.items() if k != "exec"}
        out = []
        if not (zero and sure):
            out += [(j, none if zero else nonzero) for j in taken]
        if not (not zero and sure):
            out += [(j, nonzero if zero else none) for j in nxt]
        return out
    return [(j, facts) for j in taken + nxt]


def _walk_paths(body: Sequence[Tuple[int, str]], apart: bool) -> Dict[int, Tuple[int, str, List[Reg]]]:
    inline = _inline_lines(body)
    blocks, succs = _graph(body)
    if not blocks:
        return {}
    index = {b[0]: i for i, b in enumerate(blocks) if b[0] is not None}
    live = _live_scalars(blocks, succs) if apart else None

    def kept(facts: Facts, j: int, st: PathState) -> Facts:
        if not apart:    # (exec is judged within the block)
            return {"exec": True}
        return {k: x for k, x in facts.items()
                if k == "exec" or (st and ("vcc" in live[j] if k == "vcc" else _sregs(k) <= live[j]))}

    start = (0, frozenset({("exec", True)}))
    entry: Dict[tuple, PathState] = {start: {}}
    work = [start]
    while work:
        key = work.pop()
        st, facts = entry[key], dict(key[1])
        for ins in blocks[key[0]][1]:
            st, facts = _path_step(st, ins, inline, None), _fact_step(facts, ins)
        for j, f in _branches(blocks, index, key[0], facts):
            to = (j, frozenset(kept(f, j, st).items()))
            new = _path_join(entry.get(to), st)
            if new != entry.get(to):
                entry[to] = new
                work.append(to)
    found: Dict[int, Tuple[int, str, List[Reg]]] = {}
    for (i, _), st in entry.items():
        for ins in blocks[i][1]:
            st = _path_step(st, ins, inline, lambda ins, regs: found.setdefault(ins.line, (ins.line, ins.text, regs)))
    return found


def check_kernel_paths(body: Sequence[Tuple[int, str]]) -> List[Tuple[int, str, List[Reg]]]:
    """[(line, instruction, registers of inline loads that it names before the
    first explicit wait for them)] for one kernel."""
    merged = _walk_paths(body, False)
    if not merged:
        return []
    apart = _walk_paths(body, True)
    return [merged[n] for n in sorted(merged) if n in apart]


_SREG_RANGE = re.compile(r"^s\[(\d+):(\d+)\]$")
_SREG_ONE = re.compile(r"^s(\d+)$")
_VMEM_SGPR_WAIT_STATES = 5


def _sregs(tok: str) -> FrozenSet[int]:
    m = _SREG_RANGE.match(tok)
    if m:
        return frozenset(range(int(m.group(1)), int(m.group(2)) + 1))
    m = _SREG_ONE.match(tok)
    return frozenset({int(m.group(1))}) if m else frozenset()


def _tokens(ins: _Instr) -> List[str]:
    parts = ins.text.split(None, 1)
    return [t.strip().split(" ")[0] for t in parts[1].split(",")] if len(parts) > 1 else []


def _valu_sgpr_writes(ins: _Instr) -> FrozenSet[int]:
    """Scalar registers a vector instruction writes: the destination of a lane
    read or of a compare, and the carry-out of an addition."""
    if ins.op.startswith(("v_readlane", "v_readfirstlane", "v_cmp")):
        return _sregs(_tokens(ins)[0])
    if ins.op.startswith(("v_div_scale", "v_mad_u64", "v_mad_i64")) or (ins.op.startswith("v_") and "_co_" in ins.op):
        return _sregs(_tokens(ins)[1])
    return frozenset()


def _sgpr_step(state: Dict[int, int], ins: _Instr, report) -> Dict[int, int]:
    """state: scalar register -> wait states since a vector instruction wrote it
    (below five)."""
    if state and _is_vmem(ins.op) and report is not None:
        early = sorted(r for t in _tokens(ins) for r in _sregs(t) if r in state)
        if early:
            report(ins, [("s", r) for r in early])
    n = int(ins.text.split()[1], 0) + 1 if ins.op == "s_nop" else 1
    state = {r: k + n for r, k in state.items() if k + n < _VMEM_SGPR_WAIT_STATES}
    if ins.op.startswith("s_"):
        tok = _tokens(ins)
        for r in (_sregs(tok[0]) if tok else ()):
            state.pop(r, None)
    for r in _valu_sgpr_writes(ins):
        state[r] = 0
    return state


_MFMA_VGPR_WAIT_STATES = 2


def _mfma_step(state: Dict[Reg, int], ins: _Instr, report) -> Dict[Reg, int]:
    """state: vector register -> wait states since a vector instruction (no matrix
    instruction) wrote it (below two)."""
    mfma = ins.op.startswith("v_mfma")
    if state and mfma and report is not None:
        early = sorted({r for ops in ins.ops[1:] for r in ops if r in state})
        if early:
            report(ins, early)
    n = int(ins.text.split()[1], 0) + 1 if ins.op == "s_nop" else 1
    state = {r: k + n for r, k in state.items() if k + n < _MFMA_VGPR_WAIT_STATES}
    if ins.op.startswith("v_") and not mfma and ins.ops:
        for r in ins.ops[0]:
            state[r] = 0
    return state


def _check_wait_states(body: Sequence[Tuple[int, str]], step) -> List[Tuple[int, str, List[Reg]]]:
    """What `step` reports, over every path (the fewest wait states of the paths
    that merge)."""
    blocks, succs = _graph(body)
    entry: List[Optional[dict]] = [None] * len(blocks)
    if blocks:
        entry[0] = {}
    work = [0] if blocks else []
    while work:
        i = work.pop()
        q = dict(entry[i])
        for ins in blocks[i][1]:
            q = step(q, ins, None)
        for j in succs[i]:
            old = entry[j]
            new = dict(q) if old is None else {r: min(q.get(r, 9), old.get(r, 9)) for r in q.keys() | old.keys()}
            if new != old:
                entry[j] = new
                work.append(j)
    found = []
    for i, blk in enumerate(blocks):
        q = entry[i]
        if q is None:
            continue
        for ins in blk[1]:
            q = step(q, ins, lambda ins, regs: found.append((ins.line, ins.text, regs)))
    return found


def check_kernel_sgprs(body: Sequence[Tuple[int, str]]) -> List[Tuple[int, str, List[Reg]]]:
    """[(line, vector-memory instruction, scalar registers it reads too early)]."""
    return _check_wait_states(body, _sgpr_step)


def check_kernel_mfma(body: Sequence[Tuple[int, str]]) -> List[Tuple[int, str, List[Reg]]]:
    """[(line, matrix instruction, vector registers it reads too early)]: one of the
    two instructions is inline, as the compiler keeps the distance of its own."""
    return _check_wait_states(body, _mfma_step)


def kernels(asm: str) -> Dict[str, List[Tuple[int, str]]]:
    """Kernel name -> its (line number, text) lines, from a device assembly file."""
    lines = asm.split("\n")
    out, i = {}, 0
    while i < len(lines):
        m = _FUNC.match(lines[i])
        if not m:
            i += 1
            continue
        j = i + 1
        while j < len(lines) and not lines[j].strip().startswith(".Lfunc_end"):
            j += 1
        out[m.group(1)] = [(k + 1, lines[k]) for k in range(i + 1, j)]
        i = j
    return out


def check_asm(asm: str) -> Dict[str, List[Tuple[int, str, List[Reg]]]]:
    return {name: f for name, body in kernels(asm).items() for f in [check_kernel(body)] if f}


def check_asm_paths(asm: str) -> Dict[str, List[Tuple[int, str, List[Reg]]]]:
    return {name: f for name, body in kernels(asm).items() for f in [check_kernel_paths(body)] if f}


def check_asm_sgprs(asm: str) -> Dict[str, List[Tuple[int, str, List[Reg]]]]:
    return {name: f for name, body in kernels(asm).items() for f in [check_kernel_sgprs(body)] if f}


def check_asm_mfma(asm: str) -> Dict[str, List[Tuple[int, str, List[Reg]]]]:
    return {name: f for name, body in kernels(asm).items() for f in [check_kernel_mfma(body)] if f}


def demangle(name: str) -> str:
    try:
        return subprocess.run(["c++filt", name], capture_output=True, text=True).stdout.strip() or name
    except OSError:
        return name


if __name__ == "__main__":
    import sys

    bad = 0
    for path in sys.argv[1:]:
        text = open(path).read()
        for check, what in ((check_asm, "name registers of loads that may be in flight"),
                            (check_asm_paths, "name registers of loads before the first wait for them"),
                            (check_asm_sgprs, "read scalar registers too soon after a vector write"),
                            (check_asm_mfma, "are MFMAs that read registers too soon after a vector write")):
            for name, found in check(text).items():
                bad += 1
                print(f"{path}: {demangle(name)}: {len(found)} instructions {what}, "
                      f"first: line {found[0][0]} {found[0][1]!r} {found[0][2][:4]}")
    sys.exit(1 if bad else 0)
