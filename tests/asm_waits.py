"""Static check of the gfx950 assembly of the library's kernels for wait states
that inline assembly has to bring itself.

A vector-memory instruction may read a scalar register only 5 wait states after a
vector instruction wrote it (v_readlane, v_readfirstlane, a comparison, a carry), or it
may go to the address that the register held before.  And M0 may be read by a copy
from memory to LDS only 1 wait state after it was written.  The compiler keeps
both for the instructions that it knows, not for those in an asm statement.

`short_waits(asm_text)` lists every instruction that comes too soon on some way
through its function, branches and loops included.  An instruction is a wait state, s_nop n is
n + 1 of them.

Host-side test tooling only: the kernels never use it.
"""
import re

NEED, NEED_M0 = 5, 1
_SREG = re.compile(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b|\b(vcc|m0)\b")
_VMEM = ("global_", "buffer_", "scratch_", "flat_")
_TWO_RESULTS = re.compile(r"v_(add|addc|sub|subb|subrev|subbrev)_co_|v_div_scale_|v_mad_[ui]64_")


def _sregs(tok):
    out = set()
    for m in _SREG.finditer(tok):
        if m.group(1):
            out |= set(range(int(m.group(1)), int(m.group(2)) + 1))
        else:
            out.add(int(m.group(3)) if m.group(3) else m.group(4))
    return out


def _instructions(lines):
    """[(line number, text)] and label -> index of the instruction behind it."""
    code, at = [], {}
    for no, ln in lines:
        s = re.split(r"\s(?:;|//)", " " + ln, maxsplit=1)[0].strip()
        if s.endswith(":"):
            at[s[:-1]] = len(code)
        elif s and not s.startswith((";", ".", "//")):
            code.append((no, s))
    return code, at


def _short(lines):
    code, labels = _instructions(lines)
    most = max(NEED, NEED_M0)
    before = [None] * len(code)  # register -> wait states since its write, the fewest of all ways here
    found = {}
    todo = [(0, {})] if code else []
    while todo:
        i, state = todo.pop()
        while i < len(code):
            old = before[i]
            if old is not None:
                merged = {r: min(state.get(r, most), old.get(r, most)) for r in state.keys() | old.keys()}
                if merged == old:
                    break
                state = merged
            before[i] = dict(state)
            no, s = code[i]
            op = s.split()[0]
            args = [a.strip() for a in s[len(op):].split(",")]
            if op.startswith(_VMEM):
                reads = set().union(*map(_sregs, args))
                soonest = min(reads - {"m0"}, key=lambda r: state.get(r, most), default=None)
                if state.get(soonest, most) < NEED:
                    found[no] = (s, soonest, state[soonest], NEED)
                elif "_lds" in op and state.get("m0", most) < NEED_M0:
                    found[no] = (s, "m0", state["m0"], NEED_M0)
            passed = int(args[0], 0) + 1 if op == "s_nop" else 1
            state = {r: n + passed for r, n in state.items() if n + passed < most}
            if op.startswith("v_"):
                results = args[:2] if _TWO_RESULTS.match(op) else args[:1]
                for r in set().union(*map(_sregs, results)):
                    state[r] = 0
                if op.startswith("v_cmp") and op.endswith("_e32"):
                    state["vcc"] = 0
            elif op.startswith("s_") and "m0" in _sregs(args[0]):
                state["m0"] = 0
            if op.startswith(("s_branch", "s_cbranch")):
                to = labels.get(args[0])
                if to is not None:
                    todo.append((to, state))
            if op in ("s_branch", "s_endpgm", "s_setpc_b64", "s_trap"):
                break
            i += 1
    return [(no, *x) for no, x in sorted(found.items())]


def short_waits(asm_text):
    """[(function, line number, instruction, register, wait states, needed)]"""
    out, name, cur = [], None, []
    for i, ln in enumerate(asm_text.splitlines(), 1):
        m = re.match(r"^(_Z\S+):", ln)
        if m:
            if name:
                out += [(name, *f) for f in _short(cur)]
            name, cur = m.group(1), []
        elif name:
            cur.append((i, ln))
            if ln.strip().startswith(".Lfunc_end"):
                out += [(name, *f) for f in _short(cur)]
                name, cur = None, []
    if name:
        out += [(name, *f) for f in _short(cur)]
    return out
