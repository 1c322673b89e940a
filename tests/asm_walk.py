"""Walks a kernel's compiled control flow with the queue of its vector loads in flight:
loads complete in order, so a load appends to the queue and a wait for n drops all but the
n youngest.  A counted wait covers a copy into LDS only while enough younger loads follow
it, and the compiler may move register loads; this looks at the order it chose."""
import os
import re
import subprocess

from tenant_serving_amd import build


def assembly(source, out_dir):
    out = os.path.join(str(out_dir), source + ".s")
    subprocess.run([build.HIPCC] + build.HIP_FLAGS +
                   ["--offload-device-only", "-S", os.path.join(build.CSRC, source), "-o", out],
                   check=True, capture_output=True)
    with open(out) as f:
        return f.read()


def kernels(text, name):
    """{template arguments: [(op, argument)]} of the kernel template bd::name: the
    instructions that matter to the queue."""
    head = re.compile(r"^_ZN2bd%d%sI((?:L[ib]\d+E)+)E\w*:" % (len(name), name))
    out, cur = {}, None
    for line in text.splitlines():
        m = head.match(line)
        if m:
            cur = out.setdefault(tuple(int(v) for v in re.findall(r"L[ib](\d+)E", m.group(1))), [])
            continue
        if line.startswith(".Lfunc_end"):
            cur = None
        if cur is None:
            continue
        ins = line.split(";")[0].strip()
        if ins.startswith(".LBB") and ins.endswith(":"):
            cur.append(("label", ins[:-1]))
        elif ins.startswith("s_cbranch"):
            cur.append(("cbranch", ins.split()[1]))
        elif ins.startswith("s_branch"):
            cur.append(("branch", ins.split()[1]))
        elif ins.startswith("s_endpgm"):
            cur.append(("end", None))
        elif ins.startswith("s_barrier"):
            cur.append(("barrier", None))
        elif ins.startswith("s_waitcnt"):
            n = re.search(r"vmcnt\((\d+)\)", ins)
            if n:
                cur.append(("wait", int(n.group(1))))
        elif re.match(r"(buffer|global|flat|scratch)_(load|store|atomic)", ins):
            cur.append(("copy" if re.search(r"\blds\b", ins) else "mem", None))
    return out


def unlanded(code, first_use, barriers, turn=0):
    """first_use[c]: the barrier behind which the kernel's c-th copy into LDS is first read.
    Returns (barrier, its copies still in flight) for a path over the first `barriers` of
    them that reaches one with any, None if no path does.  turn: barriers in a turn of the
    loop, where one more stands before it; a path then has to pass each of them once a turn
    (one that skips stages of a turn and yet takes another is none the kernel can take)."""
    at = {arg: i for i, (op, arg) in enumerate(code) if op == "label"}
    # pc, copies sent, loads in flight, barriers passed, what was late, the turn's barriers
    todo, seen, reached = [(0, 0, (), 0, None, ())], set(), False
    while todo:
        state = todo.pop()
        pc, sent, flight, bar, late, trail = state
        while pc < len(code) and (pc, sent, flight, bar, late, trail) not in seen:
            seen.add((pc, sent, flight, bar, late, trail))
            op, arg = code[pc]
            pc += 1
            if op == "copy":
                flight += (sent,)
                sent += 1
            elif op == "mem":
                flight += (-1,)
            elif op == "wait":
                flight = flight[-arg:] if arg else ()
            elif op == "barrier":
                if turn and bar:
                    trail = trail if len(trail) < turn else ()
                    if pc in trail:
                        break
                    trail += (pc,)
                open_ = tuple(c for c in flight if c >= 0 and first_use[c] <= bar)
                late = late or (open_ and (bar, open_)) or None
                bar += 1
                if bar == barriers:
                    if late:
                        return late
                    reached = True
                    break
            elif op == "cbranch":
                todo.append((at[arg], sent, flight, bar, late, trail))
            elif op == "branch":
                pc = at[arg]
            elif op == "end":
                break
    assert reached, "no path over the stages was found"
    return None
