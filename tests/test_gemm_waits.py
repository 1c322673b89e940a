"""The tiled GEMM's stage barriers in the compiled code: when a wave reaches the barrier of
stage s, its own copies of stage s into LDS must have landed, whatever order the compiler
gave the loads around them (a counted wait covers a copy only while enough younger loads
follow it).  The kernels' control flow is walked from the entry over every branch; vector
loads complete in order, so the state is the queue of loads in flight: a load appends, a
wait for n drops all but the n youngest."""
import os
import re
import subprocess

import pytest

from tenant_serving_amd import build

KERNEL = re.compile(r"^_ZN2bd6k_gemmILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELb([01])E\w*:")
STAGES = 9  # barriers walked: past the ring's first turn for every ring length


def kernels(text):
    """{template arguments: [(op, argument)]} of the instructions that matter."""
    out, cur = {}, None
    for line in text.splitlines():
        m = KERNEL.match(line)
        if m:
            cur = out.setdefault(tuple(int(v) for v in m.groups()), [])
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


def unlanded(code, per_stage):
    """(stage, copies of stages up to it still in flight) at the first barrier that finds
    any, None if none does."""
    at = {arg: i for i, (op, arg) in enumerate(code) if op == "label"}
    todo, seen = [(0, 0, 0, ())], set()  # pc, barriers passed, copies sent, loads in flight
    while todo:
        pc, stage, sent, flight = todo.pop()
        while pc < len(code) and stage < STAGES:
            if (pc, stage, sent, flight) in seen:
                break
            seen.add((pc, stage, sent, flight))
            op, arg = code[pc]
            pc += 1
            if op == "copy":
                flight += (sent,)
                sent += 1
            elif op == "mem":
                flight += (-1,)
            elif op == "wait":
                flight = flight[len(flight) - arg:] if arg and len(flight) > arg else flight if arg else ()
            elif op == "barrier":
                late = [c for c in flight if 0 <= c < (stage + 1) * per_stage]
                if late:
                    return stage, late
                stage += 1
            elif op == "cbranch":
                todo.append((at[arg], stage, sent, flight))
            elif op == "branch":
                pc = at[arg]
            elif op == "end":
                break
    assert any(s == STAGES - 1 for _, s, _, _ in seen), "no path over the stages was found"
    return None


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no HIP compiler")
def test_copies_of_a_stage_land_before_its_barrier(tmp_path):
    asm = tmp_path / "bd_gemm.s"
    subprocess.run([build.HIPCC] + build.HIP_FLAGS +
                   ["--offload-device-only", "-S", os.path.join(build.CSRC, "bd_gemm.hip"), "-o", str(asm)],
                   check=True, capture_output=True)
    found = kernels(asm.read_text())
    assert sum(k[5] for k in found) == 5 and len(found) == 10  # the INT8 and the bf16 tiles
    bad = {}
    for (br, bt, bk, ns, nw, q8), code in found.items():
        copies = bt * bk * 2 // 1024 // nw + (0 if q8 else br * bk * 2 // 1024 // nw)
        late = unlanded(code, copies)
        if late:
            bad[f"{br}x{bt}{' int8' if q8 else ''}"] = late
    assert not bad, f"(stage, copies in flight at its barrier): {bad}"
