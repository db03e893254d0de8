"""The LDS ring of `Shared` (csrc/mxfp4_device.hpp): before any wave reads a
stage's activations, every wave has waited for its own transfers of them.

A wave's loads complete in the order of issue, so the hand-written
`s_waitcnt vmcnt(n)` before the barrier leaves at most the n newest in flight;
n counts the loads of the stages issued after the one to be read.  The count is
wrong if the compiler drops a load that the source has.  Here the sources are
compiled for gfx950 and the load queue is followed through every path of every
kernel, with the hand-written waits alone: waits that the compiler adds for
registers are not counted on.

The waits carry the number of a stage's transfers as an assembly comment
("; stage of n transfers"), the drained wait after the last stage
"; end of stages"."""
import importlib.util
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MEMORY = re.compile(r"(buffer|global|flat|scratch)_(load|store|atomic)")
COUNTER = 63  # vmcnt's range: no more are ever in flight


def assembly(source):
    spec = importlib.util.spec_from_file_location(
        "_dg_build", os.path.join(ROOT, "fp8_block_scaled_dg_amd", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    r = subprocess.run([b.HIPCC, *b.CFLAGS, "-x", "hip", "--offload-device-only", "-S",
                        source if os.path.isabs(source) else os.path.join(b.CSRC, source), "-o", "-"],
                       capture_output=True, text=True, check=True)
    return r.stdout


def kernels(text):
    """name -> its blocks (label, instructions): instructions are ("load",),
    ("transfer",), ("wait", n, transfers or 0), ("jump", label), ("branch",
    label) or ("end",)."""
    found = {}
    for m in re.finditer(r"^(_Z\w+):\s*; @\1\n(.*?)^\.Lfunc_end", text, re.M | re.S):
        blocks, hand, wait = [("", [])], False, None
        for line in m.group(2).splitlines():
            code = line.strip()
            label = re.match(r"(\.LBB\w+):", code)
            if label:
                blocks.append((label.group(1), []))
            elif code.startswith(";;#ASMSTART"):
                hand = True
            elif code.startswith(";;#ASMEND"):
                hand = False
            out = blocks[-1][1]
            op = code.split()[0] if code else ""
            if MEMORY.match(op):
                out.append(("transfer",) if re.search(r"\blds\b", code) else ("load",))
            elif op.startswith("s_cbranch"):
                out.append(("branch", code.split()[1]))
            elif op == "s_branch":
                out.append(("jump", code.split()[1]))
            elif op == "s_endpgm":
                out.append(("end",))
            assert op not in ("s_setpc_b64", "s_swappc_b64")
            if hand:
                n = re.search(r"s_waitcnt vmcnt\((\d+)\)", code)
                wait = int(n.group(1)) if n else wait
                stage = re.search(r"; stage of (\d+) transfers", code)
                if stage:
                    out.append(("wait", wait, int(stage.group(1))))
                elif "; end of stages" in code:
                    out.append(("wait", wait, 0))
        found[m.group(1)] = blocks
    return found


def follow(blocks):
    """(waits met, faults).  The queue holds, oldest first, -1 for a load into
    registers and otherwise the number of a transfer, counted from the first one
    of the stage that the next wait is for; loads older than every such transfer
    do not matter and are left out."""
    index = {label: i for i, (label, _) in enumerate(blocks)}
    seen, work, waits, faults = set(), [(0, (), 0)], set(), set()
    while work:
        state = work.pop()
        if state in seen:
            continue
        seen.add(state)
        assert len(seen) < 100000, "transfers without a wait for their stage"
        at, queue, count = state
        queue = list(queue)
        ended = False
        for ins in blocks[at][1]:
            if ins[0] == "load":
                if queue:
                    queue.append(-1)
            elif ins[0] == "transfer":
                queue.append(count)
                count += 1
            elif ins[0] == "wait":
                _, n, per = ins
                waits.add(ins)
                flying = queue[len(queue) - n:] if n < len(queue) else queue
                if per and any(0 <= q < per for q in flying):
                    faults.add((blocks[at][0], ins))
                if per:  # the next stage's turn
                    queue = [max(q - per, -1) for q in flying]
                    count = max(count - per, 0)
                else:
                    queue, count = [], 0
                while queue and queue[0] < 0:
                    queue.pop(0)
            elif ins[0] == "branch":
                work.append((index[ins[1]], tuple(queue), count))
            elif ins[0] == "jump":
                work.append((index[ins[1]], tuple(queue), count))
                ended = True
                break
            elif ins[0] == "end":
                ended = True
                break
            queue = queue[-COUNTER:]
        if not ended and at + 1 < len(blocks):
            work.append((at + 1, tuple(queue), count))
    return waits, faults


@pytest.mark.parametrize("source,expect", [("gemm_mxfp4.hip", 3), ("moe_layer.hip", 9)])
def test_every_stage_has_landed_before_it_is_read(source, expect):
    with_stages = 0
    for name, blocks in kernels(assembly(source)).items():
        if not any(ins[0] == "wait" for _, code in blocks for ins in code):
            continue
        waits, faults = follow(blocks)
        assert not faults, (name, sorted(faults))
        with_stages += any(w[2] for w in waits)
    assert with_stages == expect


def test_the_check_finds_a_short_wait():
    """A ring of three stages, each of one transfer and one register load: two
    loads may be in flight when a stage is read, and one where the loop's
    register loads are dropped."""
    def ring(tail_wait):
        return [("", [("transfer",), ("load",), ("transfer",), ("load",)]),
                ("loop", [("wait", 2, 1), ("transfer",), ("load",), ("branch", "loop")]),
                ("t0", [("wait", tail_wait, 1)]), ("t1", [("wait", 0, 1)]),
                ("out", [("wait", 0, 0), ("end",)])]
    assert not follow(ring(2))[1]
    assert follow(ring(4))[1]
    dropped = ring(2)
    dropped[1] = ("loop", [("wait", 2, 1), ("transfer",), ("branch", "loop")])
    assert follow(dropped)[1]
