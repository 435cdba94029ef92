"""CPU model of the MXFP4 GEMM's counted waits (no GPU; hipcc cross-compiles).

The kernels copy stages of both matrices straight into LDS and wait with
`s_waitcnt vmcnt(N)`: N of a wave's memory operations, the last ones it issued,
may still be on their way.  What a wave reads from LDS between barriers k and k + 1 is
stage k, copied by all waves, so at the wait in front of barrier k none of the N may be
a copy of stage k or of one before.
Scale fetches are such operations too: a wait that leaves room for one is right only
if the compiler kept the fetch behind the copies of its stage.

A stage's copies go to the place of the stage RING before it, which every wave has read
when it comes to the barrier behind that stage; they must not be issued before it.

The kernels are compiled to assembly with the library's flags, and with other
instruction schedulers as well, because an order that the source does not pin holds in
one build only by chance; the operations, waits and barriers along every path through
the stages are then replayed.
"""
import os
import re
import shutil
import subprocess

import pytest

from q8_quantized_matmul_amd import build

NAME = re.compile(r"gemm_kernelILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d)E")
SCHEDULERS = [None, "ilpmin", "gcn-max-ilp", "gcn-iterative-minreg"]


def _assembly(scheduler, out):
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-Wall")]
    if scheduler:
        flags += ["-mllvm", "-misched=" + scheduler]
    cmd = [build.hipcc(), *flags, "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"),
           "--cuda-device-only", "-S", "-o", str(out), os.path.join(build.CSRC, "mxfp4_gemm.hip")]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    return out.read_text()


def _events(lines):
    """copy, load, read (of LDS), barrier, and the counts of waits, in order."""
    out = []
    for line in lines:
        op = line.split(None, 1)[0] if line.split() else ""
        if op.startswith(("global_load_lds", "buffer_load")) and "lds" in line:
            out.append("copy")
        elif op.startswith(("global_", "buffer_", "flat_", "scratch_")):
            out.append("load")
        elif op.startswith("ds_read"):
            out.append("read")
        elif op == "s_barrier":
            out.append("barrier")
        elif op == "s_waitcnt":
            m = re.search(r"vmcnt\((\d+)\)", line)
            if m:
                out.append(int(m.group(1)))
    return out


def _paths(body):
    """The operations up to the loop over groups of four stages, in it, and behind it up
    to the barrier that ends the last stage."""
    loops = [(i, m.group(1)) for i, line in enumerate(body)
             if (m := re.match(r"(\.L\w+):.*Inner Loop Header: Depth=1", line))]
    spans = []
    for first, label in loops:
        last = max(i for i, line in enumerate(body) if re.search(r"s_c?branch\w*\s+%s\b" % re.escape(label), line))
        if any("v_mfma" in line for line in body[first:last]):
            spans.append((first, last))
    assert len(spans) == 1, spans
    first, last = spans[0]
    rest = _events(body[last + 1:])
    # Behind the loop: the stages taken alone, then a barrier behind a wait for everything,
    # from which on there are no copies.
    copies = [i for i, e in enumerate(rest) if e == "copy"]
    tail = rest[:copies[-1] + 1] if copies else []
    return _events(body[:first]), _events(body[first:last + 1]), tail


def _check(events, copies_a_stage, ring, where):
    """Replays a wave's operations: reads behind barrier k find stages 0..k landed at it,
    and copies of stage k + ring stand behind barrier k + 1."""
    queue, issued, landed, at_barrier, stage = [], 0, 0, 0, 0
    for e in events:
        if e in ("copy", "load"):
            queue.append(e)
            if e == "copy":
                of = issued // copies_a_stage
                assert of < ring or stage >= of - ring + 2, f"{where}: copy of stage {of} behind barrier {stage - 1}"
                issued += 1
        elif e == "barrier":
            at_barrier, stage = landed, stage + 1
        elif e == "read":
            assert stage > 0, f"{where}: LDS read in front of the first barrier"
            assert at_barrier >= stage * copies_a_stage, (
                f"{where}: {at_barrier} copies landed at barrier {stage - 1}, {stage * copies_a_stage} needed")
        else:
            while len(queue) > e:
                landed += queue.pop(0) == "copy"
    return stage


@pytest.mark.skipif(shutil.which(build.hipcc()) is None and not os.path.exists(build.hipcc()),
                    reason="hipcc not available")
@pytest.mark.parametrize("scheduler", SCHEDULERS)
def test_a_stage_has_landed_at_its_barrier(scheduler, tmp_path):
    text = _assembly(scheduler, tmp_path / "gemm.s")
    bodies = re.findall(r"^(\S*gemm_kernel\S*):[^\n]*\n(.*?)s_endpgm", text, re.S | re.M)
    kernels = {}
    for name, body in bodies:
        kernels[tuple(int(v) for v in NAME.search(name).groups())] = [line.strip() for line in body.splitlines()]
    assert len(kernels) == 12, sorted(kernels)  # four tiles, three output types
    for (wm, wn, tm, tn, ring, typ), body in kernels.items():
        where = f"{32 * tm * wm}x{32 * tn * wn} tile, type {typ}, scheduler {scheduler}"
        copies = 32 * (tm * wm + tn * wn) // 8 // (wm * wn)
        front, loop, tail = _paths(body)
        assert front.count("copy") == ring * copies and front.count("barrier") == 1, where
        assert loop.count("copy") == 4 * copies and loop.count("barrier") == 4, where
        assert tail.count("copy") == (2 * copies if tm * tn <= 4 else 0), where
        for times in range(4):
            stages = _check(front + times * loop + tail, copies, ring, where)
            assert stages == 1 + 4 * times + tail.count("barrier")


def test_the_model_sees_a_fetch_in_front_of_its_copies():
    """Two places, two copies a stage, a wait that leaves room for one fetch."""
    front = ["copy"] * 4 + [2, "barrier"]
    good = [0, "barrier", "read", "copy", "copy", "load", 1, "barrier", "read"]
    bad = [0, "barrier", "read", "load", "copy", "copy", 1, "barrier", "read"]
    assert _check(front + good, 2, 2, "good") == 3
    with pytest.raises(AssertionError, match="landed"):
        _check(front + bad, 2, 2, "bad")


def test_the_model_sees_a_copy_into_a_place_that_is_still_read():
    front = ["copy"] * 4 + [2, "barrier", "read"]
    with pytest.raises(AssertionError, match="copy of stage 2"):
        _check(front + ["copy", "copy", 0, "barrier", "read"], 2, 2, "bad")
