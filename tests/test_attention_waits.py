"""The attention kernels' direct transfers to LDS are complete before the barrier that
hands their tile to the other waves.  A workgroup barrier orders LDS accesses, not
transfers still on their way from memory, and a late one only shows as a wrong sum
now and then: so this follows the compiled kernels' control flow instead.  No GPU."""
import os
import re
import shutil
import subprocess

import pytest

from bit_nf4_quantized_13_amd import build


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """name -> instructions and labels of each kernel of attention.hip."""
    if shutil.which(build.HIPCC) is None:
        pytest.skip("no hipcc")
    out = tmp_path_factory.mktemp("asm") / "attention.s"
    subprocess.run([build.HIPCC, "-x", "hip", "-S", "--cuda-device-only", os.path.join(build.CSRC, "attention.hip"), "-o",
                    str(out)] + build.COMMON_FLAGS, check=True, capture_output=True, timeout=300)
    found, lines = {}, None
    for line in out.read_text().splitlines():
        line = line.split(";")[0].strip()
        start = re.fullmatch(r"(_Z\w*attention_\w+):", line)
        if start:
            lines = found.setdefault(start.group(1), [])
        elif line.startswith(".Lfunc_end"):
            lines = None
        elif lines is not None and line and (not line.startswith(".") or line.endswith(":")):
            lines.append(line)
    return found


def unfinished(code):
    """The barriers (and ends) of a kernel that some path reaches with transfers to LDS under way."""
    label = {line[:-1]: i for i, line in enumerate(code) if line.endswith(":")}
    seen, bad, todo = set(), set(), [(0, False)]
    while todo:
        at = todo.pop()
        if at in seen:
            continue
        seen.add(at)
        i, flying = at
        op, rest = (code[i].split(None, 1) + [""])[:2]
        if op.startswith("buffer_load") and re.search(r"\blds\b", rest):
            flying = True
        elif op == "s_waitcnt" and "vmcnt(0)" in rest:
            flying = False
        elif op in ("s_barrier", "s_endpgm") and flying:
            bad.add((i, op))
        assert op not in ("s_setpc_b64", "s_swappc_b64"), "a call: its target is not followed"
        if op == "s_endpgm":
            continue
        if op == "s_branch":
            todo.append((label[rest], flying))
            continue
        if op.startswith("s_cbranch"):
            todo.append((label[rest], flying))
        todo.append((i + 1, flying))
    return bad


@pytest.mark.parametrize("kind", ["fwd", "dq", "dkv"])
def test_no_barrier_with_a_transfer_under_way(kernels, kind):
    code = {n: c for n, c in kernels.items() if f"attention_{kind}_kernel" in n}
    assert code
    for name, lines in code.items():
        assert any(re.search(r"^buffer_load.*\blds\b", x) for x in lines) and "s_barrier" in lines, name
    bad = {n: unfinished(c) for n, c in code.items()}
    assert not any(bad.values()), {n: sorted(b) for n, b in bad.items() if b}


def test_the_search_sees_a_missing_wait():
    """A kernel with a wait on one of two paths to its barrier."""
    head = ["buffer_load_dwordx4 v1, s[4:7], 0 offen lds", "s_cbranch_scc1 .L1"]
    tail = [".L1:", "s_barrier", "s_endpgm"]
    assert unfinished(head + ["s_waitcnt vmcnt(0)"] + tail) == {(4, "s_barrier"), (5, "s_endpgm")}
    assert unfinished(head + tail[:1] + ["s_waitcnt vmcnt(0) lgkmcnt(0)"] + tail[1:]) == set()
    assert unfinished(head + tail[:1] + ["s_waitcnt vmcnt(4)"] + tail[1:])
