"""Static check of the library's gfx950 code for the wait states of loads that go straight into LDS.

Such a load takes its LDS address from M0, and one wait state must pass between the write of M0 and the load; five must
pass between a VALU instruction that writes a scalar register and a vector-memory instruction that reads it. The
compiler counts both for its own loads, but not for those in inline assembly. This test compiles the sources that hold
such loads with the library's flags and reads every load and what stands before it (one wait state per instruction,
s_nop N counting N + 1).
"""
import os
import re
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

from chunk_wise_weight_amd import build as B

LOAD = re.compile(r"^(buffer|global|scratch)_load_\w+ .*\blds$")


def _sregs(text):
    regs = {int(r) for r in re.findall(r"\bs(\d+)\b", text)}
    for lo, hi in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        regs.update(range(int(lo), int(hi) + 1))
    return regs


def loads_and_exposed(asm_text):
    """The loads into LDS, and (instruction, load) pairs that are too close."""
    lines = [l.split(";")[0].strip() for l in asm_text.splitlines()]
    lines = [l for l in lines if l and not l.startswith(".") and not l.endswith(":")]
    count, bad = 0, []
    for i, l in enumerate(lines):
        if not LOAD.match(l):
            continue
        count += 1
        reads, waits = _sregs(l.partition(" ")[2]), 0
        for p in reversed(lines[max(0, i - 5):i]):
            op, _, rest = p.partition(" ")
            if op == "s_nop":
                waits += int(rest, 0) + 1
            else:
                written = rest.split(",")[0].strip()
                if waits < 1 and written == "m0" and op.startswith("s_"):
                    bad.append((p, l))
                if op.startswith("v_") and _sregs(written) & reads:
                    bad.append((p, l))
                waits += 1
            if waits >= 5:
                break
    return count, bad


def test_what_is_too_close_is_found():
    load = "buffer_load_dwordx4 v1, s[8:11], s0 offen lds\n"
    assert loads_and_exposed("s_mov_b32 m0, s4\n" + load) == (1, [("s_mov_b32 m0, s4", load.strip())])
    assert loads_and_exposed("s_mov_b32 m0, s4\ns_nop 0\n" + load) == (1, [])
    assert loads_and_exposed("s_mov_b32 m0, s4\nv_add_u32_e32 v1, 1, v1\n" + load) == (1, [])
    assert len(loads_and_exposed("v_readfirstlane_b32 s9, v2\ns_nop 3\n" + load)[1]) == 1
    assert loads_and_exposed("v_readfirstlane_b32 s9, v2\ns_nop 4\n" + load) == (1, [])
    assert loads_and_exposed("v_readfirstlane_b32 s12, v2\n" + load) == (1, [])
    assert loads_and_exposed("buffer_load_dwordx4 v[4:7], v1, s[8:11], 0 offen\n") == (0, [])


def test_library_loads_into_lds_wait_for_m0_and_their_descriptors():
    try:
        hipcc = B._hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    inc = ["-I", os.path.join(B.ROOT, "include"), "-I", B.CSRC]
    flags = [f for f in B.HIPCC_FLAGS if f != "-fPIC"]

    def holds_loads(src):
        with open(os.path.join(B.CSRC, src)) as fh:
            return "load_lds" in fh.read()

    with tempfile.TemporaryDirectory() as tmp:
        def check(src):
            out = os.path.join(tmp, src + ".s")
            r = subprocess.run([hipcc, *flags, *inc, "-S", "--cuda-device-only", os.path.join(B.CSRC, src),
                                "-o", out], capture_output=True, text=True)
            assert r.returncode == 0, r.stderr[-2000:]
            with open(out) as fh:
                return src, *loads_and_exposed(fh.read())

        sources = [s for s in B.SOURCES if holds_loads(s)]
        with ThreadPoolExecutor(max_workers=4) as ex:
            got = list(ex.map(check, sources))
    assert {"kernels_bf16.hip", "kernels_dense.hip"} <= {src for src, _, _ in got}
    for src, count, bad in got:
        assert count > 0 and bad == [], (src, len(bad), bad[:3])
