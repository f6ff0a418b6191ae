"""The wait states before every direct load to LDS, in the assembly of each source file that has such loads.

gfx950 leaves these waits to software, and the compiler adds none around inline assembly: one wait state between a
scalar write of M0 (the load's LDS address) and the load, five between a vector instruction's write of a scalar
register and a memory instruction that reads it (the load's base, or M0)."""
import concurrent.futures
import os
import re
import subprocess

import pytest

from nvfp4_weight_only_amd import build as BUILD

VECTOR = 5      # wait states behind a vector write of a scalar operand; one behind a scalar write of M0


def scalar_regs(text):
    """Indices of the scalar registers that the operands name ("m0" among them)."""
    regs = set(re.findall(r"\bm0\b", text))
    for lo, hi in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        regs |= set(range(int(lo), int(hi) + 1))
    return regs | {int(r) for r in re.findall(r"\bs(\d+)\b", text)}


def written(op, rest):
    """Scalar registers that an instruction writes: its first operand (and a carry, the second one, of v_add_co etc.)."""
    ops = re.split(r",\s*(?![^\[]*\])", rest)
    return scalar_regs(",".join(ops[:2] if op.startswith("v_") and "_co_" in op else ops[:1]))


def short_waits(asm):
    """(number of direct loads to LDS, [(line, what)] of those with too few wait states before them).

    Looked at backwards until the last write of every scalar operand is found or enough states have passed; a label
    before that counts as too few, since what a jump brings is not known (M0, which no vector instruction may write
    anywhere, needs one state there)."""
    lines, loads, bad = asm.split("\n"), 0, []
    for i, line in enumerate(lines):
        ins = line.split(";")[0].strip()
        if re.match(r"v_\w+ m0\b", ins):
            bad.append((i + 1, ins))
        if not re.match(r"(global|buffer|scratch)_load_lds_", ins):
            continue
        loads += 1
        pending, states, j = scalar_regs(ins) | {"m0"}, 0, i
        while pending and states < VECTOR and j > 0:
            j -= 1
            ins = lines[j].split(";")[0].strip()
            if ins.endswith(":"):
                if states == 0 or pending != {"m0"}:
                    bad.append((i + 1, "a label"))
                break
            if not ins or ins.startswith((".", "#")):
                continue
            op, _, rest = ins.partition(" ")
            if op == "s_nop":
                states += int(rest, 0) + 1
                continue
            hit = set() if op.startswith(("s_cmp", "s_cbranch", "s_waitcnt", "v_cmpx")) else written(op, rest) & pending
            if hit and (op.startswith("v_") or ("m0" in hit and states == 0)):
                bad.append((i + 1, f"{ins} {states} states before"))
                break
            pending -= hit
            states += 1
    return loads, bad


def test_the_scan_finds_planted_faults():
    load = "\tglobal_load_lds_dwordx4 v1, s[4:5]\n"
    assert short_waits("\ts_mov_b32 m0, s2\n\tglobal_load_lds_dword v[0:1], off\n")[1]
    assert short_waits("\tv_readfirstlane_b32 m0, v2\n\ts_nop 3\n\tglobal_load_lds_dword v[0:1], off\n")[1]
    assert short_waits("\tv_readfirstlane_b32 s5, v2\n\ts_mov_b32 m0, s2\n\ts_nop 2\n" + load)[1]
    assert short_waits("\tv_cmp_eq_u32_e64 s[4:5], v1, v2\n\ts_nop 3\n" + load)[1]
    assert short_waits(".L1:\n\ts_mov_b32 m0, s2\n\ts_nop 1\n" + load)[1]
    assert short_waits("\tv_readfirstlane_b32 s5, v2\n\ts_mov_b32 m0, s2\n\ts_nop 3\n" + load) == (1, [])
    assert short_waits("\tv_readfirstlane_b32 s3, v2\n\tv_readfirstlane_b32 s5, v2\n\ts_nop 4\n" + load) == (1, [])
    assert short_waits("\tv_readfirstlane_b32 s5, v2\n\ts_mov_b32 m0, s2\n\ts_mov_b64 s[4:5], s[6:7]\n" + load) == (1, [])
    assert short_waits("\tv_readfirstlane_b32 s5, v2\n\ts_mov_b32 m0, s2\n\ts_mov_b32 s4, s6\n" + load)[1]
    assert short_waits("\ts_mov_b32 m0, s2\n\ts_nop 0\n.L1:\n\tglobal_load_lds_dword v[0:1], off\n")[1]


def _assembly(source):
    cmd = [BUILD.hipcc(), *BUILD.compile_flags(), "--offload-device-only", "-S", "-o", "-", os.path.join(BUILD.CSRC, source)]
    return subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, check=True).stdout.decode()


@pytest.fixture(scope="module")
def assembly():
    """Assembly of every source file, compiled side by side."""
    with concurrent.futures.ThreadPoolExecutor(min(len(BUILD.SOURCES), os.cpu_count() or 1)) as pool:
        return dict(zip(BUILD.SOURCES, pool.map(_assembly, BUILD.SOURCES)))


@pytest.mark.parametrize("source", BUILD.SOURCES)
def test_direct_loads_to_lds_have_their_wait_states(assembly, source):
    loads, bad = short_waits(assembly[source])
    assert not bad, f"{len(bad)} of {loads} loads, first {bad[:3]}"


def test_the_files_with_direct_loads_are_looked_at(assembly):
    found = {s for s in BUILD.SOURCES if short_waits(assembly[s])[0]}
    assert found == {"small_m.hip", "skinny.hip", "prefill.hip", "mxfp4.hip", "fp8_gemm.hip"}
