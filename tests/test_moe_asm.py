"""Compiled code of the mixture-of-experts products (no GPU): every read of an
MFMA result comes after the ISA's wait states, no kernel of theirs keeps
tile registers in scratch memory inside its stages, and in the LDS-poison
build every direct-to-LDS load comes after a waited-for poison write."""
from __future__ import annotations

import re
import subprocess
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

import pytest

from tests import test_asm_hazards as hazards
from tests import test_lds_poison_build as poison

UNITS = ["moe_gemm.hip"]


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    if not Path(poison.HIPCC).exists():
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("moe_asm")
    jobs = [(u, p) for u in UNITS for p in (False, True)]
    with ThreadPoolExecutor(max_workers=4) as pool:
        return dict(zip(jobs, pool.map(lambda j: poison._asm(j[0], j[1], out), jobs)))


def test_every_lds_load_is_poisoned_first(listings):
    n, guarded = poison._check(listings[("moe_gemm.hip", True)])
    assert n > 0 and guarded == n
    assert poison._check(listings[("moe_gemm.hip", False)])[0] == n


def _kernels(text):
    for m in re.finditer(r"^(_Z\w+):\s*; @", text, flags=re.M):
        end = text.index(".Lfunc_end", m.end())
        yield m.group(1), text[m.end():end]


@pytest.mark.parametrize("unit", UNITS)
def test_stages_do_not_touch_scratch(listings, unit):
    """Between two MFMAs there is no scratch access: what spills does so
    outside the loops over stages."""
    found = 0
    for name, body in _kernels(listings[(unit, False)]):
        lines = [x.strip() for x in body.splitlines()]
        mf = [i for i, x in enumerate(lines) if x.startswith("v_mfma")]
        if not mf:
            continue
        found += 1
        for a, b in zip(mf, mf[1:]):
            if b - a < 150:                       # one loop body, not the way to the next variant
                assert not any(x.startswith("scratch_") for x in lines[a:b]), name
    assert found


@pytest.mark.parametrize("unit", UNITS)
def test_mfma_results_are_read_after_their_wait_states(listings, unit):
    """The scan returns readers within 8 wait states of the required ones;
    where each comes later, as here between a tile's last MFMA and its
    epilogue, there is none to return."""
    text = listings[(unit, False)]
    assert len(re.findall(r"^\s*v_mfma", text, flags=re.M)) > 100
    _, short = hazards.scan(text)
    assert not short, f"{len(short)} MFMA results read too early, e.g. {short[0]}"


# An SGPR that a vector instruction has written may be read by a vector memory
# instruction only five wait states later.  The compiler keeps them for its
# own instructions, not for those inside inline asm, which the direct-to-LDS
# loads of these kernels are.
SGPR_WAIT = 5


def _sgprs(tok):
    m = re.match(r"s\[(\d+):(\d+)\]$", tok)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.match(r"s(\d+)$", tok)
    return {int(m.group(1))} if m else set()


def _sgpr_results(op, ops):
    """SGPRs that a vector instruction writes."""
    if op.startswith(("v_readfirstlane", "v_readlane", "v_cmp")):
        return _sgprs(ops[0])
    if op.startswith(("v_add_co", "v_sub_co", "v_subrev_co", "v_addc_co", "v_subb_co", "v_subbrev_co", "v_div_scale",
                      "v_mad_u64", "v_mad_i64")):
        return _sgprs(ops[1])
    return set()


def _early_sgpr_reads(text):
    """(vector instructions that write SGPRs, [(wait states, writer, reader)] below SGPR_WAIT), on every path."""
    lines = []
    for raw in text.splitlines():
        s = raw.split(";")[0].strip()
        if s and (not s.startswith(".") or s.endswith(":")):
            lines.append(s)
    label = {s[:-1]: i for i, s in enumerate(lines) if s.endswith(":")}
    writers, early = 0, []
    for i, s in enumerate(lines):
        p = s.replace(",", " ").split()
        dst = _sgpr_results(p[0], p[1:])
        if not dst:
            continue
        writers += 1
        paths = [(i + 1, 0, dst)]
        while paths:
            j, ws, live = paths.pop()
            while j < len(lines) and ws < SGPR_WAIT and live:
                t = lines[j]
                j += 1
                if t.endswith(":"):
                    continue
                q = t.replace(",", " ").split()
                if q[0] == "s_nop":
                    ws += int(q[1], 0) + 1
                    continue
                if q[0].startswith(("buffer_", "global_", "flat_", "scratch_")):
                    if any(live & _sgprs(a) for a in q[1:]):
                        early.append((ws, s, t))
                        break
                elif q[0].startswith("s_cbranch"):
                    paths.append((label[q[1]], ws + 1, live))
                elif q[0].startswith("s_") and len(q) > 1:
                    live = live - _sgprs(q[1])             # a scalar result takes its place
                if q[0] == "s_branch":
                    j = label[q[1]]
                if q[0] in ("s_endpgm", "s_setpc_b64"):
                    break
                ws += 1
    return writers, early


def test_the_scan_finds_an_early_read_of_an_sgpr():
    early = "v_readfirstlane_b32 s6, v1\ns_mov_b32 s7, 0\ns_nop 2\nbuffer_load_dword v1, v0, s[4:7], 0 offen lds\n"
    assert _early_sgpr_reads(early) == (1, [(4, "v_readfirstlane_b32 s6, v1",
                                             "buffer_load_dword v1, v0, s[4:7], 0 offen lds")])
    assert _early_sgpr_reads(early.replace("s_nop 2", "s_nop 3")) == (1, [])
    assert _early_sgpr_reads(early.replace("s_mov_b32 s7", "s_mov_b32 s6")) == (1, [])


@pytest.mark.parametrize("unit", UNITS)
@pytest.mark.parametrize("poisoned", [False, True])
def test_loads_read_their_descriptors_after_the_wait_states(listings, unit, poisoned):
    writers, early = _early_sgpr_reads(listings[(unit, poisoned)])
    assert writers > 100
    assert not early, f"{len(early)} SGPRs read too early, e.g. {early[0]}"


@pytest.mark.parametrize("poisoned", [False, True])
def test_the_compiler_knows_what_the_loads_do_to_m0(poisoned, tmp_path):
    """M0, which holds a load's destination, is written inside inline asm: each
    such statement has it as an output, or the compiler might take a value of
    its own to be still there (in the IR: {m0} among the asm's outputs)."""
    if not Path(poison.HIPCC).exists():
        pytest.skip("hipcc not available")
    out = tmp_path / "moe_gemm.ll"
    subprocess.run([poison.HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", f"-I{poison.ROOT / 'include'}",
                    f"-I{poison.CSRC}", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "--cuda-device-only",
                    "-S", "-emit-llvm", *(["-DDBS_LDS_POISON=1"] if poisoned else []),
                    str(poison.CSRC / "moe_gemm.hip"), "-o", str(out)], check=True, capture_output=True)
    writes = [x for x in out.read_text().splitlines() if " asm " in x and re.search(r"s_\w+ m0,", x)]
    assert len(writes) > 100
    for x in writes:
        constraints = re.findall(r'"([^"]*)"', x[x.index(" asm "):])[1]
        assert "{m0}" in [c.lstrip("=&") for c in constraints.split(",") if c.startswith("=")], x.strip()[:300]


# ---- values handed from lane to lane through LDS inside a wave ------------------

def _device(src, out, *flags):
    subprocess.run([poison.HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", f"-I{poison.ROOT / 'include'}",
                    f"-I{poison.CSRC}", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "--cuda-device-only",
                    "-S", *flags, str(src), "-o", str(out)], check=True, capture_output=True)
    return out.read_text()


HANDED = """#include <hip/hip_runtime.h>
#include "moe_device.h"
__global__ void by_nothing(float *out, const int *to, const float *x) {
    __shared__ float row[64];
    row[threadIdx.x] = 0.0f;
    out[threadIdx.x] = row[threadIdx.x];
}
__global__ void by_handover(float *out, const int *to, const float *x) {
    __shared__ float row[64];
    row[threadIdx.x] = 0.0f;
    dbs::wave_handover();
    out[threadIdx.x] = row[threadIdx.x];
}
"""


def test_a_handover_reads_lds_again(tmp_path):
    """What a lane stored may be another lane's by the time it is read: the
    compiler may not answer the read with the lane's own value, as it does
    where nothing stands between."""
    if not Path(poison.HIPCC).exists():
        pytest.skip("hipcc not available")
    src = tmp_path / "handed.hip"
    src.write_text(HANDED)
    kernels = dict(_kernels(_device(src, tmp_path / "handed.s")))
    reads = {name: "ds_read" in body for name, body in kernels.items()}
    assert [v for k, v in sorted(reads.items()) if "by_nothing" in k] == [False]
    assert [v for k, v in sorted(reads.items()) if "by_handover" in k] == [True]


@pytest.mark.parametrize("unit,kernel,handovers", [
    ("moe_route.hip", "route_bwd", 2),           # zeros, chosen experts' gradients
    ("moe_gemm.hip", "moe_dw", 2),               # table of rows, order of groups
    ("moe_gemm.hip", "moe_tilesI", 2),           # a block of results in and out of the wave's buffer
])
def test_lanes_hand_over_through_a_fence(unit, kernel, handovers, tmp_path):
    if not Path(poison.HIPCC).exists():
        pytest.skip("hipcc not available")
    found = 0
    for part in re.split(r"^(?=define )", _device(poison.CSRC / unit, tmp_path / "u.ll", "-emit-llvm"), flags=re.M):
        if not part.startswith("define ") or "amdgpu_kernel" not in part[:200] or kernel not in part[:400]:
            continue
        found += 1
        assert len(re.findall(r'fence syncscope\("wavefront"\) acquire', part)) >= handovers, part[:200]
        assert len(re.findall(r'fence syncscope\("wavefront"\) release', part)) >= handovers, part[:200]
    assert found


def test_no_bare_wave_barrier():
    for f in sorted(poison.CSRC.glob("moe_*.hip")):
        assert "__builtin_amdgcn_wave_barrier" not in f.read_text(), f.name


@pytest.mark.parametrize("unit", UNITS)
@pytest.mark.parametrize("poisoned", [False, True])
def test_every_load_statement_keeps_the_wait_states_itself(listings, unit, poisoned):
    """Whatever the compiler puts right before one: inside the statement a
    vector instruction reads an SGPR after two wait states at the earliest, a
    load after five, and a load comes one after M0 is written."""
    statements = 0
    for block in re.findall(r";+#ASMSTART\n(.*?);+#ASMEND", listings[(unit, poisoned)], flags=re.S):
        lines = [x.split(";")[0].strip() for x in block.splitlines()]
        if not any(poison.DMA.match(x) for x in lines):
            continue
        statements += 1
        ws, m0 = 0, None
        for x in lines:
            if not x:
                continue
            q = x.replace(",", " ").split()
            if q[0] == "s_nop":
                ws += int(q[1], 0) + 1
                continue
            if q[0].startswith("buffer_load"):
                assert ws >= SGPR_WAIT and m0 is not None and ws - m0 >= 1, block
            elif q[0].startswith("v_") and any(_sgprs(a) for a in q[2:]):
                assert ws >= 2, block
            ws += 1
            if q[0].startswith("s_") and q[1] == "m0":
                m0 = ws
    assert statements > 100
