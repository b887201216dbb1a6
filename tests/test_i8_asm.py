"""Compiled code of the 8-bit products (no GPU): what tests/test_moe_asm.py checks
of the experts' products in bf16 holds for these kernels too, whose loads and core
they share."""
from __future__ import annotations

import re
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

import pytest

from tests import test_asm_hazards as hazards
from tests import test_lds_poison_build as poison
from tests import test_moe_asm as moe

UNIT = "i8_gemm.hip"


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    if not Path(poison.HIPCC).exists():
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("i8_asm")
    with ThreadPoolExecutor(max_workers=2) as pool:
        return dict(zip((False, True), pool.map(lambda p: poison._asm(UNIT, p, out), (False, True))))


def test_every_lds_load_is_poisoned_first(listings):
    n, guarded = poison._check(listings[True])
    assert n > 0 and guarded == n
    assert poison._check(listings[False])[0] == n


def test_nothing_spills(listings):
    found = 0
    for m in re.finditer(r"\.private_segment_fixed_size: (\d+)", listings[False]):
        found += 1
        assert m.group(1) == "0"
    assert found == len(list(moe._kernels(listings[False])))


def test_mfma_results_are_read_after_their_wait_states(listings, monkeypatch):
    """v_mfma_i32_16x16x64_i8 takes four passes, as the bf16 instruction of its size: 7 wait states."""
    whole = hazards.required_wait_states
    monkeypatch.setattr(hazards, "required_wait_states",
                        lambda op, ops: 7 if op.startswith("v_mfma_i32_16x16x64_i8") else whole(op, ops))
    text = listings[False]
    assert len(re.findall(r"^\s*v_mfma_i32_16x16x64_i8", text, flags=re.M)) > 100
    _, short = hazards.scan(text)
    assert not short, f"{len(short)} MFMA results read too early, e.g. {short[0]}"


@pytest.mark.parametrize("poisoned", [False, True])
def test_loads_read_their_descriptors_after_the_wait_states(listings, poisoned):
    writers, early = moe._early_sgpr_reads(listings[poisoned])
    assert writers > 100
    assert not early, f"{len(early)} SGPRs read too early, e.g. {early[0]}"


@pytest.mark.parametrize("poisoned", [False, True])
def test_every_load_statement_keeps_the_wait_states_itself(listings, poisoned):
    statements = 0
    for block in re.findall(r";+#ASMSTART\n(.*?);+#ASMEND", listings[poisoned], flags=re.S):
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
                assert ws >= moe.SGPR_WAIT and m0 is not None and ws - m0 >= 1, block
            elif q[0].startswith("v_") and any(moe._sgprs(a) for a in q[2:]):
                assert ws >= 2, block
            ws += 1
            if q[0].startswith("s_") and q[1] == "m0":
                m0 = ws
    assert statements > 100


@pytest.mark.parametrize("kernel", ["i8_tilesI", "i8_tiles_deepILi128ELi128ELb0ELb0"])
def test_lanes_hand_over_through_a_fence(kernel, tmp_path):
    """A block of results in and out of the wave's buffer."""
    if not Path(poison.HIPCC).exists():
        pytest.skip("hipcc not available")
    found = 0
    for part in re.split(r"^(?=define )", moe._device(poison.CSRC / UNIT, tmp_path / "u.ll", "-emit-llvm"), flags=re.M):
        if not part.startswith("define ") or "amdgpu_kernel" not in part[:200] or kernel not in part[:400]:
            continue
        found += 1
        assert len(re.findall(r'fence syncscope\("wavefront"\) acquire', part)) >= 2, part[:200]
        assert len(re.findall(r'fence syncscope\("wavefront"\) release', part)) >= 2, part[:200]
    assert found


def test_no_bare_wave_barrier():
    for name in (UNIT, "i8_quant.hip", "moe_core.h"):
        assert "__builtin_amdgcn_wave_barrier" not in (poison.CSRC / name).read_text(), name


@pytest.mark.parametrize("poisoned", [False, True])
def test_the_compiler_knows_what_the_loads_do_to_m0(poisoned, tmp_path):
    if not Path(poison.HIPCC).exists():
        pytest.skip("hipcc not available")
    flags = ["-emit-llvm", *(["-DDBS_LDS_POISON=1"] if poisoned else [])]
    text = moe._device(poison.CSRC / UNIT, tmp_path / "u.ll", *flags)
    writes = [x for x in text.splitlines() if " asm " in x and re.search(r"s_\w+ m0,", x)]
    assert len(writes) > 100
    for x in writes:
        constraints = re.findall(r'"([^"]*)"', x[x.index(" asm "):])[1]
        assert "{m0}" in [c.lstrip("=&") for c in constraints.split(",") if c.startswith("=")], x.strip()[:300]
