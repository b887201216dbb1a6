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
