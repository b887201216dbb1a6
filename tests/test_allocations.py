"""How the binding allocates outputs (no GPU): directly where nobody sees it, through
torch.empty where a mode or deterministic algorithms would."""
from __future__ import annotations

import pytest
import torch
from torch.overrides import TorchFunctionMode
from torch.utils._python_dispatch import TorchDispatchMode

import dense_block_scaled_amd as dbs

HERE = torch.device("cpu", 0)             # stands in for the current GPU


class Dispatched(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.seen = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.seen.append(str(func))
        return func(*args, **(kwargs or {}))


class Called(TorchFunctionMode):
    def __init__(self):
        super().__init__()
        self.seen = []

    def __torch_function__(self, func, types, args=(), kwargs=None):
        self.seen.append(func)
        return func(*args, **(kwargs or {}))


@pytest.fixture
def direct(monkeypatch):
    """The shapes and strides that went to the direct allocation."""
    calls = []

    def empty_strided(shape, strides, dtype):
        calls.append((shape, strides))
        return torch.empty_strided(shape, strides, dtype=dtype)

    monkeypatch.setattr(dbs, "_empty_strided", empty_strided)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return calls


def _new(*shape, dtype=torch.float32):
    t = dbs._new(shape, dtype, HERE)
    assert t.shape == shape and t.dtype == dtype and t.is_contiguous()
    return t


def test_direct_where_nobody_sees_it(direct):
    _new(5)
    _new(3, 4)
    _new(3, 0)
    assert direct == [((5,), (1,)), ((3, 4), (4, 1)), ((3, 0), (1, 1))]
    dbs._new((2,), torch.int8, torch.device("cpu", 1))            # not the current device
    assert len(direct) == 3


def test_dispatch_modes_see_allocations(direct):
    with Dispatched() as mode:
        _new(3, 4)
    assert not direct and any("empty" in s for s in mode.seen)


def test_function_modes_see_allocations(direct):
    with Called() as mode:
        dbs._new((3, 4), torch.float32, HERE)
    assert not direct and torch.empty in mode.seen


def test_deterministic_algorithms_fill_allocations(direct):
    torch.use_deterministic_algorithms(True)
    try:
        assert torch.isnan(_new(3, 4)).all() and (_new(7, dtype=torch.int8) == 127).all()
    finally:
        torch.use_deterministic_algorithms(False)
    assert not direct


def test_without_a_way_to_see_them_nothing_is_direct(monkeypatch):
    monkeypatch.setattr(dbs, "_empty_strided", None)
    _new(3, 4)


def test_routers_need_no_workspace_where_the_binding_does_not_ask():
    L = dbs.lib()
    for workspace in (L.moe_route_workspace, L.moe_route_grouped_workspace):
        for E in (1, 8, 160, 1024):
            for T in range(1, dbs._NO_WORKSPACE_TOKENS + 1):
                assert workspace(T, E, 1) == 0 and workspace(T, E, min(E, 16)) == 0
            assert workspace(dbs._NO_WORKSPACE_TOKENS + 1, E, 1) > 0
