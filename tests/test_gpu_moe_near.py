"""Choices of the router by groups between scores that a bias nearly cancels (-m gpu)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_block_scaled_amd as dbs
from tests import _i8, _moe

pytestmark = pytest.mark.gpu

EXPERT, GROUP = 2.0 ** -39, 2.0 ** -37       # what tells two apart, of the largest score or bias


def _near(E, seed, scores, T=400):
    """Logits a few steps of fp32 apart from token to token, and the bias that cancels the first token's
    scores but for fp32's rounding."""
    g = np.random.default_rng(seed)
    first = g.standard_normal(E).astype(np.float32)
    x = first + g.integers(-40, 41, (T, E)) * np.spacing(np.abs(first))
    x[0] = first
    bias = (-_i8.scores(first.astype(np.float64), scores)).astype(np.float32)
    return x.astype(np.float32), bias


def _told_apart(x, bias, groups, best, scores):
    """Tokens whose neighbours in the order of c, and of the groups' scores, are further apart than the bound."""
    fine = np.ones(len(x), dtype=bool)
    b = bias.astype(np.float64)
    for t, row in enumerate(x.astype(np.float64)):
        s = _i8.scores(row, scores)
        c = s + b
        most = max(s.max(), np.abs(b).max())
        score = np.sort(c.reshape(groups, -1), axis=1)[:, -best:].sum(1)
        fine[t] = np.diff(np.sort(c)).min() > EXPERT * most and (groups == 1 or np.diff(np.sort(score)).min() > GROUP * most)
    return fine


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,groups,kept,best", [(8, 3, 1, 1, 2), (16, 4, 4, 2, 2), (24, 5, 3, 2, 1), (32, 8, 8, 4, 2)])
def test_biases_that_nearly_cancel(E, k, groups, kept, best, scores):
    x, bias = _near(E, E + k, scores)
    fine = _told_apart(x, bias, groups, best, scores)
    c = _i8.scores(x[1].astype(np.float64), scores) + bias
    assert fine.mean() > 0.9 and np.abs(c).max() < 2.0 ** -16        # (little is left of the terms)
    got = dbs.moe_route_grouped(torch.tensor(x).cuda(), k, torch.tensor(bias).cuda(), groups, kept, best, scores)
    want = _i8.choose(x.astype(np.float64), k, bias.astype(np.float64), groups, kept, best, scores)
    assert np.array_equal(got.experts.cpu().numpy()[fine], want[fine])
    # every token, told apart or not, has k different experts of the kept groups
    e = np.sort(got.experts.cpu().numpy(), axis=1)
    assert e.min() >= 0 and (np.diff(e, axis=1) > 0).all()
    assert max(len(set(row // (E // groups))) for row in e) <= kept


def test_the_same_logit_and_bias_go_by_index():
    x = torch.randn(50, 1, generator=torch.Generator().manual_seed(3)).repeat(1, 16)
    bias = torch.full((16,), -float(torch.sigmoid(x[0, 0])))
    for groups, kept in ((1, 1), (4, 2)):
        r = dbs.moe_route_grouped(x.cuda(), 5, bias.cuda(), groups, kept)
        assert r.experts.cpu().tolist() == [[0, 1, 2, 3, 4]] * 50
