"""The row quantiser on the GPU for more rows than one launch takes (-m gpu)."""
from __future__ import annotations

import pytest
import torch

import dense_block_scaled_amd as dbs
from tests import _i8

pytestmark = pytest.mark.gpu


def _want(x):
    """codes and scales in 64 bits.  A quotient that is a tie is exact there, and any other lies further from one
    than 2^-34 (254 |x| and (2 m + 1) amax differ by a step of x, which is at least 2^-31 of amax)."""
    a = x.double()
    amax = a.abs().amax(1, keepdim=True)
    return torch.where(amax > 0, torch.round(127 * a / amax), 0.0).to(torch.int8), amax[:, 0] / 127


# rows on both sides of one launch's, of two launches', and of where a row's 256 threads pass 2^32
@pytest.mark.parametrize("M,K,dtype", [((1 << 23) + 1, 5, torch.float32), ((1 << 24) - 1, 8, torch.bfloat16),
                                       (1 << 24, 1, torch.float32), ((1 << 24) + 1, 5, torch.float32),
                                       ((1 << 24) + 3, 17, torch.bfloat16), (1 << 25, 2, torch.bfloat16)])
def test_quant_of_many_rows(M, K, dtype):
    print("quant", M, K, dtype, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=dtype)
    x[-1] = torch.arange(1, K + 1, device="cuda")
    q, s = dbs.quant_i8(x)
    step = 1 << 22
    for m in range(0, M, step):
        codes, scales = _want(x[m:m + step])
        assert torch.equal(q[m:m + step], codes), m
        assert bool(((s[m:m + step].double() - scales).abs() <= _i8.HALF_F32 * scales).all()), m


def test_captured_quant_of_many_rows():
    M, K = (1 << 23) + 1, 3
    x = torch.zeros(M, K, device="cuda")
    dbs.quant_i8(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, s = dbs.quant_i8(x)
    for seed in range(3):
        x.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
        graph.replay()
        codes, scales = dbs.quant_i8(x)
        assert torch.equal(q, codes) and torch.equal(s, scales)
        assert torch.equal(codes[-1], _want(x[-1:])[0][0])
