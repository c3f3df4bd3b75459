"""The delta rule over new tokens where keys are much alike and write strengths above one.

Tolerance of the chunked delta rule for unit keys and write strengths b.  Its state, pseudo-values and factors pass
through products as two bf16 terms, each 2^-17 of its operand off at most (2^-18 for the terms, as much for the product
of the two small ones).  A result adds 64 such products per chunk whose factors, the entries of (I + A)^-1 and of what
is made with it, are at most b times a unit vector's: with errors of either sign, sqrt(64) * 2^-17 * b of a value.
b <= 1: a token's write takes out what was there along its key, old errors with it, so one chunk counts: 2^-14.
1 < b <= 2: a write turns what was there round instead, and the errors of the n chunks before stay: sqrt(n) 2^-13,
n = 8: below 2^-11.  bf16 outputs leave two more products of that size out of the factor M T whose entries add 64
of them themselves: 4 times as much, beside their own rounding."""
from __future__ import annotations

import pytest
import torch

from oracle import serving_oracle as orc
from tests.test_gpu_serving import BF16_TOL, Case, assert_near, f64

pytestmark = pytest.mark.gpu


def alike(shape, cosine, seed):
    """Unit rows [T][H][d], any two of a head at this cosine in the mean."""
    g = torch.Generator().manual_seed(seed)
    base = torch.nn.functional.normalize(torch.randn(1, *shape[1:], generator=g), dim=-1)
    x = torch.nn.functional.normalize(torch.randn(*shape, generator=g), dim=-1)
    return torch.nn.functional.normalize(cosine ** 0.5 * base + (1 - cosine) ** 0.5 * x, dim=-1)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("like", ["queries", "keys"])
@pytest.mark.parametrize("b,tol", [(1.0, 2.0 ** -14), (1.9, 2.0 ** -11), (2.0, 2.0 ** -11)])
@pytest.mark.parametrize("cosine", [0.5, 0.9, 0.99])
def test_extend_alike_keys(cuda_lib, cosine, b, tol, like, out):
    """512 tokens without decay; queries independent of the keys, or the keys of the tokens before."""
    c = Case([512], H=4, alpha=(1.0, 1.0), beta=b, out=out, seed=30)
    k = alike(tuple(c.k.shape), cosine, 31)
    c.k.copy_(k)
    c.q.copy_(k.roll(1, 0) if like == "keys" else alike(tuple(c.q.shape), cosine, 32))
    c.run()
    s = int(c.slot[0])
    o, S = orc.extend(f64(c.before[s]), f64(c.q), f64(c.k), f64(c.v), f64(c.alpha), f64(c.beta))
    assert_near(c.pool[s], S, tol, label="state")
    assert_near(c.o, o, *((tol,) if out == "f32" else (4 * tol, BF16_TOL)), label="o")


@pytest.mark.parametrize("out,pool", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
def test_extend_same_bits_every_time(cuda_lib, out, pool):
    """Chunks on every SM, sequences of many lengths: nothing depends on the order in which the roles run."""
    lens = [1500, 1, 700, 64, 65, 999]
    runs = [Case(lens, H=32, Hk=16, out=out, pool=pool, seed=33).run() for _ in range(4)]
    for c in runs[1:]:
        assert torch.equal(c.o, runs[0].o) and torch.equal(c.pool, runs[0].pool)
