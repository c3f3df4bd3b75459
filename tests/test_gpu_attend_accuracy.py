"""treewy_attend where errors hide behind a bound for each element."""
import numpy as np
import pytest
import torch

from tests.cache_helpers import Attend, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq", [8, 32])
def test_small_values_of_a_row_to_what_its_terms_hold(cuda_lib, Hq):
    """The draft's keys as terms: 2^-17 of the row's largest, for small values too, whose first term has few bits left.

    In units in which a key's largest value is 2^7 its second one runs through every bf16 number of [2^-12, 2^-4) and the other
    node's through the nearest multiples of 2^-9, which terms hold as they are.  Queries are unit vectors, so a
    score is scale times the value; node 1 weighs the two by values of 0 and 1, and the scores' difference
    comes back from the output.  It is off by 2^-17 scale = 1/2, and by an eighth for the weights' (2^-8 each) and
    the output's (2^-8) roundings, of an output between 0.2 and 0.8."""
    d, cols = 64, 63
    bits = np.arange(128) / 128 + 1.0
    unit = np.concatenate([bits * 2.0 ** e for e in range(-12, -4)])
    unit = np.concatenate([unit, -unit])
    unit = unit[:unit.size // cols * cols]
    R = unit.size // cols * (-(-cols // Hq))
    y = np.repeat(unit.reshape(-1, cols), -(-cols // Hq), axis=0)           # [R][cols]
    near = np.round(y * 2 ** 9) / 2 ** 9
    k = np.zeros((R, 2, 1, d))
    k[:, :, 0, 0] = 1.0
    k[:, 0, 0, 1:], k[:, 1, 0, 1:] = near / 128, y / 128
    column = 1 + (np.arange(R)[:, None] % -(-cols // Hq) * Hq + np.arange(Hq)) % cols
    q = np.zeros((R, 2, Hq, d))
    q[np.arange(R)[:, None, None], np.arange(2)[None, :, None], np.arange(Hq), column[:, None]] = 1.0
    v = np.zeros((R, 2, 1, d))
    v[:, 1] = 1.0
    scale = 2.0 ** 16
    a = Attend([0] * R, [2] * R, Hq=Hq, Hkv=1, d=d, kind="chain", scale=scale)
    for x, y0 in ((a.q, q), (a.k, k), (a.v, v)):
        x.copy_(torch.from_numpy(y0.reshape(tuple(x.shape))))
        assert np.array_equal(f64(x), y0.reshape(tuple(x.shape)))
    a.run()
    assert not a.status.any()
    o = f64(a.o).reshape(R, 2, Hq, d)[:, 1, :, 0]
    got = np.log(o / (1 - o))
    want = scale * np.take_along_axis(k[:, 1, 0] - k[:, 0, 0], column, axis=1)
    assert np.abs(got - want).max() <= 0.5 + 0.125
