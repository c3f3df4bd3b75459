"""treewy_attend where errors hide behind a bound for each element: long contexts, of which a part could be lost, and tokens
beside one that has most of the weight.  Bounds are of the norm of a row's output, or of values that mark their tile."""
import numpy as np
import pytest
import torch

from gdn_speculative_tree_gb300 import binding
from oracle import attend_oracle as orc
from tests.cache_helpers import E4M3, TYPES, Attend, f64

pytestmark = pytest.mark.gpu

GENERIC = binding.FLAG_FORCE_GENERIC


class Shared:
    """R requests of N nodes (chains) over the pages of one context: keys and values are e4m3 numbers, the scales 1."""

    def __init__(self, keys, values, *, R, N, G, page=64, scale=None, out="bf16", flags=0, seed=0):
        n, Hkv, d = keys.shape
        g = torch.Generator().manual_seed(seed)
        pages = -(-n // page)
        self.n, self.R, self.N, self.G, self.scale = n, R, N, G, d ** -0.5 if scale is None else scale
        self.k8, self.v8 = keys.to(E4M3), values.to(E4M3)

        def paged(x):
            room = torch.full((pages * page, Hkv, d), 127, dtype=torch.uint8)  # NaN behind the tokens
            room[:n] = x.view(torch.uint8)
            return room.view(pages, page, Hkv, d).transpose(1, 2).contiguous().cuda().view(E4M3)

        one = torch.ones(pages, Hkv, device="cuda")
        table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(R, 1)
        self.cache = binding.make_cache(k=paged(self.k8), v=paged(self.v8), k_scale=one, v_scale=one.clone(), page_table=table,
                                        length=torch.full((R,), n, dtype=torch.int32, device="cuda"))
        T = R * N
        self.off = torch.arange(0, T + 1, N, dtype=torch.int32, device="cuda")
        self.q = torch.randn(T, Hkv * G, d, generator=g).bfloat16().cuda()
        self.k, self.v = (torch.randn(T, Hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
        self.o = torch.full((T, Hkv * G, d), -7.0, dtype=TYPES[out], device="cuda")
        self.status, self.flags = torch.zeros(R, dtype=torch.int32, device="cuda"), flags

    def run(self):
        call = binding.make_attn(cache=self.cache, node_offset=self.off, q=self.q, k=self.k, v=self.v, o=self.o, status=self.status,
                                 scale=self.scale, max_nodes=self.N, max_context=self.n, flags=self.flags)
        binding.treewy_attend(call)
        torch.cuda.synchronize()
        assert not self.status.any()
        return self

    def want(self, r):
        at = slice(r * self.N, (r + 1) * self.N)
        keys, values = (f64(x.float()).swapaxes(0, 1) for x in (self.k8, self.v8))
        return orc.attend(f64(self.q[at]), f64(self.k[at]), f64(self.v[at]), np.arange(self.N) - 1, keys, values, self.scale)

    def off_by(self, requests):
        """The largest error of a row's output, relative to the row's norm."""
        worst = 0.0
        for r in requests:
            want, got = self.want(r), f64(self.o[r * self.N:(r + 1) * self.N])
            worst = max(worst, (np.linalg.norm(got - want, axis=2) / np.linalg.norm(want, axis=2)).max())
        return worst


# A weight is within 2^-8 of itself, an output's rounding 2^-8 of it: the errors of independent tokens add up as their values
# do, so that in the norm the output is off by no more than the two together, and by some 2^-24 of a score on the CUDA cores.
NORM = {0: 2.0 ** -7, GENERIC: 2.0 ** -8 + 1e-4}


@pytest.mark.parametrize("flags", [0, GENERIC])
@pytest.mark.parametrize("R,N,G", [(1, 1, 8), (3, 4, 2), (1, 9, 8), (160, 1, 2), (160, 5, 4)])
@pytest.mark.parametrize("n,page,d", [(9001, 16, 128), (5000, 64, 256), (4999, 128, 64)])
def test_every_tile_of_a_long_context_counts(cuda_lib, n, page, d, R, N, G, flags):
    """All scores alike, and the values of every tile of 128 tokens a number in a column of its own: the column of a tile
    that is left out, taken twice or cut short shows it."""
    keys, values = torch.randn(n, 1, d), torch.zeros(n, 1, d)
    tile = torch.arange(n) // 128
    values[torch.arange(n), 0, tile % d] = 1.0
    a = Shared(keys, values, R=R, N=N, G=G, page=page, flags=flags)
    a.q.zero_()
    a.v.zero_()
    a.run()
    seen = np.bincount(tile.numpy() % d, minlength=d)[:d]
    node = np.arange(N)[None, :, None, None]
    want = np.broadcast_to(seen / (n + node + 1.0), (R, N, G, d))
    # equal weights: 2^-8 of each and of the output's rounding
    assert (np.abs(f64(a.o).reshape(want.shape) - want) <= 2 * 2.0 ** -8 * want).all()


@pytest.mark.parametrize("flags", [0, GENERIC])
@pytest.mark.parametrize("R,N,G", [(1, 1, 8), (2, 9, 8), (3, 4, 2), (160, 1, 2), (160, 5, 4)])
@pytest.mark.parametrize("n,page", [(9001, 16), (5000, 64)])
def test_long_contexts_in_the_norm(cuda_lib, n, page, R, N, G, flags):
    """Random tokens: a lost tile of n / 128 would be some sqrt(128 / n) of the output, 0.12 to 0.16."""
    torch.manual_seed(n)
    a = Shared(torch.randn(n, 1, 128), torch.randn(n, 1, 128), R=R, N=N, G=G, page=page, flags=flags, seed=n + 1)
    assert a.run().off_by(range(0, R, 53)) <= NORM[flags]
    a.k8, a.v8 = (torch.cat([x.view(torch.uint8)[:1280], x.view(torch.uint8)[1408:]]).view(E4M3) for x in (a.k8, a.v8))
    assert a.off_by([0]) > 4 * NORM[flags]  # a definition that leaves a tile out is seen


@pytest.mark.parametrize("flags", [0, GENERIC])
@pytest.mark.parametrize("share", [0.3, 0.6])
@pytest.mark.parametrize("n", [2000, 8000, 32000])
@pytest.mark.parametrize("R,N,G", [(152, 1, 8), (152, 4, 4), (160, 5, 4)])
def test_tokens_beside_a_dominating_one(cuda_lib, R, N, G, n, share, flags):
    """A first token that has a share of every row's weight and next to no value: the outputs are the other tokens', each of
    which weighs 2^-11 to 2^-16 of it.  As many requests as leave each context in one piece."""
    torch.manual_seed(n)
    d = 128
    keys, values = torch.randn(n, 1, d), torch.randn(n, 1, d)
    keys[:, 0, 0] = 0.0
    keys[0] = 0.0
    # the others' scores have the variance |q|^2 / d = 1: e^0.5 on the average; q is 4 in the first column
    keys[0, 0, 0] = np.log(n * np.exp(0.5) * share / (1 - share)) * d ** 0.5 / 4
    values[0] *= 0.01
    a = Shared(keys, values, R=R, N=N, G=G, flags=flags, seed=n + 1)
    a.q[..., 0] = 4.0
    a.k[..., 0] = 0.0
    assert a.run().off_by([0, 70, R - 1]) <= NORM[flags]


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


@pytest.mark.parametrize("flags", [0, GENERIC])
@pytest.mark.parametrize("R,G,n,octaves", [(1, 8, 100000, 17), (1, 32, 100000, 17), (160, 8, 16000, 14), (160, 32, 16000, 14),
                                           (160, 8, 6000, 12.3), (160, 32, 6000, 12.3)])
def test_alike_tokens_that_weigh_next_to_nothing_each(cuda_lib, R, G, n, octaves, flags):
    """A first token with a weight of 1 and n of 2^-octaves each, which together count for about as much; values of -1 and 1.
    The contexts are cut into pieces (one request) or not.  Alike weights are off alike: 2^-8 of n w moves the output
    (n w - 1) / (n w + 1) by 2 n w / (n w + 1)^2, half at most, of that; and the output is rounded.  (In the piece that has
    the first token, those of 2^-17 are within 2^-4 of themselves; it has a hundredth of them.)"""
    keys, values = torch.zeros(n, 1, 64), torch.ones(n, 1, 64)
    keys[0, 0, 0], values[0] = 1.0, -1.0
    a = Shared(keys, values, R=R, N=1, G=G, scale=1.0, flags=flags)
    a.q.zero_(), a.k.zero_(), a.v.fill_(1.0)
    a.q[..., 0] = octaves * np.log(2)
    nw = n * np.exp(-float(a.q[0, 0, 0]))
    a.run()
    assert np.abs(f64(a.o) - (nw - 1) / (nw + 1)).max() <= 2.0 ** -9 + 2.0 ** -11 + 2.0 ** -8 * abs((nw - 1) / (nw + 1)) + 2.0 ** -12
