"""The serving example: its steps agree with the 64-bit definitions from end to end."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import gdn_tree_oracle as tree_orc
from oracle import serving_oracle as orc

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("serve_round", os.path.join(ROOT, "examples", "serve_round.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(x):
    return x.detach().cpu().to(torch.float64).numpy()


def test_serving_round_against_the_definitions(cuda_lib):
    """Prompt, fork, tree verification with commit, and one more token.  The
    tolerances are the verification's own: 2e-3 of the largest output, 1e-3 of
    the largest state entry, plus a bf16 output's rounding, 2^-8 of itself."""
    m = example()
    requests, heads = 2, 4
    layer, out, status = m.run(requests, 90, heads, seed=3)
    torch.cuda.synchronize()
    assert not status.any().item()
    # the same random draws again, through the definitions
    ref = m.Layer(heads, heads // 2, 2 * requests, seed=3)

    def norm(x, scale=1.0, repeat=1):
        y = orc.norm_rotate(f64(x), "l2", 1e-6, scale=scale, repeat=repeat)
        return f64(torch.from_numpy(y).to(torch.bfloat16))  # as the kernel stores them

    def extend(lengths, slots, state):
        q, k, v, a, b = ref.project(sum(lengths))
        q, k = norm(q, 128 ** -0.5), norm(k)
        o, lo = [], 0
        for n, s in zip(lengths, slots):
            r, state[s] = orc.extend(state[s], q[lo:lo + n], k[lo:lo + n], f64(v)[lo:lo + n], f64(a)[lo:lo + n],
                                     f64(b)[lo:lo + n])
            o.append(r)
            lo += n
        return np.concatenate(o)

    state = np.zeros(tuple(layer.pool.shape))
    prompt = extend([90, 53], [0, 1], state)
    state[2:] = state[:2]
    tree = m.workloads.complete_binary_parents(4)
    accepted = torch.randint(-1, len(tree), (2 * requests,), generator=ref.g, device="cuda", dtype=torch.int32).tolist()
    q, k, v, a, b = ref.project(2 * requests * len(tree))
    q, k, v, a, b = norm(q, 128 ** -0.5, 2), norm(k, 1.0, 2), f64(v), f64(a), f64(b)
    draft = []
    for s in range(2 * requests):
        at = slice(s * len(tree), (s + 1) * len(tree))
        res = tree_orc.verify_request(state[s], np.asarray(tree), q[at], k[at], v[at], a[at], b[at])
        draft.append(res.o)
        state[s] = tree_orc.commit_request(state[s], res, accepted[s])
    token = extend([1] * (2 * requests), range(2 * requests), state)
    for got, want in ((out["prompt"], prompt), (out["draft"], np.concatenate(draft)), (out["token"], token)):
        assert (np.abs(f64(got) - want) <= 2e-3 * np.abs(want).max() + 2.0 ** -8 * np.abs(want)).all()
    assert np.abs(f64(layer.pool) - state).max() <= 1e-3 * np.abs(state).max()
