"""The softmax layer of the serving example: its steps agree with the 64-bit definitions from end to end."""
import numpy as np
import pytest
import torch

from oracle import attend_oracle as orc
from oracle import serving_oracle
from tests.test_gpu_serving_round import example, f64

pytestmark = pytest.mark.gpu


def test_softmax_round_against_the_definitions(cuda_lib):
    """Prompts into the pages, a verified tree, its accepted path, one more token.

    The same random draws again, through the definitions; a normed row as the kernel stores it, in bf16, and pages as the
    kernel stores them: a key whose norm rounds to the other side, half a bf16 step off, may round to the other side in its
    page too, a step of e4m3 (2^-3) off, which is one of 256 for a few keys of a context: 2^-3 / 16 of a value at most in
    an output that weighs its tokens alike.  Outputs besides: weights 2^-8, their own rounding 2^-8."""
    m = example()
    requests, heads, prompt = 3, 16, 150
    layer, out = m.softmax_round(requests, prompt, heads, seed=5)
    torch.cuda.synchronize()
    assert not layer.status.any().item()
    tree = m.workloads.complete_binary_parents(4)
    N, lengths = len(tree), [max(1, prompt - 37 * r) for r in range(requests)]
    ref = m.SoftmaxLayer(heads, heads // 4, requests, max(lengths) + N + 1, seed=5)
    table = ref.cache._keep[4].cpu().numpy()
    P, d = 64, ref.d
    codes, scales = [np.zeros((table.size, ref.Hkv, P, d), np.uint8) for _ in range(2)], [np.ones((table.size, ref.Hkv)) for _ in range(2)]
    held = [0] * requests

    def project(T):
        x, r = (torch.randn(T, 256, generator=ref.g, device="cuda") for _ in range(2))
        wide = torch.randn(T, (heads + 2 * ref.Hkv) * d, generator=ref.g, device="cuda").bfloat16()
        q, k, v = (f64(w).reshape(T, -1, d) for w in wide.split([heads * d, ref.Hkv * d, ref.Hkv * d], dim=1))
        q, k = (f64(torch.from_numpy(serving_oracle.norm_rotate(w, "rms", 1e-6)).to(torch.bfloat16)) for w in (q, k))
        return q, k, v

    def append(r, k, v):
        for i, x in enumerate((k, v)):
            orc.append(codes[i], scales[i], table[r], held[r], x)
        held[r] += len(k)

    def attend(r, parents, q, k, v):
        ck, cv = (orc.gather(codes[i], scales[i], table[r], held[r]) for i in range(2))
        return orc.attend(q, k, v, parents, ck, cv, ref.scale)

    _, k, v = project(sum(lengths))
    lo = 0
    for r, n in enumerate(lengths):
        append(r, k[lo:lo + n], v[lo:lo + n])
        lo += n
    q, k, v = project(requests * N)
    draft = np.concatenate([attend(r, tree, *(x[r * N:(r + 1) * N] for x in (q, k, v))) for r in range(requests)])
    accepted = torch.randint(-1, N, (requests,), generator=ref.g, device="cuda", dtype=torch.int32).tolist()
    for r, a in enumerate(accepted):
        on = [r * N + i for i in orc.path(tree, a)]
        append(r, k[on], v[on])
    q, k, v = project(requests)
    token = np.concatenate([attend(r, [-1], *(x[r:r + 1] for x in (q, k, v))) for r in range(requests)])
    for got, want in ((out["draft"], draft), (out["token"], token)):
        top = max(np.abs(orc.from_e4m3(codes[1]) * scales[1][..., None, None]).max(), np.abs(v).max())
        assert (np.abs(f64(got) - want) <= (2.0 ** -8 + 2.0 ** -3 / 16) * top + 2.0 ** -8 * np.abs(want)).all()
    for r in range(requests):
        append(r, k[r:r + 1], v[r:r + 1])
    assert layer.length.tolist() == held
