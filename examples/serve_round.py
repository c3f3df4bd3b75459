"""One GDN layer of a server, from a prompt to a verified draft; and the softmax
layer of a hybrid behind it.

Requests bring prompts; their queries and keys are normed, their states made
from the prompts, each request's state is forked to two samples, a draft tree
is verified for every sample and the accepted node committed, and the next
token is taken in without a draft.  The softmax layer norms the residual
stream's rows into 8 bits, takes the prompts' keys and values into pages of 8
bits, verifies the same tree against them and takes the accepted path.  (What a
prompt's own tokens attend to is left to the server's prompt attention.)
Everything runs on one stream, without the host waiting for the device until
the end.

    python examples/serve_round.py [--requests 4] [--prompt 300] [--heads 8]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from gdn_speculative_tree_gb300 import binding, workloads  # noqa: E402


class Layer:
    """A layer's heads and its pool of states, one slot per sample."""

    def __init__(self, H: int, Hk: int, slots: int, d: int = 128, seed: int = 0):
        self.H, self.Hk, self.d = H, Hk, d
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = torch.zeros(slots, H, d, d, device="cuda")

    def project(self, T: int):
        """T tokens' rows of a fused projection (random here): q, k, v as slices
        of it, and the gates."""
        wide = torch.randn(T, (2 * self.Hk + self.H) * self.d, generator=self.g, device="cuda").bfloat16()
        q, k, v = wide.split([self.Hk * self.d, self.Hk * self.d, self.H * self.d], dim=1)
        alpha = 0.9 + 0.099 * torch.rand(T, self.H, generator=self.g, device="cuda")
        beta = torch.sigmoid(torch.randn(T, self.H, generator=self.g, device="cuda"))
        return (q.view(T, self.Hk, self.d), k.view(T, self.Hk, self.d), v.view(T, self.H, self.d), alpha, beta)

    def normed(self, q, k, repeat: int = 1):
        """q and k with unit rows, q scaled by 1/sqrt(d); `repeat` shows every
        key head to that many value heads."""
        T = q.shape[0]
        qo = torch.empty(T, self.Hk * repeat, self.d, device="cuda", dtype=q.dtype)
        ko = torch.empty_like(qo)
        binding.treewy_qk_norm(binding.make_qk(q=q, k=k, q_out=qo, k_out=ko, norm="l2", q_scale=self.d ** -0.5))
        return qo, ko

    def extend(self, lengths, slots, fresh: bool):
        """New tokens of one sequence per slot; returns their outputs and the status."""
        T, R = sum(lengths), len(lengths)
        q, k, v, alpha, beta = self.project(T)
        q, k = self.normed(q, k)
        off = torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32, device="cuda")
        o = torch.empty(T, self.H, self.d, device="cuda", dtype=torch.bfloat16)
        status = torch.zeros(R, dtype=torch.int32, device="cuda")
        seqs = binding.make_seqs(seq_offset=off, q=q, k=k, v=v, alpha=alpha, beta=beta, state=self.pool,
                                 state_slot=slots, fresh=torch.full((R,), int(fresh), dtype=torch.uint8, device="cuda"),
                                 o=o, status=status, max_len=max(lengths))
        binding.treewy_extend(seqs)
        return o, status

    def fork(self, src, dst):
        status = torch.zeros(src.numel(), dtype=torch.int32, device="cuda")
        binding.treewy_copy_slots(binding.make_slots(state=self.pool, src=src, dst=dst, status=status))
        return status

    def verify_and_commit(self, parents, slots, accepted):
        """One draft tree per slot verified, and node `accepted` of each committed."""
        R, N = slots.numel(), len(parents)
        T = R * N
        q, k, v, alpha, beta = self.project(T)
        q, k = self.normed(q, k, repeat=self.H // self.Hk)  # a row per value head
        off = torch.arange(0, T + 1, N, dtype=torch.int32, device="cuda")
        o = torch.empty(T, self.H, self.d, device="cuda")
        U, status = torch.empty_like(o), torch.zeros(R, dtype=torch.int32, device="cuda")
        batch = binding.make_batch(
            node_offset=off, parent=torch.as_tensor(parents, dtype=torch.int32).repeat(R).cuda(), q=q, k=k,
            v=v.contiguous(), alpha=alpha, beta=beta, state=self.pool, state_slot=slots, o=o, U=U, status=status,
            max_nodes=N)
        binding.treewy_verify(batch)
        binding.treewy_commit(batch, accepted)
        return o, status


class SoftmaxLayer:
    """A softmax layer's heads and its 8-bit pages of keys and values, one row of the page table per request."""

    def __init__(self, Hq: int, Hkv: int, requests: int, most: int, d: int = 128, page: int = 64, seed: int = 0):
        self.Hq, self.Hkv, self.d, self.most, self.scale = Hq, Hkv, d, most, d ** -0.5
        self.g = torch.Generator(device="cuda").manual_seed(seed + 100)
        width = -(-most // page)
        codes = torch.zeros(2, requests * width, Hkv, page, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        scales = torch.ones(2, requests * width, Hkv, device="cuda")
        table = torch.randperm(requests * width, generator=self.g, device="cuda").to(torch.int32).view(requests, width)
        self.length, self.after = (torch.zeros(requests, dtype=torch.int32, device="cuda") for _ in range(2))
        self.status = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.cache = binding.make_cache(k=codes[0], v=codes[1], k_scale=scales[0], v_scale=scales[1], page_table=table,
                                        length=self.length)

    def project(self, T: int, hidden: int = 256):
        """T tokens: the residual stream's rows normed into 8 bits for the projection, whose rows (random here) come back."""
        x, residual = (torch.randn(T, hidden, generator=self.g, device="cuda").bfloat16() for _ in range(2))
        rows = torch.empty(T, hidden, device="cuda", dtype=torch.float8_e4m3fn)
        scales = torch.empty(T, hidden // 128, device="cuda")
        binding.treewy_add_norm(binding.make_norm(x=x, residual=residual, residual_out=residual, y8=rows, y8_scale=scales,
                                                  group=128))
        wide = torch.randn(T, (self.Hq + 2 * self.Hkv) * self.d, generator=self.g, device="cuda").bfloat16()
        q, k, v = wide.split([self.Hq * self.d, self.Hkv * self.d, self.Hkv * self.d], dim=1)
        q, k, v = q.view(T, self.Hq, self.d), k.view(T, self.Hkv, self.d), v.view(T, self.Hkv, self.d)
        qo, ko = (torch.empty(x.shape, device="cuda", dtype=x.dtype) for x in (q, k))
        binding.treewy_qk_norm(binding.make_qk(q=q, k=k, q_out=qo, k_out=ko, norm="rms"))
        return qo, ko, v

    def append(self, off, k, v, most: int, parent=None, accepted=None):
        binding.treewy_append(binding.make_append(cache=self.cache, node_offset=off, parent=parent, accepted=accepted, k=k, v=v,
                                                  new_length=self.after, status=self.status, max_new=most))
        self.length.copy_(self.after)

    def attend(self, off, parent, q, k, v, most: int):
        o = torch.empty(q.shape, device="cuda", dtype=q.dtype)
        binding.treewy_attend(binding.make_attn(cache=self.cache, node_offset=off, parent=parent, q=q, k=k, v=v, o=o,
                                                status=self.status, scale=self.scale, max_nodes=most, max_context=self.most))
        return o


def softmax_round(requests: int = 4, prompt: int = 300, heads: int = 8, seed: int = 0):
    """Prompts, a verified tree with its accepted path, and a single token; returns the layer and its outputs by step."""
    tree = workloads.complete_binary_parents(4)
    lengths = [max(1, prompt - 37 * r) for r in range(requests)]
    layer = SoftmaxLayer(heads, max(1, heads // 4), requests, max(lengths) + len(tree) + 1, seed=seed)

    def offsets(n):
        return torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32, device="cuda")

    _, k, v = layer.project(sum(lengths))
    layer.append(offsets(lengths), k, v, max(lengths))
    out, off, N = {}, offsets([len(tree)] * requests), len(tree)
    parent = torch.as_tensor(tree, dtype=torch.int32).repeat(requests).cuda()
    q, k, v = layer.project(requests * N)
    out["draft"] = layer.attend(off, parent, q, k, v, N)
    accepted = torch.randint(-1, N, (requests,), generator=layer.g, device="cuda", dtype=torch.int32)
    layer.append(off, k, v, N, parent, accepted)
    q, k, v = layer.project(requests)
    out["token"] = layer.attend(offsets([1] * requests), None, q, k, v, 1)
    layer.append(offsets([1] * requests), k, v, 1)
    return layer, out


def run(requests: int = 4, prompt: int = 300, heads: int = 8, seed: int = 0):
    """One round; returns the layer, its outputs by step and every status word."""
    layer = Layer(heads, max(1, heads // 2), 2 * requests, seed=seed)
    first = torch.arange(requests, dtype=torch.int32, device="cuda")
    second = first + requests
    every = torch.cat([first, second])
    lengths = [max(1, prompt - 37 * r) for r in range(requests)]
    out, status = {}, []
    out["prompt"], s = layer.extend(lengths, first, fresh=True)
    status.append(s)
    status.append(layer.fork(first, second))
    tree = workloads.complete_binary_parents(4)
    accepted = torch.randint(-1, len(tree), (2 * requests,), generator=layer.g, device="cuda", dtype=torch.int32)
    out["draft"], s = layer.verify_and_commit(tree, every, accepted)
    status.append(s)
    out["token"], s = layer.extend([1] * (2 * requests), every, fresh=False)
    status.append(s)
    return layer, out, torch.cat(status)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--heads", type=int, default=8)
    a = ap.parse_args()
    layer, out, status = run(a.requests, a.prompt, a.heads)
    torch.cuda.synchronize()
    assert not status.any().item(), status.tolist()
    for step, o in out.items():
        print(f"{step:7s} {tuple(o.shape)} rms {o.float().square().mean().sqrt().item():.4f}")
    softmax, out = softmax_round(a.requests, a.prompt, a.heads)
    torch.cuda.synchronize()
    assert not softmax.status.any().item(), softmax.status.tolist()
    for step, o in out.items():
        print(f"softmax layer, {step:7s} {tuple(o.shape)} rms {o.float().square().mean().sqrt().item():.4f}")
    print(f"states  {tuple(layer.pool.shape)} rms {layer.pool.square().mean().sqrt().item():.4f}")


if __name__ == "__main__":
    main()
