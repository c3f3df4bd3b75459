"""One GDN layer of a server, from a prompt to a verified draft.

Requests bring prompts; their queries and keys are normed, their states made
from the prompts, each request's state is forked to two samples, a draft tree
is verified for every sample and the accepted node committed, and the next
token is taken in without a draft.  Everything runs on one stream, without the
host waiting for the device until the end.

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
    print(f"states  {tuple(layer.pool.shape)} rms {layer.pool.square().mean().sqrt().item():.4f}")


if __name__ == "__main__":
    main()
