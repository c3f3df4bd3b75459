"""treewy_append against the definition: codes, scales and lengths bit for bit."""
import numpy as np
import pytest
import torch

from gdn_speculative_tree_gb300 import binding
from oracle import attend_oracle as orc
from tests.cache_helpers import TYPES, Cache, f64, rows, trees

pytestmark = pytest.mark.gpu


class Append:
    def __init__(self, lengths, nodes, *, accepted=None, Hkv=2, d=128, page=64, kind="tree", dtype="bf16", pad=0, shift=0,
                 seed=0, size=1.0, max_new=None, null_parent=False):
        g = torch.Generator().manual_seed(seed)
        self.cache = Cache(lengths, Hkv, d, page, room=max([1] + list(nodes)), seed=seed)
        self.off = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        T = int(self.off[-1])
        self.parents = trees(nodes, kind, seed)
        self.parent = None if null_parent else torch.from_numpy(np.concatenate([np.zeros(0)] + self.parents).astype(np.int32)).cuda()
        self.accepted = None if accepted is None else torch.tensor(accepted, dtype=torch.int32, device="cuda")
        self.node_offset = torch.from_numpy(self.off).cuda()
        self.k, self.v = (rows(T, Hkv, d, TYPES[dtype], pad, g, size, shift) for _ in range(2))
        self.new_length = torch.full((len(nodes),), -5, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(len(nodes), dtype=torch.int32, device="cuda")
        self.max_new = max([0] + list(nodes)) if max_new is None else max_new

    def taken(self, r):
        if self.accepted is None:
            return list(range(self.off[r + 1] - self.off[r]))
        return orc.path(self.parents[r], int(self.accepted[r]))

    def expect(self, skip=()):
        """What the pool holds afterwards."""
        c = self.cache
        out = []
        for codes, scale, x in ((c.k, c.ks, self.k), (c.v, c.vs, self.v)):
            codes, scale, x = codes.cpu().view(torch.uint8).numpy().copy(), f64(scale), f64(x)
            for r in range(len(c.lengths)):
                if r not in skip:
                    orc.append(codes, scale, c.table_np[r], c.lengths[r], x[self.off[r] + np.array(self.taken(r), np.int64)])
            out += [codes, scale]
        return out

    def make(self):
        return binding.make_append(cache=self.cache.made(), node_offset=self.node_offset, parent=self.parent,
                                   accepted=self.accepted, k=self.k, v=self.v, new_length=self.new_length, status=self.status,
                                   max_new=self.max_new)

    def run(self, skip=()):
        want = self.expect(skip)
        binding.treewy_append(self.make())
        torch.cuda.synchronize()
        c = self.cache
        got = [c.k.cpu().view(torch.uint8).numpy(), f64(c.ks), c.v.cpu().view(torch.uint8).numpy(), f64(c.vs)]
        for name, x, y in zip(("k", "k_scale", "v", "v_scale"), got, want):
            assert np.array_equal(x, y), (name, np.argwhere(x != y)[:5])
        for r in range(len(c.lengths)):
            want_n = -5 if r in skip else c.lengths[r] + len(self.taken(r))
            assert int(self.new_length[r]) == want_n
        return self


@pytest.mark.parametrize("dtype,pad,shift", [("bf16", 0, 0), ("bf16", 8, 0), ("bf16", 3, 1), ("f32", 0, 0), ("f32", 1, 0)])
@pytest.mark.parametrize("d,Hkv,page", [(128, 2, 64), (256, 1, 128), (64, 3, 16), (80, 2, 32), (7, 2, 16)])
def test_rows_in_order(cuda_lib, d, Hkv, page, dtype, pad, shift):
    """None, one, a page's end, several pages; into empty and half full pages."""
    a = Append([0, 5, page, page - 1, 3 * page + 7, 0, 1], [1, 0, 3, 2 * page, page - 7, 5 * page + 1, 200], Hkv=Hkv, d=d, page=page,
               dtype=dtype, pad=pad, shift=shift, seed=d).run()
    assert not a.status.any()


@pytest.mark.parametrize("kind,null_parent", [("tree", False), ("chain", False), ("chain", True), ("star", False)])
@pytest.mark.parametrize("page", [16, 64])
def test_accepted_paths(cuda_lib, page, kind, null_parent):
    nodes = [1, 4, 64, 15, 33, 0, 8]
    accepted = [0, -1, 63, 7, 32, -1, 3]
    a = Append([0, 30, 63, 64, 100, 9, 15], nodes, accepted=accepted, page=page, kind=kind, null_parent=null_parent, seed=1).run()
    assert not a.status.any()


@pytest.mark.parametrize("size", [1e-20, 1e-4, 30.0, 1e6, 1e30])
def test_a_scale_that_grows_and_one_that_does_not(cuda_lib, size):
    """Tokens much smaller and much larger than those that the pages hold."""
    Append([5, 70, 0, 127], [3, 60, 9, 1], page=64, d=64, size=size, seed=2).run()


def test_no_numbers_are_stored_as_such(cuda_lib):
    a = Append([3, 0], [4, 2], d=64, page=16, seed=3)
    a.k[1, 0, 5] = float("nan")
    a.k[2, 1, 0] = float("inf")
    a.v[0, 0, 63] = -float("inf")
    a.v[5, 0] = float("nan")   # a whole row, in a page of its own numbers
    want = a.expect()
    binding.treewy_append(a.make())
    torch.cuda.synchronize()
    c = a.cache
    for got, ref in ((c.k, want[0]), (c.v, want[2])):
        got = got.cpu().view(torch.uint8).numpy()
        assert ((got == ref) | ((got & 127 == 127) & (ref & 127 == 127))).all()
    assert np.array_equal(f64(c.ks), want[1]) and np.array_equal(f64(c.vs), want[3])


def test_refused_requests_leave_everything_alone(cuda_lib):
    B = binding
    nodes = [4] * 8
    a = Append([20] * 8, nodes, accepted=[3, 4, -2, 2, 1, 0, 3, 1], kind="chain", page=16, d=64, seed=4)
    a.parent[a.off[3] + 1] = 1                      # its own parent
    a.cache.table[4, 1] = a.cache.k.shape[0]
    a.cache.length[5] = -1
    a.cache.length[6] = a.cache.table.shape[1] * 16 - 2  # room for two
    a.run(skip=range(1, 7))
    assert a.status.tolist() == [0, B.STATUS_BAD_ACCEPTED, B.STATUS_BAD_ACCEPTED, B.STATUS_BAD_TREE, B.STATUS_BAD_PAGE,
                                 B.STATUS_BAD_PAGE, B.STATUS_BAD_PAGE, 0]


def test_bad_offsets(cuda_lib):
    a = Append([20] * 4, [3] * 4, page=16, d=64, seed=5)
    a.node_offset.copy_(torch.tensor([0, 3, 7, 6, 90], dtype=torch.int32))
    a.run(skip=(1, 2, 3))
    got = a.status.tolist()
    assert got[0] == 0 and got[1] == got[2] == binding.STATUS_TOO_MANY_NODES and got[3] & binding.STATUS_BAD_TREE


def test_a_full_table_of_a_long_prompt(cuda_lib):
    """Several hundred pages of one request, one of them bad: nothing is written."""
    a = Append([7], [6000], page=16, d=64, Hkv=1, seed=6).run()
    b = Append([7], [6000], page=16, d=64, Hkv=1, seed=6)
    b.cache.table[0, 300] = -3
    b.run(skip=(0,))
    assert b.status.tolist() == [binding.STATUS_BAD_PAGE] and not a.status.any()


def test_token_by_token_is_what_one_call_is(cuda_lib):
    """A page filled by single calls holds what the largest token so far allows; values that need no new scale are the same."""
    a = Append([0], [40], page=16, d=64, seed=7)
    a.k[0, :, 0] = 100.0
    a.k[16, :, 0] = 100.0
    a.k[32, :, 0] = 100.0
    a.v.copy_(a.k)
    b = Append([0], [1], page=16, d=64, seed=8)
    b.cache = Cache([0], 2, 64, 16, room=40, seed=7)
    a.run()
    for t in range(40):
        b.k.copy_(a.k[t:t + 1])
        b.v.copy_(a.v[t:t + 1])
        b.cache.length.fill_(t)
        binding.treewy_append(b.make())
    torch.cuda.synchronize()
    for x, y in ((a.cache.k, b.cache.k), (a.cache.v, b.cache.v), (a.cache.ks, b.cache.ks), (a.cache.vs, b.cache.vs)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_graph_replays_with_other_lengths(cuda_lib):
    a = Append([10, 100], [5, 9], accepted=[4, 2], page=32, d=128, seed=9)
    call = a.make()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    keep = a.cache.k.clone(), a.cache.v.clone(), a.cache.ks.clone(), a.cache.vs.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        binding.treewy_append(call)
    a.cache.length.copy_(torch.tensor([11, 97]))
    a.cache.lengths = [11, 97]
    a.accepted.copy_(torch.tensor([3, 8]))
    # what the pages hold behind the first lengths is whatever it was
    for x, y in zip((a.cache.k, a.cache.v, a.cache.ks, a.cache.vs), keep):
        x.copy_(y)
    want = a.expect()
    graph.replay()
    torch.cuda.synchronize()
    got = [a.cache.k.cpu().view(torch.uint8).numpy(), f64(a.cache.ks), a.cache.v.cpu().view(torch.uint8).numpy(), f64(a.cache.vs)]
    assert all(np.array_equal(x & 127 if x.dtype == np.uint8 else x, y & 127 if y.dtype == np.uint8 else y) for x, y in zip(got, want))


def test_no_rows(cuda_lib):
    Append([10, 20], [0, 0], seed=10).run()
    Append([10, 20], [3, 2], accepted=[-1, -1], seed=10).run()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page,rows,R", [(256, 64, 600, 12), (64, 128, 1500, 40), (256, 16, 300, 30), (128, 64, 63, 600)])
def test_many_pages_one_after_the_other(cuda_lib, d, page, rows, R, dtype):
    """Prompts of several groups of pages, some of them short: CTAs that take more than one page."""
    r = np.random.RandomState(d + rows)
    lengths = r.randint(0, 3 * page, R)
    nodes = np.where(r.rand(R) < 0.3, r.randint(0, page, R), r.randint(rows // 2, rows + 1, R))
    a = Append(lengths, nodes, Hkv=2, d=d, page=page, dtype=dtype, seed=11, max_new=rows).run()
    assert not a.status.any()
