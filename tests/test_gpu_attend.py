"""treewy_attend against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from gdn_speculative_tree_gb300 import binding
from tests.cache_helpers import Attend, f64

pytestmark = pytest.mark.gpu

GENERIC = binding.FLAG_FORCE_GENERIC


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("flags", [0, GENERIC])
@pytest.mark.parametrize("kind,nodes", [("chain", [1, 1, 1, 1, 1, 1, 1, 1]), ("chain", [4, 3, 1, 0, 5, 7, 2, 4]),
                                        ("tree", [15, 1, 0, 8, 64, 33, 5, 16]), ("star", [9, 2, 1, 17, 31, 32, 3, 64])])
@pytest.mark.parametrize("d,Hq,Hkv,page", [(128, 4, 2, 64), (256, 16, 2, 64), (64, 5, 5, 16), (80, 6, 2, 32), (256, 8, 1, 128),
                                           (192, 7, 1, 16)])
def test_draft_over_context(cuda_lib, d, Hq, Hkv, page, kind, nodes, flags):
    """Contexts from none to a few tiles, ends inside and on the edges of pages and tiles."""
    a = Attend([0, 1, 15, 128, 129, 300, 17, 255], nodes, Hq=Hq, Hkv=Hkv, d=d, page=page, kind=kind, flags=flags, seed=d + page)
    a.run().check()
    assert not a.status.any()


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("d", [1, 31, 80, 128, 256])
def test_other_types_and_sizes(cuda_lib, d, dtype, out):
    Attend([40, 0, 200], [3, 9, 1], Hq=6, Hkv=2, d=d, page=16, dtype=dtype, out=out, pad=3, seed=d).run().check()


@pytest.mark.parametrize("d", [9, 72, 250])
def test_sizes_beside_the_tensor_cores(cuda_lib, d):
    Attend([40, 0, 200], [3, 9, 1], Hq=6, Hkv=2, d=d, page=32, seed=d).run().check()


@pytest.mark.parametrize("d", [16, 32, 48, 112, 144, 208, 240])
@pytest.mark.parametrize("Hq,Hkv,nodes", [(3, 3, [1, 5, 2]), (48, 1, [5, 1, 3]), (40, 2, [1, 1, 1]), (64, 32, [9, 0, 30])])
def test_every_head_size_and_many_heads(cuda_lib, d, Hq, Hkv, nodes):
    Attend([130, 7, 64], nodes, Hq=Hq, Hkv=Hkv, d=d, page=16, seed=d + Hq).run().check()


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (256, 3)])
@pytest.mark.parametrize("d", [64, 256])
def test_strided_and_unaligned_rows(cuda_lib, d, pad, shift):
    Attend([100, 130], [5, 2], Hq=8, Hkv=2, d=d, page=16, pad=pad, shift=shift).run().check()


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("R,nodes", [(1, 1), (1, 9), (2, 64), (3, 4)])
def test_a_long_context_in_many_pieces(cuda_lib, R, nodes, page):
    Attend([9001 - 1234 * r for r in range(R)], [nodes] * R, Hq=16, Hkv=2, d=128, page=page, seed=page).run().check()


@pytest.mark.parametrize("nodes,max_nodes", [(1, 1), (3, 8), (40, 64)])
def test_many_requests(cuda_lib, nodes, max_nodes):
    """More than the SMs, some without nodes; a bound on the nodes that none reaches."""
    r = np.random.RandomState(nodes)
    R = 400
    lengths = r.randint(0, 400, R)
    counts = np.where(r.rand(R) < 0.2, 0, r.randint(1, nodes + 1, R))
    a = Attend(lengths, counts, Hq=8, Hkv=2, d=64, page=32, max_nodes=max_nodes, max_context=5000, seed=1)
    a.run().check(range(0, R, 17))
    assert not a.status.any()


@pytest.mark.parametrize("d,page,nodes", [(128, 16, 4), (256, 64, 1), (256, 32, 8), (128, 32, 16)])
def test_several_items_of_many_tiles_to_a_piece(cuda_lib, d, page, nodes):
    """Pieces of the work that hold the end of one item, two or three whole ones and the beginning of another."""
    r = np.random.RandomState(d + nodes)
    R = 130
    lengths = np.where(r.rand(R) < 0.1, r.randint(0, 100, R), r.randint(700, 1500, R))
    a = Attend(lengths, r.randint(1, nodes + 1, R), Hq=16, Hkv=4, d=d, page=page, max_nodes=nodes, seed=nodes, quick=True)
    for _ in range(3):
        a.run()
    a.check([0, 50, 129])
    assert not a.status.any()
    b = Attend(lengths, a.nodes, Hq=16, Hkv=4, d=d, page=page, max_nodes=nodes, seed=nodes, flags=GENERIC, quick=True).run()
    # weights to 2^-8, a bf16 output's own rounding on both sides
    assert (a.o.float() - b.o.float()).abs().max() <= 2 * 2.0 ** -7 * b.o.float().abs().max()


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("nodes,Hq,Hkv,R", [(2, 8, 2, 130), (9, 1, 1, 330), (4, 12, 3, 100), (16, 2, 2, 200), (17, 1, 1, 304), (17, 1, 1, 305),
                                            (6, 12, 3, 100), (40, 16, 2, 16), (40, 16, 2, 17), (17, 1, 1, 1024), (17, 1, 1, 1025), (17, 1, 1, 152), (17, 1, 1, 153),
                                            (40, 16, 2, 12), (40, 16, 2, 13)])
def test_on_both_sides_of_every_choice(cuda_lib, d, nodes, Hq, Hkv, R):
    """8, 9, 16, 17 and more rows; tiles in a row, several items to a piece, or an item to a CTA, the
    longest first or in order."""
    r = np.random.RandomState(R)
    a = Attend(r.randint(0, 700, R), r.randint(max(1, nodes // 2), nodes + 1, R), Hq=Hq, Hkv=Hkv, d=d, page=32, max_nodes=nodes,
               max_context=700, seed=R)
    a.run().check(range(0, R, max(13, R // 25)))
    assert not a.status.any()
    first = a.o.clone()
    for _ in range(3):
        assert same(a.run().o, first)


def test_more_requests_than_fit_one_table(cuda_lib):
    r = np.random.RandomState(3)
    R = 3000
    a = Attend(r.randint(0, 40, R), r.randint(0, 3, R), Hq=2, Hkv=1, d=64, page=16, max_context=40, seed=2)
    a.run().check(range(0, R, 97))
    assert not a.status.any()


@pytest.mark.parametrize("flags", [0, GENERIC])
@pytest.mark.parametrize("spread", [2.0, 6.0])
def test_pages_of_very_different_sizes(cuda_lib, spread, flags):
    """Pages whose scales lie far apart: a large page that hardly counts takes no precision from the others."""
    a = Attend([700, 90], [6, 3], Hq=8, Hkv=2, d=128, page=32, flags=flags, spread=spread, seed=5, size=0.02)
    a.run().check()


@pytest.mark.parametrize("flags", [0, GENERIC])
def test_small_values_beside_large_ones_that_are_not_seen(cuda_lib, flags):
    """Values of 2^14 at keys that have no weight: the outputs are as exact as the small values are."""
    a = Attend([512], [2], Hq=4, Hkv=1, d=64, page=64, kind="chain", flags=flags, seed=6)
    # keys of the second page point away from every query, and its values are large
    a.q.copy_(torch.ones_like(a.q) + 0.1 * a.q)
    page = int(a.cache.table_np[0, 1])
    a.cache.k.view(torch.uint8)[page] = 0x80 + 0x50          # -8
    a.cache.ks[page] = 1.0
    a.cache.vs[page] = 2.0 ** 14
    a.run()
    want = f64(a.o)
    ck, cv = a.cache.context(0)
    keep = np.r_[0:64, 128:512]
    from oracle import attend_oracle as orc
    small = orc.attend(f64(a.q), f64(a.k), f64(a.v), a.parents[0], ck[:, keep], cv[:, keep], a.scale)
    # weights to 2^-8 of themselves or 2^-16 of the row's largest (448 tokens), scores and outputs as ever
    assert np.abs(want - small).max() <= (2.0 ** -7 + 448 * 2.0 ** -16) * np.abs(cv[:, keep]).max()


@pytest.mark.parametrize("Hq", [4, 40])
@pytest.mark.parametrize("flags", [0, GENERIC])
def test_many_tokens_that_weigh_next_to_nothing(cuda_lib, flags, Hq):
    """One token with a weight of 1 and 100,000 of 2^-17 each: together they count for 0.76, and their values are alike."""
    n = 100000
    a = Attend([n], [1], Hq=Hq, Hkv=1, d=64, page=128, kind="chain", flags=flags, seed=21)
    a.q.zero_()
    a.q[..., 0] = 8.0
    a.k.zero_()
    a.v.fill_(-1.0)
    a.cache.k.view(torch.uint8).zero_()
    a.cache.v.copy_(torch.ones_like(a.cache.v, dtype=torch.float32))
    a.cache.ks.fill_(1.0)
    a.cache.vs.fill_(1.0)
    a.scale = 1.0
    # 17 ln 2 = 8 * 1.473 in the lone token's favour; its key is bf16, so the weight is that of the key as stored
    a.k[..., 0] = 17 * np.log(2) / 8
    w = np.exp(-8 * float(a.k[0, 0, 0]))
    a.run()
    want = (n * w - 1) / (n * w + 1)
    # weights as small as these to 2^-3 of themselves at worst; of equal ones the error is the same for all
    assert np.abs(f64(a.o) - want).max() <= (2.0 ** -3 * n * w / (n * w + 1) * 2 if flags == 0 else 1e-3) + 2.0 ** -8


@pytest.mark.parametrize("flags", [0, GENERIC])
def test_rising_scores(cuda_lib, flags):
    """Scores that grow along the context, and by much: the running maximum moves in every tile."""
    a = Attend([1500], [3], Hq=4, Hkv=2, d=64, page=16, flags=flags, seed=7)
    for p in range(a.cache.table.shape[1]):
        a.cache.ks[int(a.cache.table_np[0, p])] *= 2.0 ** (p / 16)
    a.cache.ks.copy_(2.0 ** a.cache.ks.log2().round())
    a.run().check()


@pytest.mark.parametrize("flags", [0, GENERIC])
def test_scales_that_are_no_powers_of_two(cuda_lib, flags):
    a = Attend([300, 20], [3, 7], Hq=4, Hkv=2, d=128, page=32, flags=flags, seed=8)
    a.cache.ks *= 0.7
    a.cache.vs *= 1.3
    a.run().check()


@pytest.mark.parametrize("flags", [0, GENERIC])
def test_no_numbers_reach_only_who_sees_them(cuda_lib, flags):
    """A NaN key in one request's context, a NaN value in another's, an infinite key of a node with a sibling."""
    a = Attend([100, 100, 100, 0], [2, 2, 3, 2], Hq=4, Hkv=2, d=64, page=32, kind="star", flags=flags, seed=9)
    page = a.cache.table_np
    a.cache.k.view(torch.uint8)[int(page[0, 1]), 0, 3, 5] = 127
    a.cache.v.view(torch.uint8)[int(page[1, 2]), 1, 7, 9] = 255
    a.k[a.off[2] + 1, 0, 0] = float("inf")
    a.v[a.off[3], 1, 2] = float("nan")
    a.run()
    bad = torch.isnan(a.o.float())
    want = torch.zeros_like(bad)
    want[a.off[0]:a.off[1], :2] = True
    want[a.off[1]:a.off[2], 2:, 9] = True
    want[a.off[2] + 1, :2] = True
    want[a.off[3], 2:, 2] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("flags", [0, GENERIC])
def test_refused_requests_leave_the_others_alone(cuda_lib, flags):
    lengths, nodes = [300] * 8, [4] * 8
    good = Attend(lengths, nodes, flags=flags, seed=10).run()
    a = Attend(lengths, nodes, flags=flags, seed=10)
    a.cache.table[1, 4] = a.cache.k.shape[0]       # the last page of the context
    a.cache.table[2, 0] = -1
    a.parent[a.off[3] + 2] = 2
    a.cache.length[4] = -1
    a.cache.length[5] = 100000
    a.cache.table[6, 2] = -(1 << 31)
    a.run()
    B = binding
    assert a.status.tolist() == [0, B.STATUS_BAD_PAGE, B.STATUS_BAD_PAGE, B.STATUS_BAD_TREE, B.STATUS_BAD_PAGE,
                                 B.STATUS_BAD_PAGE, B.STATUS_BAD_PAGE, 0]
    for r in (0, 7):
        assert same(a.o[a.off[r]:a.off[r + 1]], good.o[a.off[r]:a.off[r + 1]])
    assert (a.o[a.off[1]:a.off[7]] == -7).all()


@pytest.mark.parametrize("flags", [0, GENERIC])
def test_bad_offsets_and_bounds(cuda_lib, flags):
    # chains without parents: rows that move to another request stay a tree
    a = Attend([50] * 5, [3] * 5, kind="chain", null_parent=True, flags=flags, seed=11, max_nodes=3, max_context=49)
    a.run()
    assert a.status.tolist() == [binding.STATUS_BAD_PAGE] * 5 and (a.o == -7).all()
    a.status.zero_()
    a.more["max_context"] = 50
    a.node_offset.copy_(torch.tensor([0, 3, 7, 5, 8, 99], dtype=torch.int32))  # four nodes, minus two, three, past the end
    a.run()
    got = a.status.tolist()
    assert got[0] == 0 and got[3] == 0
    assert got[1] == got[2] == binding.STATUS_TOO_MANY_NODES and got[4] & binding.STATUS_BAD_TREE
    assert (a.o[3:5] == -7).all() and (a.o[8:] == -7).all()


@pytest.mark.parametrize("flags", [0, GENERIC])
def test_shared_pages(cuda_lib, flags):
    """Two requests on one prefix."""
    a = Attend([128, 150], [2, 5], Hq=8, Hkv=2, d=64, page=64, flags=flags, seed=12)
    a.cache.table[1, :2] = a.cache.table[0, :2]
    a.run().check()


def test_pages_behind_four_gigabytes(cuda_lib):
    """Codes whose offset passes 32 bits."""
    d, Hkv, P = 256, 8, 128
    num = (1 << 32) // (Hkv * P * d) + 40
    a = Attend([300, 60], [2, 1], Hq=8, Hkv=Hkv, d=d, page=P, seed=13)
    small, far = a.cache.table_np.copy(), a.cache.table_np.copy()
    far[far >= 0] = num - 1 - far[far >= 0]
    for name in ("k", "v", "ks", "vs"):
        x = getattr(a.cache, name)
        big = torch.zeros((num,) + x.shape[1:], dtype=x.dtype if name in ("ks", "vs") else torch.uint8, device="cuda")
        for i, j in zip(small[small >= 0], far[far >= 0]):
            big[int(j)] = x.view(big.dtype)[int(i)]
        setattr(a.cache, name, big.view(x.dtype))
    a.cache.table = torch.from_numpy(far).cuda()
    near = Attend([300, 60], [2, 1], Hq=8, Hkv=Hkv, d=d, page=P, seed=13).run()
    a.run()
    assert same(a.o, near.o)


@pytest.mark.parametrize("case", [dict(lengths=[5000], nodes=[1]), dict(lengths=[3000, 200, 0], nodes=[30, 64, 7]),
                                  dict(lengths=[700] * 90, nodes=[64] * 90)])
def test_same_bits_every_time(cuda_lib, case):
    runs = [Attend(**case, Hq=16, Hkv=2, d=256, seed=14).run() for _ in range(3)]
    assert all(same(x.o, runs[0].o) for x in runs[1:])


@pytest.mark.parametrize("flags", [0, GENERIC])
def test_graph_on_another_stream_with_other_contents(cuda_lib, flags):
    """A captured call, replayed with other lengths, pages, queries and trees in the same tensors."""
    kw = dict(Hq=8, Hkv=2, d=128, page=32, flags=flags, max_context=1500, max_nodes=9)
    a = Attend([1500, 3, 200], [4, 9, 1], seed=15, **kw)
    call = a.make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        binding.treewy_attend(call)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        binding.treewy_attend(call)
    graph.replay()
    torch.cuda.synchronize()
    a.check()
    b = Attend([1, 1400, 700], [2, 3, 9], seed=16, kind="star", **kw)
    assert b.cache.k.shape[0] > a.cache.k.shape[0] and b.cache.table.shape[1] <= a.cache.table.shape[1]
    b.cache.table_np = np.where(b.cache.table_np >= 0, np.arange(b.cache.table_np.size).reshape(b.cache.table_np.shape) % a.cache.k.shape[0], -1)
    c = b.cache
    table = np.full(tuple(a.cache.table.shape), -1, np.int32)
    table[:, :c.table_np.shape[1]] = c.table_np
    # the second problem's lengths, rows and tree over the first one's pages (those that its own contexts use)
    used = sorted(set(a.cache.table_np[a.cache.table_np >= 0].tolist()))
    full = [p for i, n in enumerate(a.cache.lengths) for p in a.cache.table_np[i, :n // 32].tolist()]
    for r, n in enumerate(b.cache.lengths):
        table[r, :-(-n // 32)] = [full[(7 * r + i) % len(full)] for i in range(-(-n // 32))]
    assert used
    a.cache.table.copy_(torch.from_numpy(table))
    a.cache.lengths = b.cache.lengths
    a.cache.length.copy_(b.cache.length)
    a.q[:14].copy_(b.q), a.k[:14].copy_(b.k), a.v[:14].copy_(b.v)
    a.parent[:14].copy_(b.parent)
    a.node_offset.copy_(b.node_offset)
    a.off, a.nodes, a.parents = b.off, b.nodes, b.parents
    graph.replay()
    torch.cuda.synchronize()
    a.check()
    assert not a.status.any()


def test_bounds_as_large_as_they_go(cuda_lib):
    """The largest bound on the contexts, and the largest on the nodes, for small ones; a table of one empty page each."""
    for kw in (dict(Hq=4, Hkv=2), dict(Hq=32, Hkv=2), dict(Hq=4, Hkv=2, flags=GENERIC)):
        Attend([33, 200, 0], [2, 1, 3], d=64, page=32, max_context=(1 << 31) - 1, max_nodes=64, seed=22, **kw).run().check()
        a = Attend([0, 0], [3, 1], d=64, page=32, max_context=(1 << 31) - 1, seed=23, **kw)
        a.cache.table = a.cache.table[:, :0].contiguous()
        a.run().check()


@pytest.mark.parametrize("Hq", [4, 64])
def test_no_rows_at_all(cuda_lib, Hq):
    """Requests without a node, with contexts; and one whose length is refused all the same."""
    a = Attend([100, 20], [0, 0], Hq=Hq, Hkv=2, d=64, page=32, max_nodes=4)
    a.cache.length[1] = -5
    a.run()
    assert a.status.tolist() == [0, binding.STATUS_BAD_PAGE]


def test_two_calls_at_once(cuda_lib):
    """Two streams, each with its own workspace."""
    a, b = (Attend([4000, 800], [4, 60], Hq=16, Hkv=2, d=256, seed=s) for s in (17, 18))
    ca, cb = a.make(), b.make()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        binding.treewy_attend(ca, one)
        binding.treewy_attend(cb, two)
    torch.cuda.synchronize()
    a.check(), b.check()


def test_chains_need_no_parents(cuda_lib):
    a = Attend([90, 30], [5, 3], kind="chain", null_parent=True, seed=19).run().check()
    b = Attend([90, 30], [5, 3], kind="chain", seed=19).run()
    assert same(a.o, b.o)


def test_workspace_of_any_contents(cuda_lib):
    a = Attend([6000, 17], [3, 8], Hq=16, Hkv=2, d=128, seed=20)
    outs = []
    for fill in (0, 255, 127):
        n = binding.treewy_attend_workspace(a.make())
        a.more["workspace"] = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        a.o.fill_(-7)
        a.run().check()
        outs.append(a.o.clone())
    assert same(outs[0], outs[1]) and same(outs[0], outs[2])
