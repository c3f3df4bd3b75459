"""The workspace that make_attn makes, which the caller does not see, where a call runs on another stream than the one it was
made on: it is not given away while that stream still works with it."""
import pytest
import torch

from gdn_speculative_tree_gb300 import binding
from tests.cache_helpers import Attend

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def warm(cuda_lib):
    """What the first calls of a process load is loaded before a test counts on their times."""
    Attend([9000], [4], Hq=16, Hkv=2, d=128, seed=40).run()
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()


def left_alone(call_on):
    """Whether the memory of a structure that is gone stays taken until the side stream has run its call."""
    a = Attend([9000], [4], Hq=16, Hkv=2, d=128, seed=41)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = a.make()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # a fifth of a second
    call_on(call, side)
    size, where = call.workspace_bytes, call.workspace
    del call
    taken = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    busy = not side.query()
    early = any(x.data_ptr() == where for x in taken)
    torch.cuda.synchronize()
    a.check()
    assert busy, "the side stream was done too soon to say"
    return not early


def test_a_stream_object(cuda_lib):
    assert left_alone(lambda call, side: binding.treewy_attend(call, side))


def test_a_stream_handle(cuda_lib):
    assert left_alone(lambda call, side: binding.treewy_attend(call, side.cuda_stream))


def test_the_current_stream(cuda_lib):
    def run(call, side):
        with torch.cuda.stream(side):
            binding.treewy_attend(call)
    assert left_alone(run)


def test_made_on_another_stream_and_run_on_the_default_one(cuda_lib):
    a = Attend([9000], [4], Hq=16, Hkv=2, d=128, seed=42)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call = a.make()
    torch.cuda._sleep(400_000_000)
    binding.treewy_attend(call, 0)
    size, where = call.workspace_bytes, call.workspace
    del call
    with torch.cuda.stream(side):
        taken = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    busy, early = not torch.cuda.default_stream().query(), any(x.data_ptr() == where for x in taken)
    torch.cuda.synchronize()
    a.check()
    assert busy and not early


def test_a_graph_of_a_call_made_outside_it(cuda_lib):
    a = Attend([3000, 100], [4, 9], Hq=16, Hkv=2, d=128, seed=43)
    call, graph, side = a.make(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        binding.treewy_attend(call)
    for _ in range(2):
        a.o.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        a.check()


def test_one_structure_on_several_streams(cuda_lib):
    """In turn, back again, and in a graph; each stream has a workspace of its own and the same one every time."""
    a = Attend([5000, 100], [4, 9], Hq=16, Hkv=2, d=128, seed=44)
    call, streams = a.make(), [torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    used, first = [], None
    for stream in streams + streams:
        a.o.fill_(-7.0)
        torch.cuda.synchronize()
        binding.treewy_attend(call, stream)
        torch.cuda.synchronize()
        used.append(call.workspace)
        a.check()
        first = a.o.clone() if first is None else first
        assert torch.equal(a.o.view(torch.uint8), first.view(torch.uint8))
    assert used[:3] == used[3:] and len(set(used)) == 3
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        binding.treewy_attend(call)
    binding.treewy_attend(call)
    a.o.fill_(-7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.o.view(torch.uint8), first.view(torch.uint8))


def test_a_workspace_of_the_callers_is_the_one_that_is_used(cuda_lib):
    a = Attend([5000], [4], Hq=16, Hkv=2, d=128, seed=45)
    mine = torch.empty(binding.treewy_attend_workspace(a.make()), dtype=torch.uint8, device="cuda")
    call = a.make(workspace=mine)
    torch.cuda.synchronize()
    binding.treewy_attend(call, torch.cuda.Stream())
    torch.cuda.synchronize()
    assert call.workspace == mine.data_ptr()
    a.check()
