"""Moves of a slot onto itself, by hand and on the GPU: they do nothing, whatever else the list does with the slot."""
import numpy as np
import pytest

from oracle import serving_oracle as orc

LISTS = [([3, 4], [4, 4]), ([4, 3], [4, 4]), ([4, -1], [4, 4]), ([-1, 4], [4, 4]), ([4, 4], [2, 4]), ([4, 4, 1], [4, 4, 4])]


@pytest.mark.parametrize("src,dst", LISTS)
def test_a_move_onto_itself_writes_nothing(src, dst):
    pool = np.arange(1.0, 7.0).reshape(1, 6, 1)
    want = pool.copy()
    for s, d in zip(src, dst):  # at most one of them is a real move
        if s != d:
            want[:, d] = pool[:, s] if s >= 0 else 0
    out, status = orc.move_slots(pool, src, dst)
    assert not status.any()
    np.testing.assert_array_equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("src,dst", LISTS)
def test_a_move_onto_itself_on_the_gpu(cuda_lib, src, dst):
    from tests.test_gpu_serving import slots_case
    assert not slots_case(src, dst).any()
