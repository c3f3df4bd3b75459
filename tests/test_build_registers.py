"""The chunked kernel's warps exchange registers of its launch, so a build whose launch has another number of them is
refused when it is made, not at the first prompt."""
import os

import pytest

from gdn_speculative_tree_gb300 import build

LOG = """ptxas info    : 77 bytes gmem
ptxas info    : Compiling entry function '_ZN6treewy19extend_chunk_kernelILb0EEEv' for 'sm_103a'
ptxas info    : Function properties for _ZN6treewy19extend_chunk_kernelILb0EEEv
    32 bytes stack frame, 120 bytes spill stores, 152 bytes spill loads
ptxas info    : Used 80 registers, used 2 barriers, 32 bytes cumulative stack size
ptxas info    : Compiling entry function '_ZN6treewy13other_kernelEv' for 'sm_103a'
ptxas info    : Used 126 registers, used 0 barriers
ptxas info    : Compiling entry function '_ZN6treewy19extend_chunk_kernelILb1EEEv' for 'sm_103a'
ptxas info    : Used {} registers, used 2 barriers
"""


def test_the_registers_that_the_kernel_is_compiled_to():
    src = os.path.join(build.CSRC, "extend_chunk.cu")
    build.check_launch_registers(src, LOG.format(80))
    with pytest.raises(RuntimeError, match="72"):
        build.check_launch_registers(src, LOG.format(72))
    with pytest.raises(RuntimeError):
        build.check_launch_registers(src, "")
    build.check_launch_registers(os.path.join(build.CSRC, "slots.cu"), "")  # sources that name no number
