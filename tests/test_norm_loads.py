"""treewy_add_norm may write y over x and the sum over the residual: its kernels read neither by the non-coherent path, which
is defined for memory that nothing writes while the kernel runs."""
import os
import re

from gdn_speculative_tree_gb300 import build


def test_rows_that_may_be_written_are_read_with_plain_loads():
    with open(os.path.join(build.CSRC, "add_norm.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "load_qkv(" not in code                      # reads by __ldg
    assert set(re.findall(r"__ldg\(([^)]*)\)", code)) <= {"a.weight + i"}
    assert "__restrict__" not in code
