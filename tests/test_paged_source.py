"""What the sources of the paged cache's kernels must not contain."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bwd_sparse_mqa_gb300", "csrc")
FILES = ["smqa_paged.cu", "smqa_paged.cuh", "smqa_paged_fwd.cu"]


def _code(name):
    """The file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", FILES)
def test_no_loads_through_the_read_only_path(name):
    """These kernels start beside the one before, whose writes they read once it has ended:
    __ldg and ld.global.nc are defined only for data that nothing writes while the kernel lives."""
    code = _code(name)
    assert "__ldg" not in code and ".nc." not in code and "__restrict__" not in code


@pytest.mark.parametrize("name", FILES)
def test_no_error_is_kept_between_calls(name):
    """A call that failed once (no memory, a busy device) must not decide the next: statics hold
    what succeeded, never an error code."""
    assert not re.search(r"static\s+(const\s+)?cudaError_t\s+\w+\s*(=|\{)", _code(name))
