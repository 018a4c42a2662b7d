"""The sizes of fp8_paths.py take the kernels that they are listed under."""
import pytest

import fp8_paths as paths


@pytest.mark.parametrize("name", paths.PATHS)
def test_sizes_take_their_kernel(name):
    counts, n, k, dtype = paths.PATHS[name]
    assert paths.kernel(sum(counts), len(counts), n, k, dtype) == name
