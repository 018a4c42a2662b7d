"""Files that can be run: what they run is defined before it."""
import ast
import os

import pytest

from conftest import ROOT

SCRIPTS = ["__graft_entry__.py", "bench.py", "examples/decode_step.py", "examples/fp8_layer.py",
           "block_scaled_fp4_05_amd/build.py"]


@pytest.mark.parametrize("path", SCRIPTS)
def test_nothing_is_defined_behind_the_main_block(path):
    with open(os.path.join(ROOT, path)) as f:
        body = ast.parse(f.read()).body
    main = [i for i, node in enumerate(body) if isinstance(node, ast.If) and "__main__" in ast.dump(node.test)]
    assert main == [len(body) - 1]
