"""The example that runs the cache's operators together with the indexer."""
import os
import sys

import pytest

from gpu_helpers import say

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def test_sparse_attention_example():
    say("case: examples/sparse_attention.py")
    import sparse_attention

    assert sparse_attention.main(["--prompt", "1100", "--chunk", "500", "--requests", "2",
                                  "--tokens", "3"]) == 0
