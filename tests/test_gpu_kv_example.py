"""The serving example runs and agrees with plain attention over its cache."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example():
    import kv_decode
    # kv_read rounds the values to bf16 (2^-8 each) and the output rounds once
    # more: three roundings of 2^-8 relative at most, over many terms
    assert kv_decode.main(requests=5, tokens=20, prompt=150) < 3 * 2.0 ** -8
