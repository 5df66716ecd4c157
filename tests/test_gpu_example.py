"""The example program: a hybrid model's speculative decoding through the public calls."""
import pytest

pytestmark = pytest.mark.gpu


def test_verified_windows_equal_greedy_decoding(cuda_device):
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_verify.py")
    spec = importlib.util.spec_from_file_location("hybrid_verify", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    want, got, windows = m.main(batch=3, steps=20, T=5)
    assert windows < 20
    assert (got == want).all()
