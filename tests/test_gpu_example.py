"""The residual block example runs the operators together: decoding a token
agrees with prefilling it, and the feed-forward half's gradient with a
difference quotient.  Needs an MI355X."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_residual_block_example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "residual_block.py")
    spec = importlib.util.spec_from_file_location("residual_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    ahead, off = example.main(batch=2, L=70, D=256, H=4, P=64, N=64, F=704)
    # a handful of bf16 roundings on either side (2^-8 each); the quotient's own error is about step^2
    assert ahead < 4 * 2.0 ** -8
    assert off < 1e-2
