"""The example's attention layer with its cache in 8 bits runs, and agrees with itself."""
import pytest

from test_gpu_examples import load

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompts,steps", [([300, 37, 1], 9), ([128], 1), ([5, 5, 257, 16], 4)])
def test_hybrid_serving_fp8(prompts, steps):
    """Prompt + steps against one prompt. The bf16 roundings of three layers (18 * 2^-9) can move
    what is cached across a border of e4m3, by half a step of 2^-4 either way: keys and values, in
    both passes, 4 * 2^-4 of the largest value."""
    assert load("hybrid_serving.py").serve(prompts, steps, fp8=True) < 18 * 2.0 ** -9 + 4 * 2.0 ** -4
