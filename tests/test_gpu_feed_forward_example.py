"""The feed-forward example from training to serving, at a small size."""
import importlib.util
import pathlib

import pytest

pytestmark = pytest.mark.gpu

PATH = pathlib.Path(__file__).resolve().parent.parent / "examples" / "feed_forward.py"


@pytest.mark.parametrize("fmt", ("mxfp4", "nvfp4"))
def test_training_lowers_the_loss_and_serving_follows(fmt):
    spec = importlib.util.spec_from_file_location("feed_forward_example", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.main(["--model", "128", "--inner", "320", "--tokens", "256", "--steps", "120", "--format", fmt])
    assert got["last"] < 0.7 * got["first"]
    # E2M1 rounds a value by a quarter of it at most, about a tenth on average; x, the weights
    # (twice) and h: some tenths in all
    assert got["serving"] < 0.5
    # a token alone takes the split kernel, the prompt the pairs' tiles: sums of another order,
    # a bfloat16 rounding and a code of h here and there
    assert got["token"] < 0.02
    # 32-bit sums of 128 products
    assert got["product"] < 1e-5
