"""The example of answers over a 4-bit cache runs, from prompts to captured steps."""
import importlib.util
import pathlib

import pytest

pytestmark = pytest.mark.gpu

PATH = pathlib.Path(__file__).resolve().parent.parent / "examples" / "answers.py"


@pytest.mark.parametrize("fmt", ("mxfp4", "nvfp4"))
@pytest.mark.parametrize("group", (1, 4))
def test_it_runs(fmt, group):
    import torch
    spec = importlib.util.spec_from_file_location("answers_example", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.main(["--layers", "3", "--model", "128", "--group", str(group), "--prompts", "4", "--longest", "150", "--answer", "12", "--format", fmt])
    assert got["answers"].shape == (4, 12, 128)
    assert torch.isfinite(got["answers"]).all()
    # steps and the one pass round at other places (a code of 4 bits here and there, a quarter of
    # its value at most); tokens, pages or positions that are not the same give a drift of order 1
    assert got["drift"] < 0.25
