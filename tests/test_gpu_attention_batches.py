"""Batches as captured steps pad them: parts of prompts among slots without tokens."""
import pytest

import extended_precision_gemm_gb300 as ddg

from attention_bounds import near
from attention_util import Batch, filled, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ("mxfp4", "nvfp4"))
@pytest.mark.parametrize("window,sinks", ((0, 0), (90, 2)))
@pytest.mark.parametrize("part,slots,at", ((255, 256, 0), (255, 256, 255), (60, 40, 17), (300, 1000, 500), (300, 64, 63), (9, 2000, 1999)))
def test_a_part_among_empty_slots(fmt, window, sinks, part, slots, at):
    """Few or many rows a slot on average, whichever kernel that makes: the same answers; the cache as well."""
    import torch
    sizes = [(0, 0)] * slots
    sizes[at] = (max(part, 310), part)
    batch = Batch(sizes, 16, seed=part, lead=1, tail=2)
    cache, values = filled(batch, 1, 64, fmt)
    q = queries(batch, 8, 64, "bfloat16")
    near(ddg.mx4_attention(q, cache, *batch.dev, window=window, sinks=sinks), q, batch, values, "bfloat16", window, sinks)
    k, v = ddg.mx4_cache_read(cache, batch.tokens, *batch.dev, dtype=torch.float32)
    empty = ddg.mx4_cache(batch.pages, 16, 1, 64, fmt)
    ddg.mx4_cache_append(empty, k, v, *batch.dev)
    again = ddg.mx4_cache_read(empty, batch.tokens, *batch.dev, dtype=torch.float32)
    rows = slice(batch.starts[0], batch.starts[-1])
    assert torch.equal(k[rows], again[0][rows]) and torch.equal(v[rows], again[1][rows])
    assert k[rows].any()
