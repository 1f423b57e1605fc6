"""4-bit weights that were laid out on another stream than the one they are used on."""
import pytest

import extended_precision_gemm_gb300 as ddg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ("mxfp4", "nvfp4"))
def test_their_memory_is_not_given_away_while_the_callers_stream_reads_them(fmt):
    import torch
    D, F = 1024, 1536
    w = [torch.randn(s, device="cuda").bfloat16() for s in ((F, D), (F, D), (D, F))]
    x = torch.randn(3, D, device="cuda").bfloat16()
    want = ddg.mx4_ff_gated(x, *ddg.mx4_ff_weights(*w, fmt))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    w4 = ddg.mx4_ff_weights(*w, fmt, stream=side)
    side.synchronize()
    parts = [t for q in w4 for t in (q.codes, q.scales, q.exponents) if t is not None]
    places = {t.data_ptr(): t.numel() * t.element_size() for t in parts}
    torch.cuda._sleep(1_000_000_000)  # the current stream is busy for about half a second, then reads the weights
    y = ddg.mx4_ff_gated(x, *w4)
    done = torch.cuda.Event()
    done.record()
    del w4, parts
    with torch.cuda.stream(side):
        new = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in places.values() for _ in range(16)]
    busy = not done.query()
    taken = {t.data_ptr() for t in new} & set(places)
    torch.cuda.synchronize()
    assert busy and not taken
    assert torch.equal(y, want)
