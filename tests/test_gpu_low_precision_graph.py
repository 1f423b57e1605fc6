"""The 4-bit and feed-forward calls captured in a CUDA graph and replayed on new inputs."""
import pytest

import extended_precision_gemm_gb300 as ddg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", (1, 40, 300))
def test_replays_follow_their_inputs(tokens):
    import torch
    D, F = 256, 416
    w = [torch.randn(s, device="cuda").bfloat16() for s in ((F, D), (F, D), (D, F))]
    x, dy = (torch.randn(tokens, D, device="cuda").bfloat16() for _ in range(2))

    def everything():
        out = []
        for fmt in ("mxfp4", "nvfp4"):
            q = ddg.mx4_quantize(x, fmt)
            out += [ddg.mx4_dequantize(q), ddg.mx4_gemm(q, weights[fmt][0]), ddg.mx4_ff_gated(x, *weights[fmt]),
                    ddg.mx4_dequantize(ddg.mx4_quantize(x, fmt, cols=True))]
        y, saved = ddg.ff_gated(x, *w, save=True)
        return out + [y, *ddg.ff_gated_backward(dy, x, *w, saved)]

    weights = {fmt: ddg.mx4_ff_weights(*w, fmt) for fmt in ("mxfp4", "nvfp4")}
    everything()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = everything()
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(tokens, D, generator=g, device="cuda"))
        dy.copy_(torch.randn(tokens, D, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        for a, b in zip(got, everything()):
            assert torch.equal(a, b)
    assert ddg.wait_timeouts() == 0
