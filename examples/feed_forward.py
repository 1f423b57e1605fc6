"""A gated feed-forward block from training to 4-bit serving.

Trains y = (silu(x Wg^T) * (x Wu^T)) Wd^T in bfloat16 to follow a fixed teacher
block (random inputs, Adam on 32-bit master weights), turns its weights into 4
bits, serves single tokens and a prompt with them, and measures the 4-bit
product against the same product in double doubles.

    python examples/feed_forward.py [--model 512] [--inner 1408] [--tokens 1024] [--steps 200] [--format mxfp4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import extended_precision_gemm_gb300 as ddg  # noqa: E402


def weights(model, inner, generator):
    shapes = (inner, model), (inner, model), (model, inner)
    return [torch.randn(s, generator=generator, device="cuda") * s[1] ** -0.5 for s in shapes]


def train(student, teacher, tokens, steps, rate, generator):
    """Adam on the mean squared error to the teacher; the losses of the first and last ten steps."""
    model = student[0].shape[1]
    optimiser = torch.optim.Adam(student, lr=rate)
    half = lambda ws: [w.to(torch.bfloat16) for w in ws]  # noqa: E731
    fixed = half(teacher)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, model, generator=generator, device="cuda").to(torch.bfloat16)
        w = half(student)
        y, saved = ddg.ff_gated(x, *w, save=True)
        error = y.float() - ddg.ff_gated(x, *fixed).float()
        losses.append(error.square().mean())
        dy = (error * (2.0 / tokens)).to(torch.bfloat16)
        grads = ddg.ff_gated_backward(dy, x, *w, saved, need=(False, True, True, True))[1:]
        for p, g in zip(student, grads):
            p.grad = g.float()
        optimiser.step()
    losses = torch.stack(losses)
    return losses[:10].mean().item(), losses[-10:].mean().item()


def relative(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--model", type=int, default=512)
    ap.add_argument("--inner", type=int, default=1408)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--rate", type=float, default=2e-3)
    ap.add_argument("--format", choices=sorted(ddg.MX4_FORMATS), default="mxfp4")
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    teacher = weights(a.model, a.inner, g)
    student = [torch.nn.Parameter(w) for w in weights(a.model, a.inner, g)]
    first, last = train(student, teacher, a.tokens, a.steps, a.rate, g)
    print(f"training: mean squared error {first:.4f} -> {last:.4f} over {a.steps} steps")

    # serving: the weights in 4 bits, laid out once
    trained = [w.detach().to(torch.bfloat16) for w in student]
    w_in, w_out = ddg.mx4_ff_weights(*trained, a.format)
    prompt = torch.randn(a.tokens, a.model, generator=g, device="cuda").to(torch.bfloat16)
    y16, y4 = ddg.ff_gated(prompt, *trained), ddg.mx4_ff_gated(prompt, w_in, w_out)
    error = relative(y4, y16)
    print(f"serving a prompt of {a.tokens} tokens in {a.format}: {error:.4f} from the 16-bit block")
    token = ddg.mx4_ff_gated(prompt[:1], w_in, w_out)
    drift = relative(token, y4[:1])
    print(f"its first token alone: {drift:.1e} from the prompt's")

    # the 4-bit product beside the exact one: the values it multiplies, in double doubles
    x4 = ddg.mx4_quantize(prompt, a.format)
    c = ddg.mx4_gemm(x4, w_in, dtype=torch.float32)
    left, right = (ddg.mx4_dequantize(q, torch.float32).double() for q in (x4, w_in))
    right = right.t().contiguous()
    hi, lo = ddg.dd_gemm_tc(left, torch.zeros_like(left), right, torch.zeros_like(right))
    product = relative(c, hi)
    print(f"4-bit product ({a.tokens} x {w_in.rows} x {a.model}) against double doubles: {product:.1e}")
    timeouts = ddg.wait_timeouts()
    if timeouts:
        raise SystemExit(f"{timeouts} waits gave up")
    return {"first": first, "last": last, "serving": error, "token": drift, "product": product}


if __name__ == "__main__":
    main()
