"""Answers to several prompts at once, over a paged 4-bit cache of keys and values.

A stack of layers with random weights: rotary attention over the cache (every
second layer sees a window and the first tokens only) beside the gated block in 4
bits.  The prompts, of different lengths, go through together; then every sequence
answers token by token, a step captured once as a CUDA graph.  The same tokens in
one pass, without the steps, show what the steps change.

    python examples/answers.py [--layers 4] [--model 512] [--heads 2] [--group 4] [--prompts 6] [--longest 700] [--answer 40] [--format mxfp4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import extended_precision_gemm_gb300 as ddg  # noqa: E402

DIM, PAGE = 64, 16


def normed(x):
    return torch.nn.functional.rms_norm(x.float(), x.shape[-1:]).to(x.dtype)


class Layer:
    def __init__(self, a, window, generator):
        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=generator, device="cuda") * cols**-0.5).bfloat16()

        self.heads, self.group = a.heads, a.group
        self.window, self.sinks = (window, 4) if window else (0, 0)
        self.into = weight((a.group + 2) * a.heads * DIM, a.model)
        self.out = weight(a.model, a.group * a.heads * DIM)
        inner = 2 * a.model
        self.ff = ddg.mx4_ff_weights(weight(inner, a.model), weight(inner, a.model), weight(a.model, inner), a.format)

    def __call__(self, x, cache, batch, positions, rotation):
        q, k, v = (normed(x) @ self.into.T).split([n * self.heads * DIM for n in (self.group, 1, 1)], dim=1)
        k, v = (t.unflatten(1, (self.heads, DIM)) for t in (k, v))
        q = ddg.rotary(q.unflatten(1, (self.heads * self.group, DIM)), positions, rotation)
        ddg.mx4_cache_append(cache, k, v, *batch, rotary=rotation)
        y = ddg.mx4_attention(q, cache, *batch, window=self.window, sinks=self.sinks)
        x = x + y.flatten(1) @ self.out.T
        return x + ddg.mx4_ff_gated(normed(x), *self.ff)


class Stack:
    """Layers, and a cache for each over the same pages."""

    def __init__(self, layers, pages, a):
        self.layers = layers
        self.caches = [ddg.mx4_cache(pages, PAGE, a.heads, DIM, a.format) for _ in layers]
        # rotations stretched for four times the length that they are made for
        self.rotation = ddg.rotary_table(DIM, scaling="bands", factor=4.0, original=a.longest)

    def __call__(self, x, batch, positions):
        for layer, cache in zip(self.layers, self.caches):
            x = layer(x, cache, batch, positions, self.rotation)
        return normed(x)


def batch_of(lengths, new, table):
    """Starts, lengths and pages for `new` tokens of each sequence, its last ones, and their positions."""
    starts = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).int().cuda()
    positions = torch.cat([torch.arange(n - m, n) for n, m in zip(lengths, new)]).cuda()
    return (starts, torch.tensor(lengths, dtype=torch.int32, device="cuda"), table), positions


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--model", type=int, default=512)
    ap.add_argument("--heads", type=int, default=2, help="of keys and values")
    ap.add_argument("--group", type=int, default=4, help="query heads for each of them")
    ap.add_argument("--prompts", type=int, default=6)
    ap.add_argument("--longest", type=int, default=700)
    ap.add_argument("--answer", type=int, default=40)
    ap.add_argument("--format", choices=sorted(ddg.MX4_FORMATS), default="mxfp4")
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = [max(1, a.longest * (i + 1) // a.prompts) for i in range(a.prompts)]
    ends = [n + a.answer for n in prompts]
    # pages as they come, none in order
    need = [-(-n // PAGE) for n in ends]
    order = torch.randperm(sum(need), generator=g, device="cuda").int()
    table = torch.full((a.prompts, max(need)), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(need):
        table[b, :n] = order[sum(need[:b]) :][:n]
    layers = [Layer(a, a.longest // 3 if i % 2 else 0, g) for i in range(a.layers)]
    words = torch.randn(sum(ends), a.model, generator=g, device="cuda").bfloat16()  # every sequence's tokens
    first = [sum(ends[:b]) for b in range(a.prompts)]

    # the prompts together, then a token of each at a time
    stack = Stack(layers, sum(need), a)
    batch, positions = batch_of(prompts, prompts, table)
    stack(torch.cat([words[f : f + n] for f, n in zip(first, prompts)]), batch, positions)
    one, place = batch_of([n + 1 for n in prompts], [1] * a.prompts, table)
    at = torch.tensor([f + n for f, n in zip(first, prompts)], device="cuda")

    def step():
        y = stack(words[at], one, place)
        for t in (at, one[1], place):
            t += 1
        return y

    answers = [step()]  # outside the graph once: library handles and workspaces
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for _ in range(a.answer - 1):
        graph.replay()
        answers.append(y.clone())
    answers = torch.stack(answers, 1)

    # the same in one pass over all tokens
    whole = Stack(layers, sum(need), a)
    batch, positions = batch_of(ends, ends, table)
    y = whole(words, batch, positions)
    y = torch.stack([y[f + n : f + n + a.answer] for f, n in zip(first, prompts)])
    drift = ((answers.double() - y.double()).norm() / y.double().norm()).item()
    print(f"{a.prompts} prompts of {prompts[0]} to {prompts[-1]} tokens, {a.answer} tokens each in {a.format}: {drift:.1e} from one pass over all of them")

    # what a step takes, and what the cache holds
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for t in (at, one[1], place):
        t -= 1  # the last token again
    begin.record()
    graph.replay()
    end.record()
    torch.cuda.synchronize()
    cache = stack.caches[0]
    size = sum(t.numel() * t.element_size() for t in (cache.codes, cache.scales, cache.exponents)) * a.layers
    values = a.layers * 2 * a.heads * sum(need) * PAGE * DIM
    print(f"a step of {a.layers} layers: {begin.elapsed_time(end) * 1e3:.0f} us; the cache: {size / 1e6:.1f} MB, {8 * size / values:.2f} bits a value")
    timeouts = ddg.wait_timeouts()
    if timeouts:
        raise SystemExit(f"{timeouts} waits gave up")
    return {"drift": drift, "answers": answers}


if __name__ == "__main__":
    main()
