"""A layer's attention served from a 4-bit key/value cache of bounded length, on
one GPU.

    python examples/serve_bounded.py [--steps N] [--budget N] [--codes e2m1|e4m3|int8]

Queries and keys are normed and rotated, keys and values written, attention adds
to each cached position the weight it got.  When a sequence has come to `budget`
positions plus `slack`, it is cut to its recent positions and those of most weight,
each head by itself; the pages it had are handed out again.  The step between two
cuts is captured in a graph once and replayed.  Queries, keys and values are random
numbers; a model computes them.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lossless_tensor_compression_amd as ltc  # noqa: E402


class Pages:
    """A cache's free pages."""

    def __init__(self, count):
        self.free = list(range(count))

    def take(self, sequences, each):
        return torch.tensor([[self.free.pop() for _ in range(each)] for _ in range(sequences)], dtype=torch.int32, device="cuda")

    def give(self, table):
        self.free += table.flatten().tolist()


def main(steps=300, prompts=(400, 90, 257), budget=192, slack=64, recent=32, heads=4, group=4, dim=128, page=32, codes="e2m1", seed=0):
    """Returns (cuts, positions held at the end, positions come to, largest
    difference of a last row from attention in 32 bits over what its cache holds)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(prompts)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    def count(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    rotation = ltc.Rotation(dim, theta=500000.0)
    q_weight, k_weight = 1 + 0.1 * normal(dim), 1 + 0.1 * normal(dim)
    wide, kept = -(-max(max(prompts), budget + slack) // page), -(-(budget + slack) // page)
    pages = Pages(B * (wide + kept))
    cache = ltc.KVCache.empty(len(pages.free), heads, dim, page=page, codes=codes)
    weights = cache.no_weights()
    table = pages.take(B, wide)

    # the prompts, one after another in one call
    cu, total = count([0, *torch.tensor(prompts).cumsum(0).tolist()]), count(prompts)
    held = total.clone()  # positions of the cache; total goes on counting
    q, k, v = normal(sum(prompts), heads * group, dim), normal(sum(prompts), heads, dim), normal(sum(prompts), heads, dim)
    q, k = ltc.norm_rotate(q, k, rotation, total, cu, q_weight, k_weight)
    ltc.cache_write(cache, k, v, table, held, cu)
    ltc.cache_attend(cache, q, table, held, cu, weights=weights)

    def cut():
        nonlocal table
        to = pages.take(B, kept)  # room for the budget, and for what comes until the next cut
        new, _ = ltc.cache_evict(cache, weights, table, held, to, budget, recent)
        pages.give(table)
        table = to
        held.copy_(new)

    q1, k1, v1 = normal(B, heads * group, dim), normal(B, heads, dim), normal(B, heads, dim)

    def step(at):
        total.add_(1)
        held.add_(1)
        a, b = ltc.norm_rotate(q1, k1, rotation, total, None, q_weight, k_weight)
        ltc.cache_write(cache, b, v1, at, held)
        return a, ltc.cache_attend(cache, a, at, held, weights=weights)

    cut()
    cuts, since = 1, 0
    fixed = table.clone()  # the tables of the captured step: copied over after a cut
    query, out = step(fixed)
    since += 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        query, out = step(fixed)
    for _ in range(steps - 1):
        if since == slack:
            cut()
            fixed.copy_(table)
            cuts, since = cuts + 1, 0
        for x in (q1, k1, v1):
            x.copy_(normal(*x.shape))
        graph.replay()
        since += 1
    cache.check()
    rotation.check()

    # the last rows against attention in 32 bits over the numbers that the cache holds
    n, worst = held.tolist(), 0.0
    rows = count([0, *torch.tensor(n).cumsum(0).tolist()])
    k0, v0 = ltc.cache_read(cache, table, held, rows, rows=sum(n))
    for i, (ki, vi) in enumerate(zip(k0.split(n), v0.split(n))):
        kf, vf = (x.float().transpose(0, 1).repeat_interleave(group, 0) for x in (ki, vi))
        p = torch.softmax((kf * query[i].float()[:, None]).sum(-1) * dim ** -0.5, -1)
        worst = max(worst, float(((p[..., None] * vf).sum(1) - out[i].float()).abs().max()))
    return cuts, n, total.tolist(), worst


if __name__ == "__main__":
    parser = argparse.ArgumentParser()
    parser.add_argument("--steps", type=int, default=300)
    parser.add_argument("--budget", type=int, default=192)
    parser.add_argument("--codes", choices=("e2m1", "e4m3", "int8"), default="e2m1")
    a = parser.parse_args()
    cuts, held, total, worst = main(a.steps, budget=a.budget, codes=a.codes)
    print(f"{cuts} cuts; sequences at {total} positions hold {held}; last rows differ by at most {worst:.4f} from attention "
          "in 32 bits over what is held")
