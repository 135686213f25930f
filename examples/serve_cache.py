"""A layer's attention served from the 8-bit key/value cache, on one GPU.

    python examples/serve_cache.py [--steps N]

Three ragged prompts are written and attended to in one call each, then tokens
are decoded one at a time: write and attention of a step are captured in a
graph once and replayed with the lengths counted up on the GPU.  At the end a
sequence is read back, compared with what was written, and its pages are
parked: compressed losslessly with the codec, and restored bit for bit.
Keys, values and queries are random numbers; a model computes them.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lossless_tensor_compression_amd as ltc  # noqa: E402


def main(steps=32, prompts=(700, 33, 260), heads=8, group=4, dim=128, page=64, seed=0):
    """Returns (largest difference of a decoded row from attention in 32 bits
    over the unquantised numbers, compressed share of the parked bytes)."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    # pages are handed out in any order; here, enough for every sequence's end
    need = [-(-(n + steps) // page) for n in prompts]
    cache = ltc.KVCache.empty(sum(need), heads, dim, page=page)
    order = torch.randperm(sum(need)).to(torch.int32).split(need)
    table = torch.zeros((len(prompts), max(need)), dtype=torch.int32)
    for row, pages in zip(table, order):
        row[:len(pages)] = pages
    table = table.cuda()

    # the prompts, one after another in one call
    cu = torch.cumsum(torch.tensor([0, *prompts]), 0).to(torch.int32).cuda()
    lengths = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    q, k, v = normal(sum(prompts), heads * group, dim), normal(sum(prompts), heads, dim), normal(sum(prompts), heads, dim)
    ltc.cache_write(cache, k, v, table, lengths, cu)
    ltc.cache_attend(cache, q, table, lengths, cu)
    keys = [list(x.split(prompts)) for x in (k, v)]

    # one token a sequence and step
    q1, k1, v1 = normal(len(prompts), heads * group, dim), normal(len(prompts), heads, dim), normal(len(prompts), heads, dim)

    def step():
        lengths.add_(1)
        ltc.cache_write(cache, k1, v1, table, lengths)
        return ltc.cache_attend(cache, q1, table, lengths)

    def keep():
        for all_rows, new in zip(keys, (k1, v1)):
            for i in range(len(prompts)):
                all_rows[i] = torch.cat([all_rows[i], new[i:i + 1]])

    out = step()
    keep()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(steps - 1):
        for x in (q1, k1, v1):
            x.copy_(normal(*x.shape))
        graph.replay()
        keep()
    cache.check()

    # against attention in 32 bits over the numbers before they were coded
    worst = 0.0
    for i in range(len(prompts)):
        kf, vf = (x[i].float().transpose(0, 1).repeat_interleave(group, 0) for x in keys)
        p = torch.softmax((kf * q1[i].float()[:, None]).sum(-1) * dim ** -0.5, -1)
        worst = max(worst, float(((p[..., None] * vf).sum(1) - out[i].float()).abs().max()))

    # a sequence as 16-bit rows again
    n = prompts[0] + steps
    k0, v0 = ltc.cache_read(cache, table[:1], lengths[:1], torch.tensor([0, n], dtype=torch.int32, device="cuda"), rows=n)
    assert (k0.float() - keys[0][0].float()).abs().max() < 0.5 and v0.shape == (n, heads, dim)

    # its pages parked and restored
    pages = order[0].long().cuda()
    parked = [ltc.compress(x[pages].reshape(-1)) for x in (cache.k_codes, cache.v_codes)]
    for x, blob in zip((cache.k_codes, cache.v_codes), parked):
        held = x[pages].clone()
        x[pages] = 0
        x[pages] = ltc.decompress(blob, shape=held.shape)
        assert torch.equal(x[pages], held)
    share = sum(b.numel() for b in parked) / (2 * pages.numel() * heads * page * dim)
    return worst, share


if __name__ == "__main__":
    parser = argparse.ArgumentParser()
    parser.add_argument("--steps", type=int, default=32)
    worst, share = main(parser.parse_args().steps)
    print(f"decoded rows differ by at most {worst:.4f} from attention over unquantised numbers; "
          f"parked pages take {share:.3f} of their bytes")
