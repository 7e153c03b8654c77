"""The attention half of one decoder layer, served: a batch of prompts in
chunks, then decode steps replayed from a HIP graph.

    python examples/decode_layer.py [--prompts 700,45,1,320] [--steps 32]

A step is four launches of the library: the Q/K/V projection (one W8A16
product), `kv_append` (rotates queries and keys, stores keys and values in
the paged FP8 cache), `kv_attention`, and the output projection (another
W8A16 product).  At the end every output is compared with plain FP32
arithmetic over the same weights and unquantised keys and values.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_fp8_w8a16_amd as w8  # noqa: E402


def random_weight(n, k, seed, device="cuda"):
    """FP8 codes [n, k] and scales [ceil(n/128), k/128] of a random matrix
    whose products keep the size of their inputs."""
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(n, k, generator=g) * k ** -0.5
    pad = -n % 128
    blocks = torch.nn.functional.pad(w, (0, 0, 0, pad)).view((n + pad) // 128, 128, k // 128, 128)
    s = blocks.abs().amax((1, 3)) / 448.0
    codes = (blocks / s[:, None, :, None]).view(n + pad, k)[:n].to(torch.float8_e4m3fn)
    return codes.to(device), s.to(device)


def dequantised(weight):
    codes, s = weight
    n, k = codes.shape
    return codes.float() * s.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)


class AttentionLayer:
    """Projections, rotation, cache and attention of one layer.  It owns the
    weights and the cache; the sequences' pages and lengths are the caller's."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, pages, page_size, positions, seed=0):
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.w_qkv = random_weight((q_heads + 2 * kv_heads) * head_dim, hidden, seed)
        self.w_out = random_weight(hidden, q_heads * head_dim, seed + 1)
        self.cache = w8.kv_cache(pages, kv_heads, page_size, head_dim)
        self.table = w8.rope_table(positions, head_dim)

    def project(self, x):
        """Views of one product's output: q, k, v [tokens, heads, head_dim]."""
        qkv = w8.gemm(x, *self.w_qkv).view(x.shape[0], -1, self.head_dim)
        return qkv.split([self.q_heads, self.kv_heads, self.kv_heads], 1)

    def attend(self, q, k, v, block_table, kv_lens, **seqs):
        q = w8.kv_append(self.cache, k, v, block_table, kv_lens, table=self.table, q=q, **seqs)
        return w8.kv_attention(q, self.cache, block_table, kv_lens, **seqs)

    def __call__(self, x, block_table, kv_lens, **seqs):
        """x [tokens, hidden]: the sequences' new tokens, kv_lens counting
        them (cu_seqlens and max_new as in kv_append)."""
        out = self.attend(*self.project(x), block_table, kv_lens, **seqs)
        return w8.gemm(out.view(x.shape[0], -1), *self.w_out)


class DecodeGraph:
    """One decode step of a fixed batch, captured: step(x) appends a token to
    every sequence of kv_lens (advanced on the GPU) and returns the output,
    which the next step overwrites."""

    def __init__(self, layer, block_table, kv_lens, hidden):
        self.x = torch.zeros(kv_lens.shape[0], hidden, dtype=torch.bfloat16, device="cuda")

        def one():
            kv_lens.add_(1)
            return layer(self.x, block_table, kv_lens)
        # an eager step first: the workspaces cannot grow during the capture.
        # The token it stores is the first replay's place.
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            one()
            kv_lens.sub_(1)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph, stream=stream):
                self.out = one()
        torch.cuda.current_stream().wait_stream(stream)

    def step(self, x):
        self.x.copy_(x)
        self.graph.replay()
        return self.out


def lay_out_pages(lengths, page_size):
    """int32 block table [seqs, width] for sequences of up to `lengths`
    tokens, each with pages of its own, and the number of pages."""
    need = [-(-n // page_size) for n in lengths]
    table = torch.zeros(len(need), max(need), dtype=torch.int32)
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(0)).to(torch.int32)
    first = 0
    for row, n in zip(table, need):
        row[:n] = order[first:first + n]
        first += n
    return table.cuda(), sum(need)


def prefill(layer, xs, block_table, chunk):
    """Runs the prompts xs (a list of [tokens, hidden]) through the layer, at
    most `chunk` tokens of each per call.  Returns their outputs and kv_lens."""
    device = block_table.device
    done, outs = [0] * len(xs), [[] for _ in xs]
    while any(d < len(x) for d, x in zip(done, xs)):
        new = [min(chunk, len(x) - d) for d, x in zip(done, xs)]
        batch = torch.cat([x[d:d + n] for d, n, x in zip(done, new, xs)])
        done = [d + n for d, n in zip(done, new)]
        cu = torch.tensor([0] + new).cumsum(0).to(device, torch.int32)
        lens = torch.tensor(done, dtype=torch.int32, device=device)
        out = layer(batch, block_table, lens, cu_seqlens=cu, max_new=max(new))
        for o, part in zip(outs, out.split(new)):
            o.append(part)
    return [torch.cat(o) for o in outs], lens


def plain(layer, x):
    """The layer on one sequence x [tokens, hidden] in FP32, with the keys
    and values as the projection gives them."""
    t, d = x.shape[0], layer.head_dim
    qkv = (x.float() @ dequantised(layer.w_qkv).T).view(t, -1, d)
    cos, sin = layer.table[:t, None, :, 0], layer.table[:t, None, :, 1]

    def rotated(y):
        a, b = y[..., :d // 2], y[..., d // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    q, k, v = qkv.split([layer.q_heads, layer.kv_heads, layer.kv_heads], 1)
    group = layer.q_heads // layer.kv_heads
    q = rotated(q).transpose(0, 1)
    k = rotated(k).transpose(0, 1).repeat_interleave(group, 0)
    v = v.transpose(0, 1).repeat_interleave(group, 0)
    s = (q @ k.transpose(1, 2).contiguous()) * d ** -0.5
    s = s.masked_fill(torch.ones(t, t, dtype=torch.bool, device=x.device).triu(1), float("-inf"))
    out = (s.softmax(-1) @ v).transpose(0, 1).reshape(t, -1)
    return out @ dequantised(layer.w_out).T


def run(prompts, steps, hidden=4096, q_heads=32, kv_heads=8, head_dim=128, page_size=64, chunk=256):
    """Serves the prompts, then `steps` tokens more of each.  Returns the
    largest relative error (root mean square, per sequence) against plain()
    and the time of a decode step in microseconds."""
    g = torch.Generator().manual_seed(1)
    xs = [torch.randn(n + steps, hidden, generator=g).to(torch.bfloat16).cuda() for n in prompts]
    table, pages = lay_out_pages([n + steps for n in prompts], page_size)
    layer = AttentionLayer(hidden, q_heads, kv_heads, head_dim, pages, page_size, max(prompts) + steps)
    outs, lens = prefill(layer, [x[:n] for x, n in zip(xs, prompts)], table, chunk)
    graph = DecodeGraph(layer, table, lens, hidden)
    inputs = torch.stack([torch.stack([x[n + i] for x, n in zip(xs, prompts)]) for i in range(steps)])
    tail = torch.empty_like(inputs)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for i in range(steps):
        tail[i] = graph.step(inputs[i])
    torch.cuda.synchronize()
    us = (time.perf_counter() - t0) / steps * 1e6
    worst = 0.0
    for b, x in enumerate(xs):
        want = plain(layer, x)
        got = torch.cat([outs[b], tail[:, b]]).float()
        worst = max(worst, ((got - want).norm() / want.norm()).item())
    return worst, us


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--prompts", default="700,45,1,320", help="prompt lengths")
    ap.add_argument("--steps", type=int, default=32, help="tokens decoded of each")
    args = ap.parse_args()
    prompts = [int(n) for n in args.prompts.split(",")]
    worst, us = run(prompts, args.steps)
    print("%d sequences, %d decode steps of %.1f us; relative error against plain FP32 %.4f" %
          (len(prompts), args.steps, us, worst))
    # a value is rounded to E4M3 by at most 2^-4 of itself
    if not worst < 2.0 ** -4:
        sys.exit("outputs differ from the plain layer by more than the cache's rounding")


if __name__ == "__main__":
    main()
