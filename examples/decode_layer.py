"""One decoder layer, served: a batch of prompts in chunks, then decode steps
replayed from a HIP graph.

    python examples/decode_layer.py [--prompts 700,45,1,320] [--steps 32]
    python examples/decode_layer.py --prefix 512         # the whole layer

A step of the attention half is four launches of the library: the Q/K/V
projection (one W8A16 product), `kv_append` (rotates queries and keys, stores
keys and values in the paged FP8 cache), `kv_attention`, and the output
projection (another W8A16 product).  The whole layer adds what lies around
them to the products' epilogues (biases, the gated feed-forward, residuals),
rotates by positions of three axes, a picture at the start of each prompt, and
serves the prompts behind a common prefix or with a window and sinks.  At the
end every output is compared with plain FP32 arithmetic over the same weights
and unquantised keys and values.
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


def norm(x):
    f = x.float()
    return (f * (f.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()).to(x.dtype)


class DecoderLayer(AttentionLayer):
    """Normalisation (torch), attention with a bias on its projection, and a
    gated feed-forward, each added to what it started from.  sections: pairs
    of each axis of positions; window, sinks and shared as in kv_attention."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, pages, page_size, positions, seed=0, ffn=None,
                 sections=None, window=0, sinks=0, shared=0):
        super().__init__(hidden, q_heads, kv_heads, head_dim, pages, page_size, positions, seed)
        ffn = ffn or 2 * hidden
        self.b_qkv = torch.randn((q_heads + 2 * kv_heads) * head_dim,
                                 generator=torch.Generator().manual_seed(seed + 2)).cuda() * 0.1
        self.w_up, self.w_gate = random_weight(ffn, hidden, seed + 3), random_weight(ffn, hidden, seed + 4)
        self.w_down = random_weight(hidden, ffn, seed + 5)
        self.sections, self.span = sections, dict(window=window, sinks=sinks, shared=shared)

    def project(self, x):
        qkv = w8.gemm_epilogue(x, *self.w_qkv, bias=self.b_qkv).view(x.shape[0], -1, self.head_dim)
        return qkv.split([self.q_heads, self.kv_heads, self.kv_heads], 1)

    def attend(self, q, k, v, block_table, kv_lens, positions=None, **seqs):
        q = w8.kv_append(self.cache, k, v, block_table, kv_lens, table=self.table, q=q, positions=positions,
                         sections=self.sections, **seqs)
        return w8.kv_attention(q, self.cache, block_table, kv_lens, **self.span, **seqs)

    def __call__(self, x, block_table, kv_lens, **seqs):
        """As AttentionLayer's; positions int32 [axes, tokens] with sections."""
        out = self.attend(*self.project(norm(x)), block_table, kv_lens, **seqs)
        x = w8.gemm_epilogue(out.view(x.shape[0], -1), *self.w_out, residual=x)
        h = norm(x)
        up = w8.gemm(h, *self.w_up)
        h = w8.gemm_epilogue(h, *self.w_gate, activation="silu", gate=up)
        return w8.gemm_epilogue(h, *self.w_down, residual=x)


class DecodeGraph:
    """One decode step of a fixed batch, captured: step(x) appends a token to
    every sequence of kv_lens (advanced on the GPU, as positions is if given)
    and returns the output, which the next step overwrites."""

    def __init__(self, layer, block_table, kv_lens, hidden, positions=None):
        self.x = torch.zeros(kv_lens.shape[0], hidden, dtype=torch.bfloat16, device="cuda")
        kw = {} if positions is None else dict(positions=positions)

        def one():
            kv_lens.add_(1)
            if kw:
                positions.add_(1)
            return layer(self.x, block_table, kv_lens, **kw)
        # an eager step first: the workspaces cannot grow during the capture.
        # The token it stores is the first replay's place.
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            one()
            kv_lens.sub_(1)
            if kw:
                positions.sub_(1)
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


def share_pages(lengths, prefix, page_size):
    """The same for sequences behind a common prefix of whole pages, which
    come first in every row."""
    common = prefix // page_size
    table, pages = lay_out_pages(lengths, page_size)
    front = torch.arange(pages, pages + common, dtype=torch.int32, device=table.device)
    return torch.cat([front.expand(len(lengths), -1), table], 1), pages + common


def picture_positions(rows, cols, text, start=0):
    """int32 [3, rows * cols + text]: places of a picture's tokens (one time,
    their row and column) and of the text after it, on which all axes agree."""
    r, c = torch.meshgrid(torch.arange(rows), torch.arange(cols), indexing="ij")
    seen = torch.stack([torch.zeros_like(r), r, c]).flatten(1)
    return (start + torch.cat([seen, (max(rows, cols) + torch.arange(text)).expand(3, -1)], 1)).to(torch.int32)


def prefill(layer, xs, block_table, chunk, held=0, positions=None):
    """Runs the prompts xs (a list of [tokens, hidden]) through the layer, at
    most `chunk` tokens of each per call, behind `held` tokens that the cache
    has of each; positions: int32 [axes, tokens] of each.  Returns their
    outputs and kv_lens."""
    device = block_table.device
    done, outs = [0] * len(xs), [[] for _ in xs]
    while any(d < len(x) for d, x in zip(done, xs)):
        new = [min(chunk, len(x) - d) for d, x in zip(done, xs)]
        batch = torch.cat([x[d:d + n] for d, n, x in zip(done, new, xs)])
        kw = {} if positions is None else dict(
            positions=torch.cat([p[:, d:d + n] for d, n, p in zip(done, new, positions)], 1))
        done = [d + n for d, n in zip(done, new)]
        cu = torch.tensor([0] + new).cumsum(0).to(device, torch.int32)
        lens = torch.tensor([held + d for d in done], dtype=torch.int32, device=device)
        out = layer(batch, block_table, lens, cu_seqlens=cu, max_new=max(new), **kw)
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


def plain_layer(layer, x, positions=None):
    """The whole layer on one sequence, likewise; positions int32 [axes, tokens]."""
    t, d = x.shape[0], layer.head_dim
    x = x.float()
    qkv = (norm(x) @ dequantised(layer.w_qkv).T + layer.b_qkv).view(t, -1, d)
    place = torch.arange(t, device=x.device)
    at = place.expand(d // 2, -1)
    if layer.sections:
        axis = torch.arange(len(layer.sections)).repeat_interleave(torch.tensor(layer.sections))
        at = positions[axis.to(x.device)].long()
    angles = layer.table[at, torch.arange(d // 2, device=x.device)[:, None]]      # [pairs, tokens, 2]
    cos, sin = angles.permute(2, 1, 0)[:, :, None]

    def rotated(y):
        a, b = y[..., :d // 2], y[..., d // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    q, k, v = qkv.split([layer.q_heads, layer.kv_heads, layer.kv_heads], 1)
    group = layer.q_heads // layer.kv_heads
    q = rotated(q).transpose(0, 1)
    k = rotated(k).transpose(0, 1).repeat_interleave(group, 0)
    v = v.transpose(0, 1).repeat_interleave(group, 0)
    s = (q @ k.transpose(1, 2).contiguous()) * d ** -0.5
    window, sinks = layer.span["window"] or t, layer.span["sinks"]
    seen = (place <= place[:, None]) & ((place > place[:, None] - window) | (place < sinks))
    out = (s.masked_fill(~seen, float("-inf")).softmax(-1) @ v).transpose(0, 1).reshape(t, -1)
    x = x + out @ dequantised(layer.w_out).T
    h = norm(x)
    h = torch.nn.functional.silu(h @ dequantised(layer.w_gate).T) * (h @ dequantised(layer.w_up).T)
    return x + h @ dequantised(layer.w_down).T


def run_layer(prompts, steps, prefix, hidden=4096, q_heads=32, kv_heads=8, head_dim=128, page_size=64, chunk=256,
              window=0, sinks=0, picture=(6, 9)):
    """As run(), with the whole layer: every prompt starts with the same
    prefix (its whole pages are held once) and then shows a picture, as far as
    the prompt goes."""
    prefix = prefix // page_size * page_size
    g = torch.Generator().manual_seed(1)
    xs = [torch.randn(n + steps, hidden, generator=g).to(torch.bfloat16).cuda() for n in prompts]
    common = torch.randn(prefix, hidden, generator=g).to(torch.bfloat16).cuda()
    table, pages = share_pages([n + steps for n in prompts], prefix, page_size)
    pairs = head_dim // 2
    sections = [pairs - 2 * (3 * pairs // 8), 3 * pairs // 8, 3 * pairs // 8]
    layer = DecoderLayer(hidden, q_heads, kv_heads, head_dim, pages, page_size, prefix + max(prompts) + steps,
                         sections=sections, window=window, sinks=sinks, shared=prefix)
    before = torch.arange(prefix, dtype=torch.int32).expand(3, -1).contiguous().cuda()
    places = [picture_positions(*picture, n + steps, prefix)[:, :n + steps].contiguous().cuda() for n in prompts]
    if prefix:
        prefill(layer, [common], table[:1], chunk, positions=[before])
    outs, lens = prefill(layer, [x[:n] for x, n in zip(xs, prompts)], table, chunk, prefix, places)
    # (decoded tokens are text: the last place of each, one further a step)
    last = torch.stack([p[:, n - 1] for p, n in zip(places, prompts)], 1).contiguous()
    graph = DecodeGraph(layer, table, lens, hidden, last)
    inputs = torch.stack([torch.stack([x[n + i] for x, n in zip(xs, prompts)]) for i in range(steps)])
    tail = torch.empty_like(inputs)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for i in range(steps):
        tail[i] = graph.step(inputs[i])
    torch.cuda.synchronize()
    us = (time.perf_counter() - t0) / steps * 1e6
    worst = 0.0
    for b, (x, n) in enumerate(zip(xs, prompts)):
        at = torch.cat([before, places[b][:, :n], places[b][:, n - 1:n] + 1 + torch.arange(
            steps, dtype=torch.int32, device="cuda")], 1)
        want = plain_layer(layer, torch.cat([common, x]), at)[prefix:]
        got = torch.cat([outs[b], tail[:, b]]).float()
        worst = max(worst, ((got - want).norm() / want.norm()).item())
    return worst, us


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
    ap.add_argument("--prefix", type=int, help="the whole layer, behind a common prefix of that many tokens")
    ap.add_argument("--window", type=int, default=0, help="of the whole layer's attention")
    ap.add_argument("--sinks", type=int, default=0, help="first tokens seen behind the window")
    args = ap.parse_args()
    prompts = [int(n) for n in args.prompts.split(",")]
    if args.prefix is None and not args.window:
        worst, us = run(prompts, args.steps)
    else:
        worst, us = run_layer(prompts, args.steps, args.prefix or 0, window=args.window, sinks=args.sinks)
    print("%d sequences, %d decode steps of %.1f us; relative error against plain FP32 %.4f" %
          (len(prompts), args.steps, us, worst))
    # a value is rounded to E4M3 by at most 2^-4 of itself
    if not worst < 2.0 ** -4:
        sys.exit("outputs differ from the plain layer by more than the cache's rounding")


if __name__ == "__main__":
    main()
