"""The example layer: each of its stages against the plain references, and
its captured decode steps against the same steps run one by one."""

import os
import sys

import numpy as np
import pytest
import torch

import attention_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import decode_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu
HALF_ULP = 2.0 ** -8      # bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def f32(t):
    return t.float().cpu().numpy()


def make(prompts, steps, page=32, hidden=256, hq=4, hkv=2, dim=64):
    table, pages = ex.lay_out_pages([n + steps for n in prompts], page)
    layer = ex.AttentionLayer(hidden, hq, hkv, dim, pages, page, max(prompts) + steps, seed=7)
    g = torch.Generator().manual_seed(3)
    xs = [torch.randn(n + steps, hidden, generator=g).to(torch.bfloat16).cuda() for n in prompts]
    return layer, table, xs


def test_stages_match_the_references():
    prompts, chunk = [70, 5, 1, 33], 24
    layer, table, xs = make(prompts, 0)
    hq, hkv, d = layer.q_heads, layer.kv_heads, layer.head_dim
    host = ref.Cache(layer.cache.k.shape[0], hkv, 32, d)
    rows, cos = table.cpu().numpy(), layer.table.cpu().numpy()
    done = [0] * len(xs)
    while any(n < len(x) for n, x in zip(done, xs)):
        new = [min(chunk, len(x) - n) for n, x in zip(done, xs)]
        x = torch.cat([x[n:n + m] for n, m, x in zip(done, new, xs)])
        cu = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device="cuda")
        before, done = done, [n + m for n, m in zip(done, new)]
        lens = torch.tensor(done, dtype=torch.int32, device="cuda")
        q, k, v = layer.project(x)
        assert not q.is_contiguous()      # strided views go in as they are
        out = layer.attend(q, k, v, table, lens, cu_seqlens=cu, max_new=max(new))
        whole = layer(x, table, lens, cu_seqlens=cu, max_new=max(new))
        pos = np.concatenate([np.arange(a, b) for a, b in zip(before, done)])
        kr = ref.rotate32(f32(k), cos, pos, "half")
        qr = torch.from_numpy(ref.rotate32(f32(q), cos, pos, "half")).to(torch.bfloat16)
        first = 0
        for b, (a, e) in enumerate(zip(before, done)):
            for h in range(hkv):
                host.append(None, False, h, rows[b], a, e, kr[first:first + e - a, h])
                host.append(None, True, h, rows[b], a, e, f32(v)[first:first + e - a, h])
            first += e - a
        for b, e in enumerate(done):      # what the sequences hold, byte for byte
            held = layer.cache.k.cpu().numpy()
            heldv = layer.cache.v.cpu().numpy()
            for blk in range(-(-e // 16)):
                pg, i, m = rows[b][blk // 2], blk % 2, min(16, e - 16 * blk)
                assert np.array_equal(held[pg][:, 16 * i:16 * i + m], host.k[pg][:, 16 * i:16 * i + m])
                assert np.array_equal(heldv[pg][:, i, :, :m], host.v[pg][:, i, :, :m])
        want, _, tol, _ = ref.attention64(qr.double().numpy(), host, rows, done, new, hq // hkv,
                                          d ** -0.5, True, 0)
        err = np.abs(out.double().cpu().numpy() - want)
        assert (err <= tol + HALF_ULP * np.abs(want) + 2.0 ** -24).all()
        # a second append of the same tokens changes nothing
        assert np.array_equal(bits(whole), bits(ex.w8.gemm(out.view(len(x), -1), *layer.w_out)))


def test_graph_steps_are_the_eager_steps():
    prompts, steps = [40, 1, 15, 16, 700], 20
    layer, table, xs = make(prompts, steps)
    eager, _, _ = make(prompts, steps)
    heads = [x[:n] for x, n in zip(xs, prompts)]
    _, lens = ex.prefill(layer, heads, table, 64)
    _, elens = ex.prefill(eager, heads, table, 64)
    graph = ex.DecodeGraph(layer, table, lens, 256)
    for i in range(steps):
        x = torch.stack([x[n + i] for x, n in zip(xs, prompts)])
        got = graph.step(x).clone()
        elens += 1
        want = eager(x, table, elens)
        torch.cuda.synchronize()
        assert np.array_equal(bits(got), bits(want)), i
    assert torch.equal(lens, elens)
    for a, b in zip(layer.cache, eager.cache):
        assert torch.equal(a, b)


@pytest.mark.parametrize("prompts,chunk", [([130, 3, 1], 64), ([16, 17], 256)])
def test_served_sequences_match_the_plain_layer(prompts, chunk):
    # keys and values are rounded to E4M3, by at most 2^-4 of each
    worst, _ = ex.run(prompts, 6, hidden=512, q_heads=8, kv_heads=2, head_dim=64, page_size=16,
                      chunk=chunk)
    assert worst < 2.0 ** -4
