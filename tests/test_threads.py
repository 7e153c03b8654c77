"""Threads that share a stream, and so its workspace: each call's result is
what it is alone."""

import threading

import numpy as np
import pytest

import block_scaled_fp8_w8a16_amd as w8mod
from test_attention import DT, cuda, i32
from test_kv_span import make, own_plan, w8  # noqa: F401
from test_product_epilogue import operands

torch = pytest.importorskip("torch")


def together(calls, want, rounds):
    """Thread i runs calls[i] `rounds` times on the current stream."""
    got = [[] for _ in calls]
    stream = torch.cuda.current_stream()
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(stream):
            for _ in range(rounds):
                got[i].append(calls[i]())
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert len(g) == rounds and all(torch.equal(x, w) for x in g)


@pytest.mark.gpu
def test_products_of_one_stream(w8):
    """K splits of the tile kernel: their sums are added by a second launch."""
    m, n, k = 40, 2304, 8192
    assert w8.plan(m, n, k).kernel == w8.KERNEL_TILE and w8.plan(m, n, k).splits > 1
    a, w, scale, _ = operands(m, n, k, 1)
    calls = [lambda x=a * (i + 1), f=f: f(x, w, scale) for i in range(2) for f in (
        w8.gemm, lambda *o: w8.gemm_epilogue(*o, activation="silu"))]
    together(calls, [c() for c in calls], 50)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["shared", "tiles", "sinks"])
def test_attention_of_one_stream(w8, kind):
    rng = np.random.default_rng(2)
    new, totals, shared = ([1] * 6, [300 + 9 * i for i in range(6)], 256) if kind == "shared" else \
        ([40, 30], [400, 333], 0)
    kw = dict(shared=shared, plan_=own_plan(w8, new, 2, chunk=1))
    if kind == "sinks":
        kw.update(window=200, sinks=30)
    calls = []
    for _ in range(3):
        cache, table, q = make(rng, new, totals, 4, 2, 64, 32, "bf16", shared)
        dev, bt, lens, qd = cache.to(w8), cuda(table.astype(np.int32)), i32(totals), cuda(q, DT["bf16"])
        cu = i32(np.concatenate([[0], np.cumsum(new)]).tolist())
        calls.append(lambda o=(qd, dev, bt, lens), c=cu: w8.kv_attention(*o, cu_seqlens=c, max_new=max(new), **kw))
    together(calls, [c() for c in calls], 50)
