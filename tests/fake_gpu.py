"""The library's host code without a GPU: run as ``python tests/fake_gpu.py
STAND_IN.so CHECK``, it loads the stand-in for the HIP runtime
(tests/host/fake_hip.cpp), then the library, and runs one of the checks below
(their tests: test_fake_gpu.py).  Kernels do not run; launches are recorded."""

import ctypes
import os
import sys
import threading

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

P = 1 << 20      # an address: never read
_keep = []


def launches(fake):
    """(thread, stream, workgroups, threads of each) of every launch so far."""
    out, buf = [], (ctypes.c_uint64 * 4)()
    for i in range(fake.fake_launches()):
        fake.fake_launch(ctypes.c_uint64(i), buf)
        out.append(tuple(buf))
    fake.fake_forget()
    return out


def attention(w8, seqs, new, pages, q_heads, kv_heads, dim, page=64, plan=None, span=None, stream=0, **kw):
    """Status of an attention call of `seqs` sequences of `new` tokens."""
    A = w8.attention
    page_bytes = kv_heads * page * dim
    cache = A.KVCacheDesc(P, P, P, P, page_bytes, page_bytes, kv_heads * page // 16, kv_heads * page // 16, 1 << 20,
                          page, kv_heads, dim)
    s = A.KVSeqs(P, P, None, pages, pages, seqs, seqs * new, new)
    a = A.KVAttentionArgs(P, P, None, q_heads * dim, dim, q_heads * dim, dim,
                          ctypes.pointer(plan) if plan else None, 0.1, q_heads, 1, 1, kw.get("window", 0), 0)
    lib = w8.library()
    if span:
        return lib.w8a16_kv_attention_span(cache, s, a, A.KVSpan(*span), stream)
    return lib.w8a16_kv_attention(cache, s, a, stream)


def calls_are_whole(w8, fake):
    """Launches that hand partial results to each other through a stream's
    workspace follow each other, whatever other threads do on that stream."""
    lib, m, n, k = w8.library(), 40, 2304, 8192
    tile = dict(kernel=2, row_blocks=8, waves=4, chunk_tiles=2)
    e = w8.Epilogue(out_dtype=1)
    plan = w8.plan(m, n, k)
    assert plan.kernel == w8.KERNEL_TILE and plan.splits > 1

    def with_plan(**kw):
        p = w8.KVPlan(**kw)
        return attention(w8, 2, 40, 8, 8, 2, 64, plan=p)
    ways = {
        "shared prefix": lambda: attention(w8, 6, 1, 36, 32, 8, 128, span=(0, 1984),
                                           plan=w8.KVPlan(kernel=1, row_blocks=1, waves=4, chunk_tiles=4)),
        "tile kernel in chunks": lambda: with_plan(**tile),
        "sinks in chunks": lambda: attention(w8, 2, 40, 8, 8, 2, 64, plan=w8.KVPlan(**tile), span=(4, 0), window=100),
        "product": lambda: lib.w8a16_gemm(P, k, P, P, P, n, m, n, k, 0),
        "product by a plan": lambda: lib.w8a16_gemm_planned(P, k, P, P, P, n, m, n, k, plan, 0),
        "product without allocation": lambda: lib.w8a16_gemm_noalloc(P, k, P, P, P, n, m, n, k, 0),
        "product with an epilogue": lambda: lib.w8a16_gemm_epilogue(P, k, P, P, P, n, m, n, k, e, 0),
    }
    for name, call in ways.items():
        fake.fake_thread(ctypes.c_uint64(0))
        assert call() == 0, (name, w8.last_error())
        launches(fake)      # (the first call may clear what it has allocated)
        call()
        one = len(launches(fake))
        assert one >= 2, name
        fake.fake_pause_us(ctypes.c_uint64(2000))
        status = []

        def work(i):
            fake.fake_thread(ctypes.c_uint64(i))
            for _ in range(4):
                status.append(call())
        threads = [threading.Thread(target=work, args=(i,)) for i in (1, 2, 3)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        fake.fake_pause_us(ctypes.c_uint64(0))
        got = launches(fake)
        assert status == [0] * 12 and len(got) == 12 * one, name
        for i in range(0, len(got), one):
            assert len({g[0] for g in got[i:i + one]}) == 1, "%s: launches of threads %s" % (name, [g[0] for g in got])


def plans_are_the_calls(w8, fake):
    """The public default plan of a window with sinks is the one that a call
    launches by itself, and a call takes it."""
    import random
    rng = random.Random(3)

    def shapes():
        yield 1, 1, 313, 64, 8, 8, 128, 16, 100000          # (20032 keys, all of them sinks)
        for _ in range(1500):
            kv = rng.choice([1, 2, 8])
            yield (rng.randint(1, 40), rng.choice([1, 3, 40, 300]), int(2 ** rng.uniform(0, 9)),
                   rng.choice([16, 64, 256]), kv * rng.choice([1, 4, 5]), kv, 16 * rng.randint(1, 16),
                   rng.choice([0, int(2 ** rng.uniform(0, 14)), 1 << 31]), int(2 ** rng.uniform(0, 17)))
    for seqs, new, pages, page, hq, hkv, dim, window, sinks in shapes():
        shape = (seqs, new, pages, page, hq, hkv, dim, window, sinks)
        p = w8.plan_kv_attention(seqs, new, pages * page, hq, hkv, dim, window, sinks=sinks)
        seen = []
        for plan in (None, p):
            st = attention(w8, seqs, new, pages, hq, hkv, dim, page, plan, (sinks, 0), window=window)
            assert st == 0, (shape, w8.last_error())
            seen.append([g[2:] for g in launches(fake)])
        assert seen[0] == seen[1], shape
        assert seen[0][0] == (p.grid, 64 * p.waves), shape
        assert len(seen[0]) == (2 if p.kernel == w8.KV_KERNEL_TILE and p.chunks > 1 else 1), shape


def all_launches_or_none(w8, fake):
    """A call one of whose launches would pass 2^32 threads (both passes over a
    shared prefix, or the join: a wave per row and KV head) takes another way
    or is refused before the first."""
    tile = dict(kernel=2, row_blocks=8, waves=4)
    rows = dict(kernel=1, row_blocks=1, waves=4)
    refused = 0
    for seqs, new, pages, hq, dim, plan, span, window in [
            (1 << 20, 1, 560, 64, 64, None, (0, 30016), 0), (1 << 18, 40, 560, 64, 64, None, (0, 30016), 0),
            ((1 << 21) - 1, 1, 560, 8, 64, None, (0, 30016), 0),
            (1 << 20, 1, 560, 64, 64, dict(rows, chunk_tiles=100), (0, 30016), 0),
            (1 << 17, 20, 560, 64, 128, dict(tile, chunk_tiles=100), (0, 30016), 0),
            (1 << 18, 16, 40, 64, 128, dict(tile, chunk_tiles=20), (0, 0), 0),
            (1 << 18, 16, 40, 64, 128, dict(tile, chunk_tiles=5), (9, 0), 1500)]:
        launches(fake)
        st = attention(w8, seqs, new, pages, hq, 8, dim, 64, w8.KVPlan(**plan) if plan else None, span, window=window)
        n = len(launches(fake))
        case = (seqs, new, plan, span, st, n, w8.last_error())
        if plan is None:
            assert st == 0, case
        assert st == 0 or (st == w8.ERR_SHAPE and n == 0 and "too many" in w8.last_error()), case
        refused += st != 0
    assert refused


def no_exception_leaves(w8, fake):
    """Where the host has no memory left a call returns a status, with or
    without a message of its own, and the next one is right again."""
    lib, m, n, k = w8.library(), 40, 2304, 8192
    e, plan = w8.Epilogue(out_dtype=1), w8.plan(m, n, k)
    descs = (w8.GemmDesc * 1)(w8.GemmDesc(P, P, P, P, 256, 256, 4, 256, 256))
    ways = {        # on a stream of its own, whose workspace is to be noted
        "gemm": lambda s: lib.w8a16_gemm(P, k, P, P, P, n, m, n, k, s),
        "planned": lambda s: lib.w8a16_gemm_planned(P, k, P, P, P, n, m, n, k, plan, s),
        "epilogue": lambda s: lib.w8a16_gemm_epilogue(P, k, P, P, P, n, m, n, k, e, s),
        "noalloc": lambda s: lib.w8a16_gemm_noalloc(P, k, P, P, P, n, m, n, k, s),
        "batched": lambda s: lib.w8a16_gemm_batched(descs, 1, s),
        "quantiser": lambda s: lib.w8a16_act_quant_fp8(P, 256, P, 256, P, 4, 256, s),
        "w8a8": lambda s: lib.w8a16_gemm_w8a8(P, 256, P, P, P, P, 256, 4, 256, 256, s),
        "w4a4": lambda s: lib.w8a16_gemm_w4a4(P, 256, P, P, P, P, 256, 4, 256, 256, s),
        "attention": lambda s: attention(w8, 6, 1, 36, 32, 8, 128, span=(0, 1984), stream=s, plan=w8.KVPlan(
            kernel=1, row_blocks=1, waves=4, chunk_tiles=4)),
    }
    stopped = 0
    for i, (name, call) in enumerate(ways.items()):
        fake.fake_no_memory(1)
        st = call(i + 1)
        fake.fake_no_memory(0)
        assert st in (0, w8.ERR_HIP), (name, st)
        stopped += st != 0
        if st:
            assert "bad_alloc" in w8.last_error(), (name, w8.last_error())
        assert call(i + 1) == 0, name
    assert stopped >= 4
    # refusals: their messages
    fake.fake_no_memory(1)
    st = [lib.w8a16_gemm(P, 64, P, P, P, n, m, n, k, 0), lib.w8a16_plan(0, 1, 128, 0, plan),
          lib.w8a16_gemm_epilogue(P, k, P, P, P, n, m, n, k, None, 0)]
    fake.fake_no_memory(0)
    assert st == [w8.ERR_PITCH_TOO_SHORT, w8.ERR_M_ZERO, w8.ERR_NULL_PTR] and "null epilogue" in w8.last_error()


def main():
    # (bound with symbols before the library's own dependencies)
    fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
    import block_scaled_fp8_w8a16_amd as w8
    globals()[sys.argv[2]](w8, fake)
    print("done")


if __name__ == "__main__":
    main()
