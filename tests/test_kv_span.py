"""Attention with a window and sinks, and over a prefix that the sequences
share, against FP64 with the bounds of ``attention_ref.attention64``."""

import math

import numpy as np
import pytest

import attention_ref as ref
import block_scaled_fp8_w8a16_amd as w8mod
from block_scaled_fp8_w8a16_amd import attention as A
from test_attention import COMMON_REFUSALS, DT, HALF_ULP, STATUS, _descs, cuda, i32, layout_pages, rounded

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w8mod.library()
    return w8mod


# ---------------------------------------------------------------- CPU side

@pytest.mark.parametrize("kw,want", COMMON_REFUSALS + [
    (dict(at__q=None), "NULL"), (dict(at__dtype=3), "SHAPE"), (dict(at__q_heads=3), "SHAPE"),
    (dict(at__scale=-1.0), "SHAPE")])
@pytest.mark.parametrize("span", [(4, 0), (0, 32)])
def test_refusals(kw, want, span):
    c, s, _, at = _descs(**kw)
    assert w8mod.library().w8a16_kv_attention_span(c, s, at, A.KVSpan(*span), 0) == STATUS[want]
    assert w8mod.last_error().startswith("w8a16_kv_attention_span: ")


def test_calls_without_tokens_are_ok():
    c, s, _, at = _descs(s__tokens=0, s__seqs=0, s__block_table=None, s__kv_lens=None, at__q=None,
                         at__out=None, s__max_new=0)
    for span in (None, A.KVSpan(4, 64)):
        assert w8mod.library().w8a16_kv_attention_span(c, s, at, span, 0) == w8mod.OK


def test_negative_spans_are_refused():
    cache = w8mod.kv_cache(1, 1, 16, 16, device="cpu")
    for kw in (dict(sinks=-1, window=3), dict(shared=-1)):
        with pytest.raises(ValueError):
            w8mod.kv_attention(torch.zeros(1, 1, 16, dtype=torch.bfloat16), cache,
                               torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), **kw)


SHARED_SHAPES = [(64, 64, 1, 8704, 8192, 32, 8, 128), (6, 6, 1, 2400, 1984, 32, 8, 128),
                 (24, 96, 4, 30200, 30016, 64, 8, 128), (2, 2, 1, 100000, 99984, 1, 1, 16),
                 (2, 2, 1, 64, 64, 8, 1, 256), (3, 700, 600, 5000, 4000, 8, 8, 64)]


@pytest.mark.parametrize("shape", SHARED_SHAPES, ids=str)
def test_plans_cover_both_parts(shape):
    seqs, tokens, new, kv, shared, hq, hkv, dim = shape
    first, own = w8mod.plan_kv_shared(*shape)
    if first is None:
        assert own.as_dict() == w8mod.plan_kv_attention(seqs, new, kv, hq, hkv, dim).as_dict()
        return
    group = hq // hkv
    for p, rows, keys, n in ((first, tokens * group, shared, 1), (own, new * group, kv - shared, seqs)):
        assert p.row_tiles * p.row_blocks * 16 >= rows and p.chunks * p.chunk_tiles * 64 >= keys
        assert p.grid == n * hkv * p.row_tiles * p.chunks and p.chunks <= 64
        assert p.workspace_bytes == p.grid * p.row_blocks * 16 * (dim + 4) * 4


@pytest.mark.parametrize("args", [(0, 1, 1, 9, 0, 1, 1, 64), (2, 1, 2, 9, 0, 1, 1, 64), (2, 2, 1, 9, 16, 1, 1, 64),
                                  (2, 2, 1, 9, 0, 3, 2, 64), (2, 2, 1, 9, 0, 1, 1, 65)])
def test_plan_refusals(args):
    with pytest.raises(w8mod.W8A16Error) as e:
        w8mod.plan_kv_shared(*args)
    assert e.value.status == w8mod.ERR_SHAPE


# --------------------------------------------------------------- reference

def attention(q, cache, table, lens, new, group, scale, causal, window, sinks):
    """Outputs, log-sums and bounds; q float64.  As attention64, over an
    explicit list of visible keys."""
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    tol_o, tol_l = np.zeros(q.shape), np.zeros(q.shape[:2])
    first, d = 0, q.shape[2]
    for b, (n, t) in enumerate(zip(new, lens)):
        for h in range(cache.heads):
            k, v = cache.read(h, table[b], max(t, 0))
            for i in range(n):
                p = t - n + i
                if p < 0:
                    continue
                j = np.arange(t)
                see = j[(j <= p if causal else j >= 0) & ((j > p - window) | (j < sinks) if window else j >= 0)]
                kk, vv, m = k[see], v[see], len(see)
                at = first + i, slice(h * group, (h + 1) * group)
                qq = q[at]
                s = qq @ kk.T * scale
                e = (np.abs(qq) @ np.abs(kk).T).max(1) * scale * (d + 4) * 2.0 ** -24
                top = s.max(1)
                w = np.exp(s - top[:, None])
                l = w.sum(1)
                out[at], lse[at] = w @ vv / l[:, None], top + np.log(l)
                rel = 4 * e + 2.0 ** -20 + 2.0 ** -11 + 2 * m * 2.0 ** -24
                tol_o[at] = rel[:, None] * (w @ np.abs(vv)) / l[:, None] + 2.0 ** -25 * np.abs(vv).sum(0) / l[:, None]
                tol_l[at] = 2 * e + 2.0 ** -19 + m * 2.0 ** -24 + 2.0 ** -21 * np.abs(top)
        first += n
    return out, lse, tol_o, tol_l


def compare(out, lse, want, dtype):
    o, ls, to, tl = want
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    bad = ~(np.abs(got - o) <= to + HALF_ULP[dtype] * (np.abs(o) + to) + 2.0 ** -24)
    assert not bad.any(), "%d outputs off, first %s: %r, want %r +- %r" % (
        bad.sum(), np.argwhere(bad)[0], got[bad][0], o[bad][0], to[bad][0])
    none = np.isinf(ls)
    assert np.array_equal(none, np.isinf(gl)) and (gl[none] < 0).all() and (got[none] == 0).all()
    bad = ~(np.abs(gl[~none] - ls[~none]) <= tl[~none])
    assert not bad.any(), "%d log-sums off" % bad.sum()


def make(rng, new, totals, hq, hkv, dim, page, dtype, shared=0):
    """Cache (its unused places hold whatever), table, q; the first `shared`
    tokens' pages are everyone's."""
    common = shared // page
    own = [max(0, -(-t // page) - common) for t in totals]
    pages = common + sum(own) + 3
    cache = ref.Cache(pages, hkv, page, dim, rng)
    perm = rng.permutation(pages)
    width = common + max(own) + 1
    table = np.full((len(new), width), 1 << 30, np.int64)
    at = common
    for b, t in enumerate(totals):
        have = min(common, -(-max(t, 0) // page))
        table[b, :have] = perm[:have]
        table[b, common:common + own[b]] = perm[at:at + own[b]]
        at += own[b]
    longest = int(np.argmax(totals))
    for b, t in enumerate(totals):
        start = 0 if b == longest else min(shared, t)
        if t > start:
            for h in range(hkv):
                for is_v in (False, True):
                    x = rng.normal(size=(t - start, dim)) * np.exp(0.5 * rng.normal(size=(t - start, 1)))
                    cache.append(None, is_v, h, table[b], start, t, x)
    q = rounded(rng.normal(size=(sum(new), hq, dim)) * 0.7, dtype)
    return cache, table, q


def call(w8, cache, table, q, dtype, new, totals, uniform=None, **kw):
    cu = np.concatenate([[0], np.cumsum(new)])
    if uniform is None:
        uniform = min(new) == max(new)
    out, lse = w8.kv_attention(cuda(q, DT[dtype]), cache, cuda(table.astype(np.int32)), i32(totals),
                               cu_seqlens=None if uniform else i32(cu.tolist()), max_new=max(new),
                               return_lse=True, **kw)
    torch.cuda.synchronize()
    return out, lse


# ------------------------------------------------------------------- sinks

SINKS = [
    # new, held before, q heads, kv heads, dim, page, window, sinks, causal, dtype
    ([1], [0], 2, 1, 16, 16, 1, 1, True, "bf16"),
    ([1] * 6, [14, 15, 63, 64, 200, 777], 8, 2, 128, 32, 100, 4, True, "bf16"),
    ([1] * 5, [3, 66, 130, 192, 500], 4, 4, 64, 16, 64, 64, True, "fp16"),
    ([1, 1, 1], [300, 1, 900], 6, 2, 80, 48, 17, 67, True, "bf16"),
    ([1, 1], [1000, 333], 4, 1, 256, 64, 130, 200, True, "bf16"),
    ([5, 0, 3, 1], [300, 40, 0, 129], 10, 2, 64, 16, 33, 5, True, "fp16"),
    ([4, 4], [260, 70], 8, 2, 192, 32, 65, 130, False, "bf16"),
    ([70, 33], [300, 0], 8, 2, 128, 64, 48, 4, True, "bf16"),           # tile kernel from here on
    ([150], [0], 4, 1, 64, 16, 20, 7, True, "fp16"),
    ([90, 1, 40], [64, 700, 210], 12, 3, 80, 32, 129, 70, True, "bf16"),
    ([60], [400], 6, 2, 256, 16, 100, 128, False, "bf16"),
    ([40], [500], 8, 1, 192, 64, 63, 1000, True, "bf16"),               # sinks past everything
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", SINKS, ids=[str(i) for i in range(len(SINKS))])
@pytest.mark.parametrize("chunk", [0, 1, 2])
def test_sinks(w8, case, chunk):
    new, past, hq, hkv, dim, page, window, sinks, causal, dtype = case
    rng = np.random.default_rng(dim + window)
    totals = [n + p for n, p in zip(new, past)]
    cache, table, q = make(rng, new, totals, hq, hkv, dim, page, dtype)
    kw = dict(window=window, sinks=sinks, causal=causal)
    if chunk:      # keys cut finely, by either kernel
        tile = max(new) * hq // hkv > 32
        kw["plan_"] = w8.KVPlan(kernel=2 if tile else 1, row_blocks=8 if tile else 1, waves=4, chunk_tiles=chunk)
    out, lse = call(w8, cache.to(w8), table, q, dtype, new, totals, **kw)
    want = attention(q.astype(np.float64), cache, table, totals, new, hq // hkv, dim ** -0.5, causal, window, sinks)
    compare(out, lse, want, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 5, 40])
def test_keys_between_sinks_and_window_are_nothing(w8, new):
    """Whatever the hidden keys' places hold, NaN and blocks without a scale
    among it, the same bits."""
    rng = np.random.default_rng(new)
    window, sinks, total, hq, hkv, dim, page = 50, 37, 600 + new, 8, 2, 64, 32
    cache, table, q = make(rng, [new], [total], hq, hkv, dim, page, "bf16")
    kw = dict(window=window, sinks=sinks)
    clean = call(w8, cache.to(w8), table, q, "bf16", [new], [total], **kw)
    lo = 600 + 1 - window          # of the first new token
    for p in range(sinks, lo):
        pg, b = table[0][p // page], p % page // 16
        for h in range(hkv):
            kc, vc = cache.parts(pg, h, b)
            kc[p % 16], vc[p % 16] = 0x7F, 0xFF
    for b16 in range(-(-sinks // 16), lo // 16):       # whole blocks
        pg, b = table[0][b16 * 16 // page], b16 % (page // 16)
        cache.ks[pg, :, b], cache.vs[pg, :, b] = 0, 255
    dirty = call(w8, cache.to(w8), table, q, "bf16", [new], [total], **kw)
    assert not clean[0].isnan().any()
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])
    # a NaN among the sinks is seen by all
    kc, _ = cache.parts(table[0][0], 0, 0)
    kc[3] = 0x7F
    out, _ = call(w8, cache.to(w8), table, q, "bf16", [new], [total], **kw)
    assert out[:, :hq // hkv].isnan().all() and not out[:, hq // hkv:].isnan().any()


@pytest.mark.gpu
def test_sinks_without_a_window_say_nothing(w8):
    rng = np.random.default_rng(1)
    cache, table, q = make(rng, [1, 1], [70, 200], 4, 2, 64, 32, "bf16")
    dev = cache.to(w8)
    a = call(w8, dev, table, q, "bf16", [1, 1], [70, 200], sinks=9)
    b = call(w8, dev, table, q, "bf16", [1, 1], [70, 200])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_sinks_of_padded_slots_and_lost_tokens(w8):
    """Slots without tokens, tokens in front of position 0 and tokens that no
    sequence brings give zeros."""
    rng = np.random.default_rng(4)
    cache, table, q = make(rng, [2, 2, 2, 2], [0, 1, 90, 300], 4, 2, 64, 16, "bf16")
    dev = cache.to(w8)
    out, lse = call(w8, dev, table, q, "bf16", [2] * 4, [0, 1, 90, 300], window=30, sinks=3)
    assert (out[[0, 1, 2]] == 0).all() and (out[3:] != 0).any(-1).all()
    assert lse[:3].isneginf().all() and lse[3:].isfinite().all()
    cu = i32([1, 3, 3, 5, 6])
    out, lse = w8.kv_attention(cuda(q, DT["bf16"]), dev, cuda(table.astype(np.int32)), i32([50, 7, 90, 300]),
                               cu_seqlens=cu, max_new=2, window=30, sinks=3, return_lse=True)
    assert (out[[0, 6, 7]] == 0).all() and lse[[0, 6, 7]].isneginf().all() and lse[3:6].isfinite().all()
    # the first sequence now counts tokens on pages that its row does not have
    assert out[1:3].isnan().all() and lse[1:3].isnan().all()


# ------------------------------------------------------------------ shared

SHARED = [
    # new, totals, shared, q heads, kv heads, dim, page, causal, dtype
    ([1, 1], [33, 40], 32, 2, 1, 16, 16, True, "bf16"),
    ([1] * 6, [257, 300, 258, 400, 321, 256 + 130], 256, 8, 2, 128, 32, True, "bf16"),
    ([1] * 5, [50, 49, 200, 48 * 3 + 1, 170], 48, 4, 4, 64, 16, True, "fp16"),        # a tile's middle
    ([1] * 3, [145, 500, 144 + 70], 144, 6, 2, 80, 48, True, "bf16"),
    ([1] * 40, [130 + i for i in range(40)], 128, 8, 2, 64, 64, True, "bf16"),        # tile kernel over the prefix
    ([3] * 20, [330 + 5 * i for i in range(20)], 320, 6, 2, 128, 16, True, "fp16"),
    ([5, 0, 3, 1], [205, 300, 195, 260], 192, 10, 2, 64, 16, True, "fp16"),
    ([2, 1, 7], [600, 513, 530], 512, 4, 1, 256, 64, True, "bf16"),
    ([4, 4], [300, 270], 256, 8, 2, 192, 32, False, "bf16"),
    ([60, 33, 1], [400, 300, 257], 256, 8, 2, 128, 64, True, "bf16"),                 # tile kernel over the own
    ([70, 50], [200, 130], 64, 6, 3, 80, 16, False, "fp16"),
    # a sequence whose new tokens reach into the prefix, one within it, an empty slot in front
    ([3, 2, 4, 2], [0, 200, 131, 90], 128, 4, 2, 64, 32, True, "bf16"),
    ([1, 1, 1], [20, 70, 50], 96, 4, 2, 64, 32, True, "bf16"),                        # none holds all of it
    ([40, 30], [150, 90], 128, 8, 2, 64, 32, True, "bf16"),
]


def own_plan(w8, new, group, chunk=2):
    tile = max(new) * group > 32
    return w8.KVPlan(kernel=2 if tile else 1, row_blocks=8 if tile else 1, waves=4, chunk_tiles=chunk)


@pytest.mark.gpu
@pytest.mark.parametrize("case", SHARED, ids=[str(i) for i in range(len(SHARED))])
@pytest.mark.parametrize("chunk", [1, 2, 1 << 20])
def test_shared(w8, case, chunk):
    new, totals, shared, hq, hkv, dim, page, causal, dtype = case
    rng = np.random.default_rng(dim + shared + len(new))
    cache, table, q = make(rng, new, totals, hq, hkv, dim, page, dtype, shared)
    dev = cache.to(w8)
    want = attention(q.astype(np.float64), cache, table, totals, new, hq // hkv, dim ** -0.5, causal, 0, 0)
    kw = dict(causal=causal, shared=shared + page // 2)          # whole pages of it
    out, lse = call(w8, dev, table, q, dtype, new, totals, plan_=own_plan(w8, new, hq // hkv, chunk=chunk), **kw)
    compare(out, lse, want, dtype)
    if chunk == 1:        # the default, one pass or two
        out, lse = call(w8, dev, table, q, dtype, new, totals, **kw)
        compare(out, lse, want, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("chunk", [1, 64])
def test_shared_of_padded_slots_and_lost_tokens(w8, chunk):
    """Slots without tokens, tokens in front of position 0 and tokens that no
    sequence brings give zeros; a negative length is an empty slot."""
    rng = np.random.default_rng(14)
    new, totals, shared = [2, 2, 2, 2], [0, 1, 90, 300], 64
    cache, table, q = make(rng, new, totals, 4, 2, 64, 16, "bf16", shared)
    dev = cache.to(w8)
    kw = dict(shared=shared, plan_=own_plan(w8, new, 2, chunk=chunk))
    want = attention(q.astype(np.float64), cache, table, totals, new, 2, 64 ** -0.5, True, 0, 0)
    compare(*call(w8, dev, table, q, "bf16", new, totals, **kw), want, "bf16")
    cu, bt = i32([1, 3, 3, 5, 6]), cuda(table.astype(np.int32))
    lens = [1, -3, 90, 300]
    # (the first sequence counts a token whose page is not the others': its rows are not defined)
    want = attention(q[3:6].astype(np.float64), cache, table[2:], lens[2:], [2, 1], 2, 64 ** -0.5, True, 0, 0)
    out, lse = w8.kv_attention(cuda(q, DT["bf16"]), dev, bt, i32(lens), cu_seqlens=cu, max_new=2, return_lse=True,
                               **kw)
    assert (out[[0, 6, 7]] == 0).all() and lse[[0, 6, 7]].isneginf().all()
    compare(out[3:6], lse[3:6], want, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("case", [([1] * 12, [1600 + 37 * i for i in range(12)], 1536, 8, 2, 128, 64, "bf16"),
                                  ([1] * 64, [2100 + 3 * i for i in range(64)], 2048, 4, 1, 64, 32, "fp16"),
                                  ([2] * 30, [1100 + 3 * i for i in range(30)], 1024, 16, 2, 256, 64, "bf16")],
                         ids=["12", "64", "30"])
def test_shared_by_default_plans(w8, case):
    new, totals, shared, hq, hkv, dim, page, dtype = case
    rng = np.random.default_rng(7)
    cache, table, q = make(rng, new, totals, hq, hkv, dim, page, dtype, shared)
    dev = cache.to(w8)
    want = attention(q.astype(np.float64), cache, table, totals, new, hq // hkv, dim ** -0.5, True, 0, 0)
    first = call(w8, dev, table, q, dtype, new, totals, shared=shared, max_kv=max(totals))
    compare(*first, want, dtype)
    for _ in range(3):      # the same bits on every run
        again = call(w8, dev, table, q, dtype, new, totals, shared=shared, max_kv=max(totals))
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 20])
def test_nan_in_the_prefix(w8, new):
    """A NaN key of the prefix reaches the rows that see it; one behind a
    shorter sequence's end does not reach that one."""
    rng = np.random.default_rng(new)
    totals, shared, hq, hkv, dim, page = [130 + new, 200 + new, 40 + new], 128, 8, 2, 64, 32
    cache, table, q = make(rng, [new] * 3, totals, hq, hkv, dim, page, "bf16", shared)
    plan = own_plan(w8, [new], hq // hkv)
    call_ = lambda: call(w8, cache.to(w8), table, q, "bf16", [new] * 3, totals, shared=shared, plan_=plan)
    clean = call_()
    assert not clean[0].isnan().any()
    for is_v in (0, 1):
        codes = cache.parts(table[1][3], 1, 0)[is_v]      # position 96, the second KV head
        was = codes[1].copy()
        codes[1] = 0x7F
        out, _ = call_()
        codes[1] = was
        g = hq // hkv
        assert out[:2 * new, g:].isnan().all() and not out[:, :g].isnan().any()
        assert torch.equal(out[2 * new:], clean[0][2 * new:])
    cache.vs[table[1][0], 0, 1] = 0                        # a block that was never written, seen by all
    out, _ = call_()
    assert out[:, :hq // hkv].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("window,shared", [(0, 256), (40, 0)])
def test_captured_and_on_another_stream(w8, window, shared):
    """Replays over a cache and lengths that change in between."""
    rng = np.random.default_rng(3)
    totals, hq, hkv, dim, page, seqs = [300, 390, 270, 310], 8, 2, 64, 32, 4
    cache, table, _ = make(rng, [1] * seqs, [t + 8 for t in totals], hq, hkv, dim, page, "bf16", shared)
    dev, bt, lens = cache.to(w8), cuda(table.astype(np.int32)), i32(totals)
    q = torch.randn(seqs, hq, dim, device="cuda").bfloat16()
    kw = dict(window=window, sinks=5, shared=shared, return_lse=True, plan_=own_plan(w8, [1], 4))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        w8.kv_attention(q, dev, bt, lens, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out, lse = w8.kv_attention(q, dev, bt, lens, **kw)
    for step in range(4):
        q.copy_(torch.randn(seqs, hq, dim, device="cuda"))
        lens.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        o, l = w8.kv_attention(q, dev, bt, lens, stream=stream, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(lse, l)
        want = attention(q.double().cpu().numpy(), cache, table, [t + step + 1 for t in totals], [1] * seqs,
                         hq // hkv, dim ** -0.5, True, window, 5)
        compare(out, lse, want, "bf16")


# Every width and type is a kernel of its own: rows or tiles of a window, with
# and without sinks, and of the pairs of passes over a prefix.
BUILDS = {
    # new, totals, page, call
    "window, rows": ([1, 3], [200, 333], 16, dict(window=100)),
    "window, tiles": ([70, 40], [200, 333], 16, dict(window=100)),
    "sinks, rows": ([1, 3], [200, 333], 16, dict(window=100, sinks=70)),
    "sinks, tiles": ([70, 40], [200, 333], 16, dict(window=100, sinks=70)),
    "rows, rows": ([1, 2, 1], [270, 300, 150], 32, dict(shared=256)),
    "tiles, rows": ([1] * 96, [8194 + i % 40 for i in range(96)], 64, dict(shared=8192)),
    "tiles, tiles": ([40, 50], [330, 310], 32, dict(shared=256)),
}


@pytest.mark.gpu
@pytest.mark.parametrize("kind", BUILDS)
@pytest.mark.parametrize("dim", [48, 64, 128, 192, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_build(w8, kind, dim, dtype):
    new, totals, page, kw = BUILDS[kind]
    kw = dict(kw)
    shared, hq = kw.get("shared", 0), 16 if kind == "tiles, rows" else 4
    rng = np.random.default_rng(dim + len(kind))
    cache, table, q = make(rng, new, totals, hq, 2, dim, page, dtype, shared)
    if kind == "tiles, rows":      # what the default plans choose; some of the sequences are compared
        first, own = w8.plan_kv_shared(len(new), len(new), 1, table.shape[1] * page, shared, hq, 2, dim)
        assert first.kernel == w8.KV_KERNEL_TILE and own.kernel == w8.KV_KERNEL_ROWS
        some = [0, 39, 95]
    else:
        some = list(range(len(q)))
        if shared:
            kw["plan_"] = own_plan(w8, new, 2, chunk=1)
    seqs = some if len(new) > 8 else range(len(new))
    want = attention(q[some].astype(np.float64), cache, table[seqs], [totals[b] for b in seqs],
                     [new[b] for b in seqs], hq // 2, dim ** -0.5, True, kw.get("window", 0), kw.get("sinks", 0))
    out, lse = call(w8, cache.to(w8), table, q, dtype, new, totals, **kw)
    compare(out[some], lse[some], want, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("max_kv", [1, 100, 300])
@pytest.mark.parametrize("new", [[1, 2, 1], [40, 50, 33]])
def test_longer_sequences_than_max_kv(w8, new, max_kv):
    """max_kv shapes the launch only."""
    rng = np.random.default_rng(max_kv + new[0])
    totals = [600, 1000, 290]
    cache, table, q = make(rng, new, totals, 4, 2, 64, 32, "bf16", 256)
    dev = cache.to(w8)
    for kw in (dict(shared=256), dict(shared=256, plan_=own_plan(w8, new, 2, chunk=1)), dict(window=200, sinks=70)):
        want = attention(q.astype(np.float64), cache, table, totals, new, 2, 64 ** -0.5, True, kw.get("window", 0),
                         kw.get("sinks", 0))
        compare(*call(w8, dev, table, q, "bf16", new, totals, max_kv=max_kv, **kw), want, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("shared", [0, 512])
def test_two_graphs_of_one_stream(w8, shared):
    """They share the stream's workspace; replayed in turn, between eager
    calls of another size, each gives what an eager call does."""
    rng = np.random.default_rng(6)
    calls = []
    for n in (12, 7):
        new, totals = [1] * n, [700 + 90 * i for i in range(n)]
        cache, table, q = make(rng, new, totals, 8, 2, 128, 64, "bf16", shared)
        calls.append((cuda(q, DT["bf16"]), cache.to(w8), cuda(table.astype(np.int32)), i32(totals)))
    kw = [dict(max_new=1, shared=shared, plan_=own_plan(w8, [1], 4, chunk=c) if shared else
               w8.KVPlan(kernel=1, row_blocks=1, waves=4, chunk_tiles=c)) for c in (4, 5)]
    want = [w8.kv_attention(*c, **k) for c, k in zip(calls, kw)]
    stream, graphs, outs = torch.cuda.Stream(), [], []
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for c, k in zip(calls, kw):      # the workspace grows before the captures
            w8.kv_attention(*c, **k)
        for c, k in zip(calls, kw):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                outs.append(w8.kv_attention(*c, **k))
            graphs.append(g)
        for turn in range(6):
            for o in outs:
                o.zero_()
            graphs[turn % 2].replay()
            eager = w8.kv_attention(*calls[turn % 3 % 2], **kw[turn % 3 % 2])
            graphs[1 - turn % 2].replay()
            stream.synchronize()
            assert all(torch.equal(o, w) for o, w in zip(outs, want))
            assert torch.equal(eager, want[turn % 3 % 2])


@pytest.mark.gpu
def test_strided_rows(w8):
    """Queries and outputs inside wider rows, unaligned."""
    rng = np.random.default_rng(8)
    new, totals, shared = [1, 1, 2], [150, 170, 140], 128
    cache, table, q = make(rng, new, totals, 4, 2, 64, 32, "bf16", shared)
    dev, bt, cu = cache.to(w8), cuda(table.astype(np.int32)), i32([0, 1, 2, 4])
    wide = torch.zeros(4, 4 * 64 + 3, dtype=torch.bfloat16, device="cuda")
    qv = wide[:, 1:257].unflatten(1, (4, 64))
    qv.copy_(cuda(q))
    for kw in (dict(shared=shared, plan_=own_plan(w8, new, 2)), dict(window=20, sinks=3)):
        res = torch.full((4, 4 * 64 + 5), 7.0, dtype=torch.bfloat16, device="cuda")
        out = res[:, 3:259].unflatten(1, (4, 64))
        w8.kv_attention(qv, dev, bt, i32(totals), out, cu_seqlens=cu, max_new=2, **kw)
        want = w8.kv_attention(cuda(q, DT["bf16"]), dev, bt, i32(totals), cu_seqlens=cu, max_new=2, **kw)
        assert torch.equal(out, want) and (res[:, :3] == 7).all() and (res[:, 259:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(waves=4, chunk_tiles=2), dict(waves=8, chunk_tiles=64)])
def test_plans_that_are_refused(w8, kw):      # more than 64 chunks, or 8 waves
    cache = w8.kv_cache(70, 1, 128, 16)
    bt = torch.arange(70, dtype=torch.int32, device="cuda").expand(2, 70).contiguous()
    q = torch.zeros(2, 1, 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(w8.W8A16Error) as e:
        w8.kv_attention(q, cache, bt, i32([8000, 8000]), shared=128,
                        plan_=w8.KVPlan(kernel=1, row_blocks=1, **kw))
    assert e.value.status == w8.ERR_BAD_PLAN
