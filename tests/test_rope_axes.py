"""Rotary positions of several axes, alone and while appending to the cache,
bit for bit against the one-axis reference on a table whose row t holds the
cosines and sines that token t's pairs take."""

import ctypes

import numpy as np
import pytest

import attention_ref as ref
import block_scaled_fp8_w8a16_amd as w8mod
from block_scaled_fp8_w8a16_amd import attention as A
from test_attention import DT, _descs, cuda, i32, layout_pages, rounded, same_bits

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w8mod.library()
    return w8mod


def places(sections, order):
    """(axis, table column) of every pair, by walking over the pairs."""
    out, left, taken = [], list(sections), [0] * len(sections)
    n = len(sections)
    for i in range(sum(sections)):
        if order == "turns":
            a = i % n if left[i % n] > 0 and i % n else 0
        else:
            a = next(a for a in range(n) if left[a] > 0)
        left[a] -= 1
        out.append((a, taken[a] if order == "own" else i))
        taken[a] += 1
    assert left == [0] * n
    return out


def per_token(table, pos, sections, order):
    """float32 [tokens, pairs, 2]: row t of pos [axes, tokens]; NaN outside."""
    out = np.full((pos.shape[1], sum(sections), 2), np.nan, np.float32)
    for i, (a, c) in enumerate(places(sections, order)):
        ok = (pos[a] >= 0) & (pos[a] < table.shape[0])
        out[ok, i] = table[pos[a][ok], c]
    return out


def columns(sections, order):
    return max(sections) if order == "own" else sum(sections)


# ---------------------------------------------------------------- CPU side

def test_turns_give_every_axis_its_pairs():
    got = places((4, 3, 2), "turns")
    assert [a for a, _ in got] == [0, 1, 2, 0, 1, 2, 0, 1, 0]


def axes(**kw):
    a = dict(positions=16, axis_stride=1, count=3, order=0, pairs=(16, 8, 8), table_pairs=32)
    a.update(kw)
    a["pairs"] = (ctypes.c_uint32 * 4)(*a["pairs"])
    return A.Axes(**a)


REFUSALS = [(dict(positions=0), "NULL"), (dict(count=0), "SHAPE"), (dict(count=5), "SHAPE"),
            (dict(order=3), "SHAPE"), (dict(table_pairs=31), "SHAPE"), (dict(table_pairs=33), "SHAPE"),
            (dict(order=2, table_pairs=15), "SHAPE"), (dict(pairs=(0, 0, 0)), "SHAPE"),
            (dict(order=1, pairs=(8, 12, 12)), "SHAPE"), (dict(order=1, pairs=(10, 11, 11)), "SHAPE"),
            (dict(pairs=(1 << 31, 1 << 31, 32)), "SHAPE"), (dict(pairs=(513, 0, 0), table_pairs=513), "SHAPE"),
            (dict(pairs=(17, 8, 8), table_pairs=33), "SHAPE")]       # wider than the head of 64
STATUS = {"NULL": w8mod.ERR_NULL_PTR, "SHAPE": w8mod.ERR_SHAPE}


def raw_rope(x, positions=8, table=16):
    return w8mod.library().w8a16_rope_axes(16, 64, 64, 16, 64, 64, 1, 1, 1, 64, table, positions, x, 0, 0, 0)


@pytest.mark.parametrize("kw,want", REFUSALS)
def test_rope_refusals(kw, want):
    assert raw_rope(axes(**kw)) == STATUS[want]
    assert w8mod.last_error().startswith("w8a16_rope_axes: ")


def test_rope_refuses_what_is_missing():
    assert raw_rope(None) == w8mod.ERR_NULL_PTR
    assert raw_rope(axes(), table=0) == w8mod.ERR_NULL_PTR
    assert raw_rope(axes(), positions=0) == w8mod.ERR_SHAPE


@pytest.mark.parametrize("kw,want", REFUSALS)
def test_append_refusals(kw, want):
    x = axes(**kw)
    c, s, ap, _ = _descs(ap__rot_dim=2 * min(sum(x.pairs[:3]), 100))
    assert w8mod.library().w8a16_kv_append_axes(c, s, ap, x, 0) == STATUS[want]
    assert w8mod.last_error().startswith("w8a16_kv_append_axes: ")


def test_append_refuses_what_is_missing():
    lib = w8mod.library()
    c, s, ap, _ = _descs()
    assert lib.w8a16_kv_append_axes(c, s, ap, None, 0) == w8mod.ERR_NULL_PTR
    assert lib.w8a16_kv_append_axes(c, s, None, axes(), 0) == w8mod.ERR_NULL_PTR
    c, s, ap, _ = _descs(ap__table=None, ap__q=None)
    assert lib.w8a16_kv_append_axes(c, s, ap, axes(), 0) == w8mod.ERR_NULL_PTR
    c, s, ap, _ = _descs(ap__rot_dim=32)
    assert lib.w8a16_kv_append_axes(c, s, ap, axes(), 0) == w8mod.ERR_SHAPE
    c, s, ap, _ = _descs(ap__table_positions=0)
    assert lib.w8a16_kv_append_axes(c, s, ap, axes(), 0) == w8mod.ERR_SHAPE


def test_calls_without_tokens_are_ok():
    lib = w8mod.library()
    assert lib.w8a16_rope_axes(0, 64, 64, 0, 64, 64, 1, 0, 1, 64, 0, 8, axes(positions=0), 0, 0, 0) == w8mod.OK
    c, s, ap, _ = _descs(s__tokens=0, s__seqs=0, s__block_table=None, s__kv_lens=None, ap__k=None,
                         ap__v=None, s__max_new=0)
    assert lib.w8a16_kv_append_axes(c, s, ap, axes(positions=0), 0) == w8mod.OK


def test_python_side_refusals():
    t = torch.zeros
    pos = t(2, 3, dtype=torch.int32)
    for kw in (dict(sections=(1, 1), order="other"), dict(sections=()), dict(sections=(1,) * 5),
               dict(sections=(3, -1)), dict(sections=(1, 1))):       # the last: no GPU tensor
        with pytest.raises(ValueError):
            w8mod.rope(t(3, 1, 4), t(4, 2, 2), pos, **kw)


# ---------------------------------------------------------------- rotation

ROPES = [
    # tokens, heads, dim, sections, order, layout, dtype, pitch (0: contiguous)
    (1, 1, 16, (4, 4), "split", "half", "bf16", 0),
    (5, 3, 64, (16, 8, 8), "split", "half", "bf16", 0),
    (7, 2, 128, (24, 20, 20), "turns", "half", "bf16", 3 * 128),
    (9, 2, 80, (20, 20), "own", "half", "fp16", 0),
    (4, 5, 96, (13, 11, 7, 5), "split", "interleaved", "fp16", 5 * 96 + 16),
    (6, 3, 40, (3, 5, 2), "split", "half", "fp32", 3 * 40 + 1),
    (3, 2, 72, (4, 3, 3, 3), "turns", "interleaved", "fp32", 0),
    (11, 1, 64, (0, 32, 0), "split", "half", "bf16", 0),
    (2, 2, 64, (32,), "turns", "half", "bf16", 0),
    (5, 2, 66, (9, 24), "own", "interleaved", "bf16", 0),
    (3, 1, 1024, (171, 171, 170), "turns", "half", "bf16", 0),
    (2100, 33, 64, (16, 8, 8), "split", "half", "bf16", 0),      # several heads per thread
    (2100, 33, 64, (11, 11, 10), "turns", "interleaved", "fp16", 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", ROPES, ids=[str(i) for i in range(len(ROPES))])
def test_rope_bits(w8, case):
    tokens, heads, dim, sections, order, layout, dtype, pitch = case
    rng = np.random.default_rng(tokens + dim)
    width = pitch or heads * dim
    x = rounded(rng.normal(size=(tokens, width)), dtype)
    xd = cuda(x, DT[dtype])[:, :heads * dim].unflatten(1, (heads, dim))
    xs = x[:, :heads * dim].reshape(tokens, heads, dim)
    table = ref.table64(61, 2 * columns(sections, order), magnitude=1.1).astype(np.float32)
    pos = rng.integers(0, 61, (len(sections), tokens))
    rows = per_token(table, pos, sections, order)
    # the axes' rows further apart than the tokens
    apart = torch.full((len(sections), tokens + 3), 1 << 30, dtype=torch.int32, device="cuda")
    apart[:, :tokens] = cuda(pos.astype(np.int32))
    for inverse in (False, True):
        want = torch.from_numpy(ref.rotate32(xs, rows, range(tokens), layout, inverse)).to(DT[dtype])
        got = w8.rope(xd, cuda(table), apart[:, :tokens], layout=layout, inverse=inverse,
                      sections=sections, order=order)
        same_bits(got, want)
    y = cuda(x, DT[dtype])
    view = y[:, :heads * dim].unflatten(1, (heads, dim))
    w8.rope(view, cuda(table), apart[:, :tokens], view, layout=layout, inverse=True, sections=sections,
            order=order)
    same_bits(view, want)
    assert (y[:, heads * dim:].cpu().float().numpy() == x[:, heads * dim:]).all()


@pytest.mark.gpu
def test_one_axis_is_the_plain_rotation(w8):
    x = torch.randn(70, 4, 64, device="cuda", dtype=torch.bfloat16)
    table = w8.rope_table(90, 64)
    pos = torch.arange(70, dtype=torch.int32, device="cuda") + 20
    same_bits(w8.rope(x, table, pos.expand(3, 70), sections=(11, 11, 10), order="turns"),
              w8.rope(x, table, pos).cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["split", "turns", "own"])
def test_positions_outside_the_table_are_nan_in_their_axis(w8, order):
    sections, dim = (3, 3, 2), 24
    table = ref.table64(10, 2 * columns(sections, order)).astype(np.float32)
    pos = np.array([[0, -1, 9, 1 << 30], [9, 3, 10, 1], [5, 2, -1 << 31, 0]])
    x = np.random.default_rng(2).normal(size=(4, 2, dim)).astype(np.float32)
    want = ref.rotate32(x, per_token(table, pos, sections, order), range(4), "half")
    got = w8.rope(cuda(x), cuda(table), cuda(pos.astype(np.int32)), sections=sections, order=order)
    same_bits(got, torch.from_numpy(want))
    assert np.isnan(want).any() and not np.isnan(want[:, :, 16:]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("order,layout", [("split", "half"), ("turns", "interleaved"), ("own", "half")])
def test_gradient(w8, order, layout):
    """Against the transpose of the formula in FP64, and central differences."""
    rng = np.random.default_rng(5)
    sections = (3, 3, 2)
    x, dy = (rng.normal(size=(3, 2, 20)).astype(np.float32) for _ in range(2))
    table = ref.table64(50, 2 * columns(sections, order), magnitude=1.3).astype(np.float32)
    pos = rng.integers(0, 50, (3, 3))
    rows = per_token(table, pos, sections, order)
    dx = w8.rope(cuda(dy), cuda(table), cuda(pos.astype(np.int32)), layout=layout, inverse=True,
                 sections=sections, order=order).cpu().numpy()

    def f(v):
        y = w8.rope(cuda(v), cuda(table), cuda(pos.astype(np.int32)), layout=layout, sections=sections,
                    order=order)
        return float((y.cpu().numpy().astype(np.float64) * dy).sum())
    top = np.abs(dy).max()
    for idx in np.ndindex(3, 2, 20):
        step = np.zeros_like(x)
        step[idx] = 0.25
        # Linear in x: no truncation.  An element enters two outputs, of two
        # products and a sum each, rounded at magnitudes below 8 in both
        # evaluations; the other outputs cancel exactly.  x + step and x - step
        # (below 4) are rounded once each and enter by at most 1.3.  dx has
        # three roundings of its own.
        assert abs((f(x + step) - f(x - step)) / 0.5 - dx[idx]) <= \
            top * 2.0 ** -24 * (2 * 2 * 3 * 8 + 2 * 2 * 4 * 1.3) / 0.5 + 3 * 8 * 2.0 ** -24
    # transposed: dx[i0] = dy0 c + dy1 s, dx[i1] = dy1 c - dy0 s
    want = dy.astype(np.float64)
    i0 = np.arange(8) if layout == "half" else 2 * np.arange(8)
    i1 = i0 + (8 if layout == "half" else 1)
    c, s = (rows[:, None, :, i].astype(np.float64) for i in (0, 1))
    want[..., i0], want[..., i1] = dy[..., i0] * c + dy[..., i1] * s, dy[..., i1] * c - dy[..., i0] * s
    # two products and a sum, each rounded once, of magnitudes below 8
    assert np.abs(dx - want).max() <= 3 * 8 * 2.0 ** -24


# ------------------------------------------------------------------ append

APPENDS = [
    # new, held before, q heads, kv heads, dim, page, sections, order, layout, dtype
    ([1], [0], 2, 1, 16, 16, (4, 4), "split", "half", "bf16"),
    ([1, 1, 1, 1], [15, 16, 0, 33], 4, 2, 128, 32, (24, 20, 20), "turns", "half", "bf16"),
    ([5, 0, 17, 1], [3, 40, 15, 31], 8, 2, 64, 16, (8, 4, 4), "split", "interleaved", "fp16"),
    ([40, 33], [7, 16], 3, 3, 80, 48, (20, 20), "own", "half", "bf16"),
    ([18, 2], [30, 14], 5, 5, 96, 64, (13, 11, 7, 5), "split", "half", "fp32"),
    ([3, 70], [61, 0], 4, 4, 256, 64, (64, 32, 32), "split", "interleaved", "bf16"),
    ([2, 9], [31, 1], 2, 1, 192, 32, (12, 10, 10), "turns", "half", "fp32"),
    ([35], [100], 2, 2, 112, 16, (28, 28), "own", "half", "fp16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", APPENDS, ids=[str(i) for i in range(len(APPENDS))])
@pytest.mark.parametrize("queries", [False, True])
def test_append_bits(w8, case, queries):
    new, past, hq, hkv, dim, page, sections, order, layout, dtype = case
    rng = np.random.default_rng(dim + page)
    totals = [n + p for n, p in zip(new, past)]
    pages = sum(-(-t // page) for t in totals) + 2
    cache = ref.Cache(pages, hkv, page, dim, rng)
    table = layout_pages(rng, totals, page, pages)
    for b, p in enumerate(past):
        for h in range(hkv):
            for is_v in (False, True):
                cache.append(None, is_v, h, table[b], 0, p, 0.05 * rng.normal(size=(p, dim)))
    dev = cache.to(w8)
    tokens = sum(new)
    x = rounded(rng.normal(size=(tokens, (hq + 2 * hkv) * dim + 8)), dtype)
    xd = cuda(x, DT[dtype])
    cut = [0, hq * dim, (hq + hkv) * dim, (hq + 2 * hkv) * dim]
    q, k, v = (xd[:, cut[i]:cut[i + 1]].unflatten(1, (-1, dim)) for i in range(3))
    qn, kn, vn = (x[:, cut[i]:cut[i + 1]].reshape(tokens, -1, dim) for i in range(3))
    rt = ref.table64(90, 2 * columns(sections, order)).astype(np.float32)
    pos = rng.integers(0, 90, (len(sections), tokens))
    pos[0, tokens // 2] = 90           # outside: its pairs are NaN
    rows = per_token(rt, pos, sections, order)
    kr = ref.rotate32(kn, rows, range(tokens), layout)
    cu = np.concatenate([[0], np.cumsum(new)])
    for b in range(len(new)):
        for h in range(hkv):
            part = slice(cu[b], cu[b + 1])
            cache.append(None, False, h, table[b], past[b], totals[b], kr[part, h])
            cache.append(None, True, h, table[b], past[b], totals[b], vn[part, h])
    got = w8.kv_append(dev, k, v, cuda(table.astype(np.int32)), i32(totals), cu_seqlens=i32(cu.tolist()),
                       max_new=max(new), table=cuda(rt), layout=layout, q=q if queries else None,
                       positions=cuda(pos.astype(np.int32)), sections=sections, order=order)
    for t, want in zip(dev, (cache.k, cache.v, cache.ks, cache.vs)):
        have = t.cpu().numpy()
        if t is dev.k or t is dev.v:       # any NaN code
            have, want = have.copy(), want.copy()
            for c in (have, want):
                c[(c & 127) == 127] = 127
        assert np.array_equal(have, want)
    if queries:
        same_bits(got, torch.from_numpy(ref.rotate32(qn, rows, range(tokens), layout)).to(DT[dtype]))
    else:
        assert got is None


@pytest.mark.gpu
def test_queries_of_no_sequence_are_zeros(w8):
    cache = w8.kv_cache(4, 1, 16, 32)
    table = w8.rope_table(8, 32)
    x = torch.ones(3, 1, 32, device="cuda", dtype=torch.bfloat16)
    q = w8.kv_append(cache, x, x, i32([[0], [1], [2]]), i32([1, 0, -5]), table=table, q=x,
                     positions=i32([[1, 2, 3], [3, 2, 1]]), sections=(8, 8))
    assert (q[0] != 0).any() and (q[1:] == 0).all()
    assert cache.k_scale[0].any() and not cache.k_scale[1:].any()


@pytest.mark.gpu
def test_captured_and_on_another_stream(w8):
    g = torch.Generator(device="cuda").manual_seed(1)
    table = w8.rope_table(64, 64)
    bt, lens = i32([[0], [1]]), i32([3, 9])
    x = torch.randn(2, 6, 64, generator=g, device="cuda").bfloat16()
    pos = i32([[3, 9], [1, 4], [2, 8]])
    cache, other = w8.kv_cache(2, 2, 16, 64), w8.kv_cache(2, 2, 16, 64)
    kw = dict(table=table, positions=pos, sections=(16, 8, 8))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        q = w8.kv_append(cache, x[:, 4:5].expand(2, 2, 64), x[:, 5:].expand(2, 2, 64), bt, lens, q=x[:, :4], **kw)
        r = w8.rope(x, table, pos, sections=(16, 8, 8))
    for step in range(3):
        x.copy_(torch.randn(2, 6, 64, generator=g, device="cuda").bfloat16())
        pos.add_(step)
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            want = w8.rope(x, table, pos, sections=(16, 8, 8))
        wq = w8.kv_append(other, x[:, 4:5].expand(2, 2, 64), x[:, 5:].expand(2, 2, 64), bt, lens, q=x[:, :4],
                          stream=stream, **kw)
        torch.cuda.synchronize()
        assert torch.equal(q, wq) and torch.equal(r, want)
        for a, b in zip(cache, other):
            assert torch.equal(a, b)
