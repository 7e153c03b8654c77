"""Rotary positions, the paged FP8 cache and attention over it, against the
plain references of ``attention_ref.py``.

The rotation and the cache's codes are compared bit for bit (their
arithmetic is stated exactly); attention against FP64 with the bounds
derived in ``attention64`` plus half an ulp of the output's type."""

import math

import numpy as np
import pytest

import attention_ref as ref
import block_scaled_fp8_w8a16_amd as w8mod

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_ULP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w8mod.library()
    return w8mod


def cuda(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rounded(x, dtype):
    """float32 numpy -> the type -> float32 numpy."""
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).float().numpy()


def same_bits(got, want):
    g, w = got.cpu(), want
    assert g.dtype == w.dtype and g.shape == w.shape
    bad = ~((g == w) | (g.isnan() & w.isnan()))
    assert not bad.any(), "%d differ, first at %s: %s, want %s" % (
        int(bad.sum()), bad.nonzero()[0].tolist(), g[bad][0].item(), w[bad][0].item())


# ---------------------------------------------------------------- CPU side

def test_reference_codes_agree_with_torch():
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.normal(size=4000) * 10.0 ** rng.uniform(-4, 2.4, 4000), ref.VALUES[:127],
                        (ref._MID), [0.0, -0.0, 448.0, -448.0]]).astype(np.float32)
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (ref.encode(x.astype(np.float64)) == want).all()


def test_scale_byte_is_the_smallest_that_fits():
    for a in (0.0, 1e-40, 2.0 ** -118, 447.0, 448.0, 448.1, 3.3e38):
        b = ref.scale_byte(a)
        assert a <= 448 * 2.0 ** (b - 127) and (b == 1 or a > 448 * 2.0 ** (b - 128))


def _raw_rope(**kw):
    a = dict(x=16, xt=64, xh=64, y=16, yt=64, yh=64, dtype=1, tokens=1, heads=1, dim=64, table=16,
             positions=8, rot=64, pos=16, layout=0, inverse=0)
    a.update(kw)
    return w8mod.library().w8a16_rope(a["x"], a["xt"], a["xh"], a["y"], a["yt"], a["yh"], a["dtype"],
                                      a["tokens"], a["heads"], a["dim"], a["table"], a["positions"],
                                      a["rot"], a["pos"], a["layout"], a["inverse"], 0)


@pytest.mark.parametrize("kw,want", [
    (dict(x=0), "NULL"), (dict(table=0), "NULL"), (dict(pos=0), "NULL"),
    (dict(dtype=0), "SHAPE"), (dict(dtype=4), "SHAPE"), (dict(layout=2), "SHAPE"),
    (dict(rot=63), "SHAPE"), (dict(rot=66), "SHAPE"), (dict(rot=0), "SHAPE"),
    (dict(heads=0), "SHAPE"), (dict(tokens=1 << 30, heads=64), "SHAPE"),
])
def test_rope_refusals(kw, want):
    assert _raw_rope(**kw) == {"NULL": w8mod.ERR_NULL_PTR, "SHAPE": w8mod.ERR_SHAPE}[want]
    assert w8mod.last_error().startswith("w8a16_rope: ")


def test_rope_without_tokens_is_ok():
    assert _raw_rope(tokens=0, x=0, y=0, pos=0) == w8mod.OK


@pytest.mark.parametrize("kw", [
    dict(base=1.0), dict(base=float("nan")), dict(scaling=4), dict(scaling=1, factor=0.5),
    dict(scaling=3, factor=4.0), dict(scaling=3, factor=4.0, original=100.0, low_turns=4.0),
    dict(rot=7), dict(rot=1026), dict(scaling=2, factor=2.0, rot=2), dict(positions=1 << 31)])
def test_rope_table_refusals(kw):
    from block_scaled_fp8_w8a16_amd.attention import RopeConfig
    c = RopeConfig(kw.get("base", 1e4), kw.get("factor", 1.0), kw.get("original", 0.0),
                   kw.get("low_turns", 1.0), 4.0, 1.0, kw.get("scaling", 0))
    st = w8mod.library().w8a16_rope_table(c, 16, kw.get("positions", 4), kw.get("rot", 8), 0)
    assert st == w8mod.ERR_SHAPE and w8mod.last_error().startswith("w8a16_rope_table: ")
    assert w8mod.library().w8a16_rope_table(c, 0, 4, 8, 0) == w8mod.ERR_NULL_PTR


def _descs(**kw):
    from block_scaled_fp8_w8a16_amd import attention as A
    c = dict(k=16, v=16, k_scale=16, v_scale=16, k_page_stride=2 * 32 * 64, v_page_stride=2 * 32 * 64,
             k_scale_page_stride=4, v_scale_page_stride=4, pages=4, page_size=32, kv_heads=2,
             head_dim=64)
    s = dict(block_table=16, kv_lens=16, cu_seqlens=None, block_table_stride=2, block_table_width=2,
             seqs=2, tokens=4, max_new=2)
    ap = dict(k=16, v=16, q=16, q_out=16, table=16, table_positions=8, rot_dim=64, layout=0, dtype=1,
              q_heads=4)
    at = dict(q=16, out=16, scale=1.0, q_heads=4, dtype=1, causal=1)
    for name, v in kw.items():
        which, field = name.split("__")
        {"c": c, "s": s, "ap": ap, "at": at}[which][field] = v
    return (A.KVCacheDesc(**c), A.KVSeqs(**s), A.KVAppendArgs(**ap), A.KVAttentionArgs(**at))


COMMON_REFUSALS = [
    (dict(c__k=None), "NULL"), (dict(c__v_scale=None), "NULL"), (dict(s__block_table=None), "NULL"),
    (dict(s__kv_lens=None), "NULL"), (dict(c__head_dim=72), "SHAPE"), (dict(c__head_dim=272), "SHAPE"),
    (dict(c__page_size=24), "SHAPE"), (dict(c__page_size=2048), "SHAPE"), (dict(c__pages=0), "SHAPE"),
    (dict(c__kv_heads=0), "SHAPE"), (dict(c__k_page_stride=4095), "SHAPE"),
    (dict(c__v_page_stride=4096 + 8), "SHAPE"), (dict(c__k=8), "SHAPE"),
    (dict(c__k_scale_page_stride=3), "SHAPE"), (dict(s__seqs=0), "SHAPE"), (dict(s__tokens=5), "SHAPE"),
    (dict(s__block_table_width=0), "SHAPE"), (dict(s__block_table_stride=1), "SHAPE"),
    (dict(s__max_new=0), "SHAPE"), (dict(s__max_new=3), "SHAPE"),
    (dict(s__cu_seqlens=16, s__max_new=5), "SHAPE"),
]
STATUS = {"NULL": w8mod.ERR_NULL_PTR, "SHAPE": w8mod.ERR_SHAPE, "PLAN": w8mod.ERR_BAD_PLAN}


@pytest.mark.parametrize("kw,want", COMMON_REFUSALS + [
    (dict(ap__k=None), "NULL"), (dict(ap__q_out=None), "NULL"), (dict(ap__dtype=0), "SHAPE"),
    (dict(ap__rot_dim=65), "SHAPE"), (dict(ap__rot_dim=66), "SHAPE"), (dict(ap__layout=2), "SHAPE"),
    (dict(ap__table=None), "SHAPE"), (dict(ap__q_heads=0), "SHAPE")])
def test_append_refusals(kw, want):
    c, s, ap, _ = _descs(**kw)
    assert w8mod.library().w8a16_kv_append(c, s, ap, 0) == STATUS[want]
    assert w8mod.last_error().startswith("w8a16_kv_append: ")


@pytest.mark.parametrize("kw,want", COMMON_REFUSALS + [
    (dict(at__q=None), "NULL"), (dict(at__out=None), "NULL"), (dict(at__dtype=3), "SHAPE"),
    (dict(at__q_heads=3), "SHAPE"), (dict(at__q_heads=0), "SHAPE"), (dict(at__scale=-1.0), "SHAPE"),
    (dict(at__scale=float("nan")), "SHAPE"), (dict(at__scale=float("inf")), "SHAPE")])
def test_attention_refusals(kw, want):
    c, s, _, at = _descs(**kw)
    assert w8mod.library().w8a16_kv_attention(c, s, at, 0) == STATUS[want]
    assert w8mod.last_error().startswith("w8a16_kv_attention: ")


def test_calls_without_tokens_are_ok():
    c, s, ap, at = _descs(s__tokens=0, s__seqs=0, s__block_table=None, s__kv_lens=None, ap__k=None,
                          ap__v=None, at__q=None, at__out=None, s__max_new=0)
    assert w8mod.library().w8a16_kv_append(c, s, ap, 0) == w8mod.OK
    assert w8mod.library().w8a16_kv_attention(c, s, at, 0) == w8mod.OK


@pytest.mark.parametrize("shape", [(1, 1, 300, 32, 8, 128, 0), (64, 1, 8192, 32, 8, 128, 0),
                                   (1, 1, 131072, 64, 8, 128, 0), (24, 5, 3006, 40, 8, 64, 1024),
                                   (2, 2048, 8192, 32, 8, 128, 0), (3, 1, 1, 1, 1, 16, 0),
                                   (7, 33, 0, 6, 2, 256, 5)])
def test_plans_cover_keys_and_rows(shape):
    seqs, new, kv, hq, hkv, dim, window = shape
    p = w8mod.plan_kv_attention(*shape[:6], window=window)
    assert p.row_tiles * p.row_blocks * 16 >= new * hq // hkv
    keys = min(kv, window + new) if window else kv
    assert p.chunks * p.chunk_tiles * 64 >= keys
    assert p.grid == seqs * hkv * p.row_tiles * p.chunks
    assert (p.workspace_bytes > 0) == (p.chunks > 1)


@pytest.mark.parametrize("args", [(0, 1, 1, 1, 1, 64), (1, 0, 1, 1, 1, 64), (1, 1, 1, 3, 2, 64),
                                  (1, 1, 1, 2, 2, 65), (1, 1, 1 << 31, 2, 2, 64)])
def test_plan_refusals(args):
    with pytest.raises(w8mod.W8A16Error) as e:
        w8mod.plan_kv_attention(*args)
    assert e.value.status == w8mod.ERR_SHAPE


def test_python_side_refusals():
    t = torch.zeros
    with pytest.raises(ValueError):
        w8mod.rope(t(2, 3), t(4, 2, 2), t(2, dtype=torch.int32))
    with pytest.raises(ValueError):      # not a GPU tensor
        w8mod.rope(t(2, 1, 4), t(4, 2, 2), t(2, dtype=torch.int32))
    cache = w8mod.kv_cache(2, 1, 32, 16, device="cpu")
    with pytest.raises(ValueError):
        w8mod.kv_append(cache, t(1, 1, 16), t(1, 1, 16), t(1, 1, dtype=torch.int32),
                        t(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        w8mod.kv_cache(2, 1, 24, 16, device="cpu")
    with pytest.raises(ValueError):
        w8mod.rope_table(4, 8, scaling="other", device="cpu")


# -------------------------------------------------------------------- rope

@pytest.mark.gpu
@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling="linear", factor=8.0), dict(scaling="base", factor=4.0),
    dict(scaling="bands", factor=8.0, original=512.0, low_turns=1.0, high_turns=4.0, magnitude=1.1)])
def test_rope_table(w8, kw):
    positions, rot = 3000, 96
    got = w8.rope_table(positions, rot, **kw).cpu().numpy()
    names = {"low_turns": "low", "high_turns": "high"}
    want = ref.table64(positions, rot, **{names.get(k, k): v for k, v in kw.items()})
    # one rounding to FP32 of values up to 1.1, and angles up to 3000 whose
    # frequencies differ by a few FP64 ulps
    assert np.abs(got - want).max() <= 2.0 ** -24 * 1.1 + 1e-11


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,dim,rot,pad", [
    (1, 1, 2, 2, 0), (3, 2, 7, 6, 0), (5, 3, 64, 64, 0), (17, 5, 80, 40, 3), (9, 4, 96, 32, 16),
    (33, 2, 128, 128, 8), (4, 7, 256, 192, 0), (2, 3, 50, 16, 0)])
def test_rope_bits(w8, dtype, layout, tokens, heads, dim, rot, pad):
    rng = np.random.default_rng(tokens * 1000 + dim)
    x = rounded(rng.normal(size=(tokens, heads * dim + pad)), dtype)
    table = ref.table64(200, rot).astype(np.float32)
    pos = rng.integers(0, 200, tokens)
    xd = cuda(x, DT[dtype])[:, :heads * dim].unflatten(1, (heads, dim))
    xs = x[:, :heads * dim].reshape(tokens, heads, dim)
    for inverse in (False, True):
        want = torch.from_numpy(ref.rotate32(xs, table, pos, layout, inverse)).to(DT[dtype])
        got = w8.rope(xd, cuda(table), i32(pos.tolist()), layout=layout, inverse=inverse)
        same_bits(got, want)
    # in place, rows apart by the padding, which stays as it was
    y = cuda(x, DT[dtype])
    view = y[:, :heads * dim].unflatten(1, (heads, dim))
    w8.rope(view, cuda(table), i32(pos.tolist()), view, layout=layout, inverse=True)
    same_bits(view, want)
    assert (y[:, heads * dim:].cpu().float().numpy() == x[:, heads * dim:]).all()


@pytest.mark.gpu
def test_rope_position_outside_the_table_is_nan(w8):
    x = torch.ones(4, 2, 32, device="cuda")
    got = w8.rope(x, w8.rope_table(10, 16), i32([0, -1, 10, 9])).cpu()
    assert got[[1, 2], :, :16].isnan().all() and not got[[0, 3]].isnan().any()
    assert (got[:, :, 16:] == 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient(w8, layout):
    """dx = rope(dy, inverse): against the formula's transpose in FP64, and
    against central differences of <dy, rope(x)>."""
    rng = np.random.default_rng(5)
    x, dy = (rng.normal(size=(3, 2, 24)).astype(np.float32) for _ in range(2))
    table = ref.table64(50, 16, magnitude=1.3).astype(np.float32)
    pos = [0, 7, 49]
    dx = w8.rope(cuda(dy), cuda(table), i32(pos), layout=layout, inverse=True).cpu().numpy()

    def f(v):
        return float((ref.rotate32(v, table, pos, layout).astype(np.float64) * dy).sum())
    for idx in np.ndindex(3, 2, 24):
        step = np.zeros_like(x)
        step[idx] = 0.25
        # linear in x: no truncation; 48 FP32 roundings of values below 8 over
        # a step of 0.5
        assert abs((f(x + step) - f(x - step)) / 0.5 - dx[idx]) <= 48 * 8 * 2.0 ** -24 / 0.5
    want = ref.rotate32(dy, table.astype(np.float64), pos, layout, inverse=True)
    assert np.abs(dx - want).max() <= 4 * 8 * 2.0 ** -24


# ------------------------------------------------------------------ append

def layout_pages(rng, totals, page, pages, width=None):
    """A block table of distinct random pages; unused columns hold numbers
    that must never be used."""
    width = width or max(1, max(-(-t // page) for t in totals))
    perm = rng.permutation(pages)
    table = np.full((len(totals), width), 1 << 30, np.int64)
    at = 0
    for b, t in enumerate(totals):
        n = -(-max(t, 0) // page)
        table[b, :n] = perm[at:at + n]
        table[b, n:] = rng.choice([-1, 1 << 30, pages])
        at += n
    return table


APPENDS = [
    # new per sequence, held before, q heads, kv heads, dim, page, rot, layout, dtype
    ([1], [0], 2, 1, 16, 16, 16, "half", "bf16"),
    ([1, 1, 1, 1], [15, 16, 0, 33], 4, 2, 128, 32, 128, "half", "bf16"),
    ([5, 0, 17, 1], [3, 40, 15, 31], 8, 2, 64, 16, 32, "interleaved", "fp16"),
    ([40, 33], [7, 16], 3, 3, 80, 48, 40, "half", "bf16"),
    ([18, 2], [30, 14], 5, 5, 96, 64, 0, "half", "fp32"),
    ([3, 70], [61, 0], 4, 4, 256, 64, 256, "interleaved", "bf16"),
    ([2, 9], [31, 1], 2, 1, 192, 32, 64, "half", "fp32"),
    ([35], [100], 2, 2, 112, 16, 112, "half", "fp16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", APPENDS, ids=[str(i) for i in range(len(APPENDS))])
@pytest.mark.parametrize("padded", [False, True])
def test_append_bits(w8, case, padded):
    new, past, hq, hkv, dim, page, rot, layout, dtype = case
    rng = np.random.default_rng(dim + page + rot)
    totals = [n + p for n, p in zip(new, past)]
    pages = sum(-(-t // page) for t in totals) + 2
    cache = ref.Cache(pages, hkv, page, dim, rng)
    table = layout_pages(rng, totals, page, pages)
    # the tokens held before, of another magnitude, so that scales grow
    for b, p in enumerate(past):
        for h in range(hkv):
            for is_v in (False, True):
                cache.append(None, is_v, h, table[b], 0, p, 0.05 * rng.normal(size=(p, dim)))
    dev = cache.to(w8, padded)
    tokens = sum(new)
    x = rounded(rng.normal(size=(tokens, (hq + 2 * hkv) * dim + 8)) *
                np.exp(rng.normal(size=(tokens, 1))), dtype)
    xd = cuda(x, DT[dtype])
    cut = [0, hq * dim, (hq + hkv) * dim, (hq + 2 * hkv) * dim]
    q, k, v = (xd[:, cut[i]:cut[i + 1]].unflatten(1, (-1, dim)) for i in range(3))
    qn, kn, vn = (x[:, cut[i]:cut[i + 1]].reshape(tokens, -1, dim) for i in range(3))
    rt = ref.table64(max(totals) + 1, rot).astype(np.float32) if rot else None
    cu = np.concatenate([[0], np.cumsum(new)])
    pos = np.concatenate([np.arange(t - n, t) for n, t in zip(new, totals)]).astype(int)
    kr = ref.rotate32(kn, rt, pos, layout) if rot else kn
    for b in range(len(new)):
        for h in range(hkv):
            rows = slice(cu[b], cu[b + 1])
            cache.append(None, False, h, table[b], past[b], totals[b], kr[rows, h])
            cache.append(None, True, h, table[b], past[b], totals[b], vn[rows, h])
    uniform = min(new) == max(new)
    got_q = w8.kv_append(dev, k, v, i32(table.tolist()), i32(totals),
                         cu_seqlens=None if uniform and not padded else i32(cu.tolist()),
                         max_new=None if padded else max(new), table=cuda(rt) if rot else None,
                         layout=layout, q=q if rot else None)
    torch.cuda.synchronize()
    assert (dev.k_scale.cpu().numpy() == cache.ks).all()
    assert (dev.v_scale.cpu().numpy() == cache.vs).all()
    for name, got, want in (("k", dev.k, cache.k), ("v", dev.v, cache.v)):
        bad = np.argwhere(got.cpu().numpy() != want)
        assert bad.size == 0, (name, len(bad), bad[0])
    if rot:
        same_bits(got_q, torch.from_numpy(ref.rotate32(qn, rt, pos, layout)).to(DT[dtype]))


@pytest.mark.gpu
def test_append_token_by_token_and_special_values(w8):
    """One sequence grown a token at a time through several blocks: every
    step equals the reference, with zeros, NaN, infinities and the type's
    largest and smallest values among the tokens."""
    rng = np.random.default_rng(11)
    dim, page, steps = 64, 32, 40
    cache = ref.Cache(3, 1, page, dim, rng)
    dev = cache.to(w8)
    table = np.array([[2, 0]])
    top = float(torch.finfo(torch.bfloat16).max)
    for t in range(steps):
        x = rounded(rng.normal(size=(1, 2, dim)) * 4.0 ** rng.integers(-6, 6), "bf16")
        if t in (0, 16):
            x[:] = 0
        if t == 3:
            x[0, 0, 5], x[0, 1, 6] = np.nan, np.inf
        if t == 20:
            x[0, 0, 1], x[0, 0, 2], x[0, 1, 3] = -np.inf, 1e-38, -1e-40
        if t == 37:
            x[0, 0, 0], x[0, 1, 0] = top, -top
        x = rounded(x, "bf16")
        for is_v in (False, True):
            cache.append(None, is_v, 0, table[0], t, t + 1, x[:, int(is_v)])
        xd = cuda(x, torch.bfloat16)
        w8.kv_append(dev, xd[:, :1], xd[:, 1:], i32(table.tolist()), i32([t + 1]))
        assert (dev.k_scale.cpu().numpy() == cache.ks).all(), t
        assert (dev.v_scale.cpu().numpy() == cache.vs).all(), t
        for got, want in ((dev.k, cache.k), (dev.v, cache.v)):
            g, w = got.cpu().numpy(), want
            nan = (g & 127 == 127) & (w & 127 == 127)      # either sign of NaN
            assert (nan | (g == w)).all(), (t, np.argwhere(~(nan | (g == w)))[0])


@pytest.mark.gpu
def test_append_skips_what_no_sequence_owns(w8):
    """Negative positions (an empty slot of a padded batch), columns past the
    block table and pages outside the cache store nothing; queries without a
    position come back as zeros."""
    rng = np.random.default_rng(12)
    cache = ref.Cache(4, 2, 16, 32, rng)
    dev = cache.to(w8)
    # sequence 0 empty, 1 has only its second token, 2 runs past its table,
    # 3 has a page outside the cache
    lens = [0, 1, 18, 2]
    table = np.array([[0], [1], [2], [4]])
    x = rounded(rng.normal(size=(8, 6, 32)), "bf16")
    rt = ref.table64(32, 32).astype(np.float32)
    pos = [-2, -1, -1, 0, 16, 17, 0, 1]
    want_q = ref.rotate32(x[:, :2], rt, [max(p, 0) for p in pos], "half")
    want_q[[0, 1, 2]] = 0
    kr = ref.rotate32(x[:, 2:4], rt, [max(p, 0) for p in pos], "half")
    for h in range(2):
        cache.append(None, False, h, table[1], 0, 1, kr[3:4, h])
        cache.append(None, True, h, table[1], 0, 1, x[3:4, 4 + h])
    xd = cuda(x, torch.bfloat16)
    got = w8.kv_append(dev, xd[:, 2:4], xd[:, 4:], i32(table.tolist()), i32(lens), table=cuda(rt),
                       q=xd[:, :2])
    same_bits(got, torch.from_numpy(want_q).to(torch.bfloat16))
    assert (dev.k.cpu().numpy() == cache.k).all() and (dev.v.cpu().numpy() == cache.v).all()
    assert (dev.k_scale.cpu().numpy() == cache.ks).all()
    # a table too short for a position: the rotated keys and queries are NaN
    got = w8.kv_append(dev, xd[:2, 2:4], xd[:2, 4:], i32([[3], [0]]), i32([1, 9]),
                       table=cuda(rt[:5]), q=xd[:2, :2])
    assert got[1].isnan().all() and not got[0].isnan().any()
    assert (dev.k[0, :, 8].cpu().numpy() & 127 == 127).all()


# --------------------------------------------------------------- attention

def check_attention(w8, new, totals, hq, hkv, dim, page, window=0, causal=True, dtype="bf16", seed=0,
                    plan=None, padded=False, scale=None, spread=1.0, poison=True, strided=False,
                    max_kv=None, uniform=None, mutate=None):
    rng = np.random.default_rng(seed + dim)
    pages = sum(-(-max(t, 0) // page) for t in totals) + 2
    cache = ref.Cache(pages, hkv, page, dim, rng if poison else None)
    table = layout_pages(rng, totals, page, pages)
    for b, t in enumerate(totals):
        for h in range(hkv):
            for is_v in (False, True):
                x = rng.normal(size=(t, dim)) * np.exp(spread * rng.normal(size=(t, 1)))
                cache.append(None, is_v, h, table[b], 0, t, x.astype(np.float32))
    if mutate:
        mutate(cache, table)
    tokens = sum(new)
    q = rounded(rng.normal(size=(tokens, hq * dim + (8 if strided else 0))), dtype)
    qd = cuda(q, DT[dtype])[:, :hq * dim].unflatten(1, (hq, dim))
    scale = dim ** -0.5 if scale is None else scale
    want, lse, tol_o, tol_l = ref.attention64(
        q[:, :hq * dim].reshape(tokens, hq, dim).astype(np.float64), cache, table, totals, new,
        hq // hkv, scale, causal, window)
    uniform = min(new) == max(new) if uniform is None else uniform
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    out = torch.full((tokens, hq, dim + (4 if strided else 0)), 7.0, dtype=DT[dtype],
                     device="cuda")[..., :dim]
    got, got_lse = w8.kv_attention(qd, cache.to(w8, padded), i32(table.tolist()), i32(totals), out,
                                   cu_seqlens=None if uniform else i32(cu), max_new=max(new),
                                   max_kv=max_kv, scale=scale, causal=causal, window=window,
                                   return_lse=True, plan_=plan)
    g, gl = got.cpu().double().numpy(), got_lse.cpu().double().numpy()
    nan = np.isnan(want)
    assert (np.isnan(g) == nan).all(), "NaN at other places: %s" % np.argwhere(np.isnan(g) != nan)[:3]
    tol = tol_o + HALF_ULP[dtype] * np.abs(want) + 2.0 ** -24
    err = np.abs(np.where(nan, 0, g) - np.where(nan, 0, want))
    tol = np.where(nan, 1, tol)
    worst = np.unravel_index(np.argmax(err / tol), err.shape)
    assert (err <= tol).all(), "out %s: %g, want %g, bound %g" % (worst, g[worst], want[worst], tol[worst])
    fin = np.isfinite(lse)
    assert (np.isnan(gl) == np.isnan(lse)).all() and ((gl == -np.inf) == (lse == -np.inf)).all()
    assert (np.abs(gl - lse)[fin] <= tol_l[fin]).all()
    return got, got_lse


ATTEND = [
    # new, held in all, q heads, kv heads, dim, page, window, causal, dtype
    ([1], [1], 1, 1, 16, 16, 0, True, "bf16"),
    ([1, 1, 1, 1, 1], [0, 15, 16, 17, 65], 4, 2, 64, 16, 0, True, "bf16"),
    ([1, 1, 1], [63, 64, 129], 8, 1, 128, 64, 0, True, "fp16"),
    ([1, 1], [300, 77], 16, 1, 128, 32, 0, True, "bf16"),
    ([1, 1], [200, 90], 17, 1, 80, 48, 0, True, "bf16"),
    ([1, 1], [130, 40], 5, 5, 32, 16, 33, True, "fp16"),
    ([4, 4], [70, 4], 6, 2, 96, 32, 0, True, "bf16"),
    ([5, 1, 0, 9], [40, 130, 17, 9], 4, 1, 112, 16, 0, True, "fp16"),
    ([3, 7], [50, 100], 4, 4, 192, 32, 20, True, "bf16"),
    ([2, 2], [66, 31], 4, 2, 256, 16, 0, False, "bf16"),
    ([6, 3], [90, 140], 3, 1, 48, 48, 40, False, "fp16"),
    ([33, 20], [33, 150], 4, 1, 64, 64, 0, True, "bf16"),
    ([70], [200], 2, 2, 128, 128, 0, True, "fp16"),
    ([40, 64], [100, 64], 4, 2, 128, 16, 17, True, "bf16"),
    ([8, 8], [3, 0], 4, 2, 64, 16, 0, True, "bf16"),       # more new tokens than are held
    ([1], [513], 4, 2, 256, 1024, 0, True, "fp16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", ATTEND, ids=[str(i) for i in range(len(ATTEND))])
def test_attention(w8, case):
    check_attention(w8, *case, seed=100)


@pytest.mark.gpu
@pytest.mark.parametrize("waves,chunk_tiles", [(4, 1), (4, 2), (4, 3), (4, 100), (8, 1), (8, 2), (8, 100)])
@pytest.mark.parametrize("case", [1, 3, 6, 8, 10, 13], ids=str)
def test_attention_plans(w8, waves, chunk_tiles, case):
    if waves == 8 and ATTEND[case][4] > 128:
        waves, chunk_tiles = 4, 4
    plan = w8.KVPlan(kernel=w8.KV_KERNEL_ROWS, row_blocks=1, waves=waves, chunk_tiles=chunk_tiles)
    check_attention(w8, *ATTEND[case], seed=200, plan=plan)


@pytest.mark.gpu
@pytest.mark.parametrize("chunk_tiles", [1, 2, 100])
@pytest.mark.parametrize("case", range(len(ATTEND)), ids=str)
def test_attention_tile_kernel(w8, chunk_tiles, case):
    plan = w8.KVPlan(kernel=w8.KV_KERNEL_TILE, row_blocks=8, waves=4, chunk_tiles=chunk_tiles)
    check_attention(w8, *ATTEND[case], seed=250, plan=plan, padded=chunk_tiles == 2,
                    strided=chunk_tiles == 2)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [
    ([150], [700], 4, 1, 128, 64, 0, True, "bf16"),        # whole tiles between hidden ones
    ([70, 3], [400, 333], 3, 1, 64, 16, 250, True, "fp16"),
    ([300], [300], 2, 1, 80, 48, 0, False, "bf16"),
    ([40], [600], 5, 1, 256, 32, 0, True, "bf16"),
    ([64], [500], 2, 1, 192, 32, 300, True, "fp16")], ids=[str(i) for i in range(5)])
def test_attention_many_rows(w8, case):
    check_attention(w8, *case, seed=260)
    for kernel, blocks, tiles in ((w8.KV_KERNEL_TILE, 8, 3), (w8.KV_KERNEL_ROWS, 1, 4)):
        plan = w8.KVPlan(kernel=kernel, row_blocks=blocks, waves=4, chunk_tiles=tiles)
        check_attention(w8, *case, seed=261, plan=plan)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [1, 7, 8, 12], ids=str)
def test_attention_strides_and_small_bounds(w8, case):
    # padded pages, strided queries and outputs, offsets given though uniform,
    # and a max_kv below the longest sequence (the last chunk takes the rest)
    plan = w8.KVPlan(kernel=w8.KV_KERNEL_ROWS, row_blocks=1, waves=4, chunk_tiles=1)
    check_attention(w8, *ATTEND[case], seed=300, padded=True, strided=True, uniform=False)
    check_attention(w8, *ATTEND[case], seed=301, plan=plan, max_kv=64)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, 1e-3, 3.0])
def test_attention_scales(w8, scale):
    check_attention(w8, [2, 3], [70, 150], 4, 2, 64, 16, scale=scale, seed=400)


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [0.0, 6.0])
def test_attention_blocks_of_unlike_size(w8, spread):
    # block scales within 2^22 of each other are exact; exp(6 n) spans about
    # 2^40, whose smallest values are below the bound's share of the largest
    check_attention(w8, [1, 2], [130, 220], 4, 1, 64, 32, spread=spread, scale=1e-6, seed=500)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [6, 8, 9, 11, 13], ids=str)
def test_attention_hidden_nan_does_not_leak(w8, case):
    """NaN codes and NaN scales of tokens some rows see and others do not:
    NaN exactly in the rows (and channels) that see them."""
    new, totals, hq, hkv, dim, page = ATTEND[case][:6]

    def mutate(cache, table):
        for b, t in enumerate(totals):
            if t < 6:
                continue
            for p, what in ((t - 2, "v"), (t // 2, "k" if b % 2 else "v"), (0, "v")):
                kc, vc = cache.parts(table[b, p // page], b % hkv, p % page // ref.BLOCK)
                if what == "v":
                    vc[p % ref.BLOCK, (7 * b + p) % dim] = 0x7F if p % 2 else 0xFF
                else:
                    kc[p % ref.BLOCK, 3] = 0xFF
    check_attention(w8, *ATTEND[case], seed=600, mutate=mutate)
    for tiles in (1, 2):
        for kernel, blocks in ((w8.KV_KERNEL_ROWS, 1), (w8.KV_KERNEL_TILE, 8)):
            plan = w8.KVPlan(kernel=kernel, row_blocks=blocks, waves=4, chunk_tiles=tiles)
            check_attention(w8, *ATTEND[case], seed=601, mutate=mutate, plan=plan)


@pytest.mark.gpu
@pytest.mark.parametrize("byte", [0, 255])
def test_attention_unwritten_block_is_nan(w8, byte):
    def mutate(cache, table):
        cache.ks[table[0, 1], 0, 0] = byte       # tokens 32.. of sequence 0, head 0
        cache.vs[table[1, 0], 1, 1] = byte       # tokens 16.. of sequence 1, head 1
    check_attention(w8, [20, 20], [60, 60], 4, 2, 64, 32, seed=700, mutate=mutate)
    # blocks that every row sees, in the kernels' loops without masks
    for kernel, blocks in ((w8.KV_KERNEL_ROWS, 1), (w8.KV_KERNEL_TILE, 8)):
        plan = w8.KVPlan(kernel=kernel, row_blocks=blocks, waves=4, chunk_tiles=100)
        check_attention(w8, [20, 20], [360, 460], 4, 2, 64, 32, seed=701, mutate=mutate, plan=plan)


@pytest.mark.gpu
def test_attention_page_outside_the_cache_is_nan(w8):
    cache = ref.Cache(4, 1, 16, 32, None)
    cache.ks[:], cache.vs[:] = 127, 127
    dev = cache.to(w8)
    q = torch.ones(3, 2, 32, dtype=torch.bfloat16, device="cuda")
    for bad in (-1, 4, 1 << 30):
        out, lse = w8.kv_attention(q, dev, i32([[0, 1], [2, bad], [3, 0]]), i32([20, 20, 40]),
                                   return_lse=True)
        out = out.cpu()
        # sequence 1 names no page; sequence 2 is longer than its table
        assert (out[0] == 0).all() and out[1].isnan().all() and out[2].isnan().all()
        assert lse[0].isfinite().all() and lse[1:].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("plan", [dict(row_blocks=0), dict(row_blocks=2), dict(kernel=3),
                                  dict(kernel=2, row_blocks=2), dict(chunk_tiles=0), dict(waves=0),
                                  dict(waves=6), dict(kernel=2, row_blocks=8, waves=8)])
def test_attention_plan_refusals(w8, plan):
    p = w8.KVPlan(**dict(dict(kernel=1, row_blocks=1, waves=4, chunk_tiles=1), **plan))
    cache = ref.Cache(1, 1, 16, 16, None).to(w8)
    q = torch.ones(1, 1, 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(w8.W8A16Error) as e:
        w8.kv_attention(q, cache, i32([[0]]), i32([5]), plan_=p)
    assert e.value.status == w8.ERR_BAD_PLAN


@pytest.mark.gpu
def test_attention_infinite_queries(w8):
    def run(v):
        cache = ref.Cache(1, 1, 16, 16, None)
        cache.k[:], cache.ks[:], cache.vs[:] = 0x38, 127, 127     # keys of 1.0
        q = torch.zeros(1, 1, 16, dtype=torch.bfloat16, device="cuda")
        q[0, 0, 0] = v
        return w8.kv_attention(q, cache.to(w8), i32([[0]]), i32([5])).cpu()
    assert run(math.inf).isnan().all() and run(math.nan).isnan().all() and (run(1.0) == 0).all()


@pytest.mark.gpu
def test_append_then_attend_is_what_was_appended(w8):
    """The two operators together, against attention over the reference's
    cache grown by the same tokens, step by step."""
    rng = np.random.default_rng(21)
    hq, hkv, dim, page = 4, 2, 64, 16
    cache = ref.Cache(6, hkv, page, dim, rng)
    dev = cache.to(w8)
    table = np.array([[5, 0, 3], [1, 4, 2]])
    rt = ref.table64(64, dim).astype(np.float32)
    lens = [0, 0]
    for n in ([17, 5], [1, 1], [1, 1], [4, 9], [1, 1]):
        lens = [a + b for a, b in zip(lens, n)]
        x = rounded(rng.normal(size=(sum(n), hq + 2 * hkv, dim)), "bf16")
        xd = cuda(x, torch.bfloat16)
        cu = np.concatenate([[0], np.cumsum(n)])
        pos = np.concatenate([np.arange(t - m, t) for m, t in zip(n, lens)])
        kr = ref.rotate32(x[:, hq:hq + hkv], rt, pos, "half")
        for b in range(2):
            for h in range(hkv):
                rows = slice(cu[b], cu[b + 1])
                cache.append(None, False, h, table[b], lens[b] - n[b], lens[b], kr[rows, h])
                cache.append(None, True, h, table[b], lens[b] - n[b], lens[b], x[rows, hq + hkv + h])
        bt, kv, cud = i32(table.tolist()), i32(lens), i32(cu.tolist())
        q = w8.kv_append(dev, xd[:, hq:hq + hkv], xd[:, hq + hkv:], bt, kv, cu_seqlens=cud,
                         max_new=max(n), table=cuda(rt), q=xd[:, :hq])
        out = w8.kv_attention(q, dev, bt, kv, cu_seqlens=cud, max_new=max(n))
        qn = rounded(ref.rotate32(x[:, :hq], rt, pos, "half"), "bf16")
        want, _, tol, _ = ref.attention64(qn.astype(np.float64), cache, table, lens, n, hq // hkv,
                                          dim ** -0.5, True, 0)
        err = np.abs(out.cpu().double().numpy() - want)
        assert (err <= tol + HALF_ULP["bf16"] * np.abs(want) + 2.0 ** -24).all()


@pytest.mark.gpu
def test_attention_offsets_past_32_bits(w8):
    """Pages more than 4 GiB into the pools: a small cache's pages spread
    over strided pools give the small cache's bits."""
    rng = np.random.default_rng(31)
    hkv, page, dim, pages = 2, 32, 64, 5
    small = ref.Cache(pages, hkv, page, dim, rng)
    table = np.array([[4, 1, 3]])
    for h in range(hkv):
        for is_v in (False, True):
            small.append(None, is_v, h, table[0], 0, 90, rng.normal(size=(90, dim)).astype(np.float32))
    dev = small.to(w8)
    stride = (1 << 30) + (1 << 28)
    pools = []
    for t in dev[:2]:
        flat = torch.empty(stride * (pages - 1) + t[0].numel(), dtype=torch.uint8, device="cuda")
        big = flat.as_strided(t.shape, (stride,) + t.stride()[1:])
        big.copy_(t)
        pools.append(big)
    far = w8.KVCache(pools[0], pools[1], dev.k_scale.clone(), dev.v_scale.clone())
    q = cuda(rng.normal(size=(1, 8, dim)), torch.bfloat16)
    a = w8.kv_attention(q, dev, i32(table.tolist()), i32([90]))
    b = w8.kv_attention(q, far, i32(table.tolist()), i32([90]))
    assert torch.equal(a, b) and not a.isnan().any()
    x = cuda(rng.normal(size=(3, hkv, dim)), torch.bfloat16)
    for c in (dev, far):
        w8.kv_append(c, x, x, i32(table.tolist()), i32([93]))
    assert torch.equal(dev.k, far.k) and torch.equal(dev.v, far.v)


@pytest.mark.gpu
def test_attention_same_bits_again_and_in_a_graph(w8):
    """Repeated calls give the same bits, on another stream too; append and
    attention captured in one graph replay to the eager results, with eager
    work between the replays, as kv_lens advances on the device."""
    rng = np.random.default_rng(41)
    seqs, hq, hkv, dim, page = 3, 8, 2, 128, 16
    table = torch.arange(seqs * 64, dtype=torch.int32, device="cuda").view(seqs, 64)
    x = cuda(rng.normal(size=(8, seqs, hq + 2 * hkv, dim)), torch.bfloat16)
    prompt = cuda(rng.normal(size=(seqs * 700, 2 * hkv, dim)), torch.bfloat16)
    rt = w8.rope_table(1024, dim)

    def fresh():
        c = w8.kv_cache(seqs * 64, hkv, page, dim)
        w8.kv_append(c, prompt[:, :hkv], prompt[:, hkv:], table, i32([700] * seqs), table=rt)
        return c

    def step(c, inp, lens, out, q):
        w8.kv_append(c, inp[:, hq:hq + hkv], inp[:, hq + hkv:], table, lens, table=rt, q=inp[:, :hq], q_out=q)
        return w8.kv_attention(q, c, table, lens, out)

    def bufs():
        e = torch.empty(seqs, hq, dim, dtype=torch.bfloat16, device="cuda")
        return e, torch.empty_like(e)
    cache, lens, eager = fresh(), i32([700] * seqs), []
    out, q = bufs()
    for i in range(8):
        lens += 1
        eager.append(step(cache, x[i], lens, out, q).clone())
    again = w8.kv_attention(q, cache, table, lens)
    assert torch.equal(again, eager[-1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(w8.kv_attention(q, cache, table, lens), eager[-1])
        # the graph, captured on this stream after a call with its plan
        c2, lens2, inp = fresh(), i32([700] * seqs), x[0].clone()
        out2, q2 = bufs()
        w8.kv_attention(q, cache, table, lens)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(c2, inp, lens2, out2, q2)
        for i in range(8):
            inp.copy_(x[i])
            lens2 += 1
            g.replay()
            side.synchronize()
            assert torch.equal(out2, eager[i]), i
            torch.randn(1000, device="cuda").sum().item()
    assert torch.equal(c2.k, cache.k) and torch.equal(c2.v, cache.v)
