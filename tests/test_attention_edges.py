"""Attention where its number ranges and its callers' shapes end: weights far
below a row's largest, blocks of very unlike scale, blocks hidden from some
rows, tokens of no sequence, and refusals."""

import math

import numpy as np
import pytest

import attention_ref as ref
import block_scaled_fp8_w8a16_amd as w8mod
from test_attention import HALF_ULP, DT, _descs, cuda, i32, rounded, w8  # noqa: F401

torch = pytest.importorskip("torch")

ROWS, TILE = (w8mod.KV_KERNEL_ROWS, 1), (w8mod.KV_KERNEL_TILE, 8)


def plan(kernel, chunk_tiles, waves=4):
    return w8mod.KVPlan(kernel=kernel[0], row_blocks=kernel[1], waves=waves, chunk_tiles=chunk_tiles)


def one_row(cache, table, length, q, scale):
    """FP64 attention of one query row q [d] over all of a sequence's keys:
    out, lse and the bound of out's error before it is rounded to its type.

    As in attention64, all but what FP16 adds below its normal range.  A
    weight is held as p 2^(e - E), e the exponent of its block's V scale and E
    a power of two such that the largest of the row is at least 2^10 (the
    reference rounds its logarithm up to a whole number, and 2^11 stands for
    it); below 2^-14 FP16 rounds by up to 2^-25, 2^-35 of that largest."""
    k, v = cache.read(0, table, length)
    unit = np.array([2.0 ** (int(cache.vs[table[p // cache.page], 0, p % cache.page // 16]) - 127)
                     for p in range(length)])
    s = k @ q * scale
    d = len(q)
    e = float(np.max(np.abs(k) @ np.abs(q))) * scale * (d + 4) * 2.0 ** -24
    m = s.max()
    w = np.exp(s - m)
    l = w.sum()
    rel = 4 * e + 2.0 ** -20 + 2.0 ** -11 + 2 * length * 2.0 ** -24
    tol = rel * (w @ np.abs(v)) / l + 2.0 ** -35 * (w * unit).max() * np.abs(v / unit[:, None]).sum(0) / l
    return w @ v / l, m + math.log(l), tol, 2 * e + 2.0 ** -19 + length * 2.0 ** -24 + 2.0 ** -21 * abs(m)


def compare_row(w8, cache, table, length, q, scale, plans, dtype="fp16"):
    want, lse, tol, tol_l = one_row(cache, table, length, q.astype(np.float64), scale)
    tol = tol + HALF_ULP[dtype] * np.abs(want) + (2.0 ** -25 if dtype == "fp16" else 2.0 ** -134)
    top = np.abs(want) - tol > torch.finfo(DT[dtype]).max      # beyond the type: infinite
    dev, qd = cache.to(w8), cuda(q[None, None], DT[dtype])
    for p in plans:
        got, gl = w8.kv_attention(qd, dev, i32([list(map(int, table))]), i32([length]), scale=scale,
                                  return_lse=True, plan_=p)
        g = got.cpu().double().numpy()[0, 0]
        assert (g[top] == np.sign(want[top]) * math.inf).all()
        err = np.abs(np.where(top, want, g) - want)
        worst = int(np.argmax(err / tol))
        assert (err <= tol).all(), "channel %d: %g off %g, bound %g" % (worst, err[worst], want[worst], tol[worst])
        assert abs(gl.item() - lse) <= tol_l


def flat_cache(rng, length, page, dim):
    """One sequence on pages 0, 1, ...: keys of zero, V codes of 0.5 .. 1.9
    of either sign, scales of 1."""
    pages = -(-length // page)
    cache = ref.Cache(pages, 1, page, dim)
    cache.ks[:], cache.vs[:] = 127, 127
    cache.v[:] = rng.integers(0x30, 0x40, cache.v.shape) + 0x80 * rng.integers(0, 2, cache.v.shape)
    return cache, np.arange(pages)


PLANS = [plan(ROWS, 1000), plan(ROWS, 1000, 8), plan(ROWS, 2), plan(TILE, 1000), plan(TILE, 3)]


def name(p):
    return "default" if p is None else "%s-%dx%d" % ("rows" if p.kernel == ROWS[0] else "tile", p.waves, p.chunk_tiles)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("gap", [8.0, 14.0, 16.0, 18.0, 20.0])
def test_weights_far_below_the_largest(w8, gap, dtype):
    """The first key takes nearly all of the weight and has a value of zero;
    the others, each `gap` nats lower, make the output."""
    cache, table = flat_cache(np.random.default_rng(1), 4096, 64, 32)
    cache.v[:] &= 0x7F
    cache.k[0, 0, 0, 0] = 0x38
    cache.v[0, 0, 0, :, 0] = 0
    q = np.zeros(32, np.float32)
    q[0] = 1
    compare_row(w8, cache, table, 4096, q, gap, PLANS, dtype)


def rows_of(w8, cache, table, total, new, q, p, window):
    out, lse = w8.kv_attention(q, cache.to(w8), i32([list(map(int, table))]), i32([total]), window=window,
                               return_lse=True, plan_=p, max_new=new)
    return out.cpu(), lse.cpu()


@pytest.mark.gpu
@pytest.mark.parametrize("byte", [1, 160, 254])
@pytest.mark.parametrize("p", PLANS, ids=name)
@pytest.mark.parametrize("dim", [64, 128, 192])
def test_scales_of_hidden_blocks_change_nothing(w8, byte, p, dim):
    """A block's V scale of any size changes only the rows that see the
    block: bit for bit in the others, whether it lies before every row's
    window in the first tile they read, before some rows' windows, or on
    tokens that only later rows see."""
    if p.waves == 8 and dim > 128:
        p = plan(ROWS, 1000)
    rng = np.random.default_rng(2)
    total, new, group = 200, 40, 2
    cache, table = flat_cache(rng, total, 16, dim)
    cache.k[:] = rng.integers(0x20, 0x38, cache.k.shape) + 0x80 * rng.integers(0, 2, cache.k.shape)
    q = cuda(rng.normal(size=(new, group, dim)), torch.bfloat16)
    pos = np.arange(total - new, total)
    for window, block in ((70, 4), (70, 6), (0, 12), (0, 11), (70, 11)):
        plain = rows_of(w8, cache, table, total, new, q, p, window)
        other = ref.Cache(cache.pages, 1, 16, dim)
        for a, b in zip((other.k, other.v, other.ks, other.vs), (cache.k, cache.v, cache.ks, cache.vs)):
            a[:] = b
        other.vs[table[block], 0, 0] = byte
        got = rows_of(w8, other, table, total, new, q, p, window)
        lo = np.maximum(0, pos - window + 1) if window else 0 * pos
        sees = torch.from_numpy((pos >= 16 * block) & (lo < 16 * block + 16))
        assert (~sees).any()
        for a, b in zip(got, plain):
            assert torch.equal(a[~sees], b[~sees]), (window, block)
        if sees.any():
            assert not torch.equal(got[0][sees], plain[0][sees])


@pytest.mark.gpu
@pytest.mark.parametrize("up", [18, 40, 100])
def test_a_large_block_of_little_weight(w8, up):
    """A block whose V scale is 2^up larger but whose keys weigh next to
    nothing leaves the others their precision."""
    cache, table = flat_cache(np.random.default_rng(3), 700, 32, 48)
    cache.k[1, 0, 16:, 0] = 0xB8                # block 3: keys of -1
    cache.vs[1, 0, 1] = 127 + up
    q = np.zeros(48, np.float32)
    q[0] = 1
    compare_row(w8, cache, table, 700, q, up * math.log(2) + 12, PLANS, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("up", [12, 15, 18, 22])
def test_subnormal_codes_beside_a_larger_block(w8, up):
    """Equal weights, one block 2^up larger with codes of zero in most
    channels, the others of subnormal codes: these keep their precision."""
    rng = np.random.default_rng(4)
    cache, table = flat_cache(rng, 600, 16, 64)
    cache.v[:] = rng.integers(1, 8, cache.v.shape)
    cache.v[7] = 0
    cache.v[7, 0, 0, ::8] = 0x38
    cache.vs[7, 0, 0] = 127 + up
    compare_row(w8, cache, table, 600, np.zeros(64, np.float32), 1.0, PLANS)


@pytest.mark.gpu
@pytest.mark.parametrize("bytes_", [(1, 127), (1, 240), (1, 254)])
def test_blocks_of_every_scale(w8, bytes_):
    """V scales at both ends of their range in one row, zero codes (what an
    append of zeros stores: byte 1) among them; the sums see the keys of all
    blocks."""
    rng = np.random.default_rng(5)
    cache, table = flat_cache(rng, 900, 16, 32)
    small = rng.random(cache.vs.shape[0]) < 0.5
    cache.v[small] = 0
    cache.vs[small], cache.vs[~small] = bytes_
    if bytes_[1] > 240:
        cache.v[~small] = rng.integers(1, 8, cache.v[~small].shape)      # within the type's range
    cache.k[:] = rng.integers(0x20, 0x38, cache.k.shape) + 0x80 * rng.integers(0, 2, cache.k.shape)
    q = rounded(rng.normal(size=32), "bf16")
    compare_row(w8, cache, table, 900, q, 0.4, PLANS, "bf16")
    cache.vs[:], cache.v[:] = rng.integers(1, 240, cache.vs.shape), rng.integers(0, 0x7F, cache.v.shape)
    compare_row(w8, cache, table, 900, q, 3.0, PLANS, "bf16")


def attend_into(w8, q, cache, table, lens, cu, p, max_new):
    """out and lse over memory that held 7 everywhere."""
    out = torch.full((q.shape[0], q.shape[1], q.shape[2] + 4), 7.0, dtype=q.dtype, device="cuda")
    for _ in range(4):      # what the call's lse may be allocated from
        torch.full((q.shape[0], q.shape[1]), 7.0, device="cuda")
    got, lse = w8.kv_attention(q, cache, table, lens, out[..., :q.shape[2]], cu_seqlens=cu, max_new=max_new,
                               plan_=p, return_lse=True)
    assert (out[..., q.shape[2]:] == 7).all()
    return got.cpu(), lse.cpu()


@pytest.mark.gpu
@pytest.mark.parametrize("p", [None] + PLANS, ids=name)
@pytest.mark.parametrize("cu,owners", [
    ([0, 3, 7], [(0, 0, 3), (1, 3, 7)]),                      # a batch of fixed capacity
    ([2, 3, 7], [(0, 2, 3), (1, 3, 7)]), ([0, 0, 0], []), ([300, 300, 300], []),
    ([0, 3, 301], [(0, 0, 3)]),                               # past the token axis
    ([0, 3, 2], [(0, 0, 3)]), ([-1, 3, 7], [(1, 3, 7)]), ([0, 1 << 30, 5], []), ([0, 290, 300], None)])
def test_tokens_of_no_sequence_give_zeros(w8, cu, owners, p):
    rng = np.random.default_rng(6)
    tokens, hq, hkv, dim, held = 300, 6, 2, 80, [400, 333]
    cache = ref.Cache(30, hkv, 32, dim, rng)
    cache.ks[:], cache.vs[:] = rng.integers(120, 125, (2,) + cache.ks.shape)
    for x in (cache.k, cache.v):
        x[:] = rng.integers(0, 0x70, x.shape)
    dev, table, lens = cache.to(w8), i32(rng.permutation(30)[:26].reshape(2, 13).tolist()), i32(held)
    q = cuda(rng.normal(size=(tokens, hq, dim)), torch.bfloat16)
    got, lse = attend_into(w8, q, dev, table, lens, i32(cu), p, 290)
    if owners is None:
        owners = [(0, 0, 290), (1, 290, 300)]
    none = torch.ones(tokens, dtype=torch.bool)
    for b, first, end in owners:
        want = w8.kv_attention(q[first:end], dev, table[b:b + 1], lens[b:b + 1], return_lse=True,
                               plan_=p if p is not None else w8.plan_kv_attention(2, 290, 416, hq, hkv, dim))
        assert torch.equal(got[first:end], want[0].cpu()) and torch.equal(lse[first:end], want[1].cpu())
        none[first:end] = False
    assert (got[none] == 0).all() and (lse[none] == -math.inf).all()


@pytest.mark.gpu
@pytest.mark.parametrize("cu,owners", [([0, 3, 9], [(0, 0, 3)]), ([0, 3, 6], [(0, 0, 3), (1, 3, 6)]),
                                       ([2, 4, 8], [(0, 2, 4), (1, 4, 8)]), ([-1, 3, 6], [(1, 3, 6)]),
                                       ([0, 0, 0], []), ([9, 9, 9], [])])
def test_append_of_tokens_of_no_sequence(w8, cu, owners):
    """What the attention takes for no sequence's token, the append does too:
    nothing stored, its query zero."""
    rng = np.random.default_rng(8)
    cache = ref.Cache(2, 2, 32, 48)
    cache.ks[:], cache.vs[:] = 120, 120      # tokens held before, of codes that are numbers
    for c in (cache.k, cache.v):
        c[:] = rng.integers(0, 0x70, c.shape)
    dev, held = cache.to(w8), [20, 31]
    x = rounded(rng.normal(size=(8, 8, 48)), "bf16")
    rt = ref.table64(40, 48).astype(np.float32)
    want = np.zeros((8, 4, 48), np.float32)
    for b, first, end in owners:
        pos, start = np.arange(held[b] - (end - first), held[b]), held[b] - (end - first)
        want[first:end] = ref.rotate32(x[first:end, :4], rt, pos, "half")
        kr = ref.rotate32(x[first:end, 4:6], rt, pos, "half")
        for h in range(2):
            cache.append(None, False, h, [b], start, held[b], kr[:, h])
            cache.append(None, True, h, [b], start, held[b], x[first:end, 6 + h])
    xd = cuda(x, torch.bfloat16)
    got = w8.kv_append(dev, xd[:, 4:6], xd[:, 6:], i32([[0], [1]]), i32(held), cu_seqlens=i32(cu),
                       table=cuda(rt), q=xd[:, :4])
    assert torch.equal(got.cpu(), torch.from_numpy(want).to(torch.bfloat16))
    for g, w in zip(dev, (cache.k, cache.v, cache.ks, cache.vs)):
        assert (g.cpu().numpy() == w).all()


@pytest.mark.gpu
@pytest.mark.parametrize("p", [None] + PLANS, ids=name)
def test_scores_of_minus_infinity_are_not_hidden_keys(w8, p):
    """A row all of whose visible keys score -inf has no softmax: NaN, and a
    log-sum of -inf, unlike a row that sees nothing; beside finite scores
    they weigh nothing."""
    cache, table = flat_cache(np.random.default_rng(7), 300, 16, 32)
    cache.k[:] = 0x38
    cache.k[0, 0, 0] = 0
    q = torch.zeros(3, 1, 32, dtype=torch.bfloat16, device="cuda")
    q[:, 0, 0] = -math.inf
    dev = cache.to(w8)
    cache.k[0, 0, 0] = 0x38
    other = cache.to(w8)
    bt = i32([list(map(int, table))] * 3)
    for c in (dev, other):
        out, lse = w8.kv_attention(q, c, bt, i32([300, 1, 0]), return_lse=True, plan_=p)
        out, lse = out.cpu(), lse.cpu()
        if c is other:
            assert out[:2].isnan().all() and (lse[:2] == -math.inf).all()
        else:       # -inf times a key of zero
            assert out[:2].isnan().all() and lse[:2].isnan().all()
        assert (out[2] == 0).all() and lse[2] == -math.inf


@pytest.mark.gpu
def test_workspace_refusal_during_capture_names_the_attention(w8):
    cache = ref.Cache(64, 1, 64, 64, None).to(w8)
    # (more chunks than any other test asks for: 142 MB)
    q = torch.ones(512, 4, 64, dtype=torch.bfloat16, device="cuda")
    table, lens = i32([list(range(64))] * 512), i32([4096] * 512)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out = torch.empty_like(q)
        x = torch.zeros(8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            x += 1
            with pytest.raises(w8.W8A16Error) as e:
                w8.kv_attention(q, cache, table, lens, out, plan_=plan(ROWS, 1))
        g.replay()
        side.synchronize()
    assert e.value.status == w8.ERR_WORKSPACE and (x == 1).all()
    assert "w8a16_kv_attention: this plan needs" in str(e.value) and "split-K" not in str(e.value)
    assert "split-K" not in w8.status_string(w8.ERR_WORKSPACE)


@pytest.mark.gpu
def test_outputs_belong_to_the_given_stream(w8):
    """A call on a given stream makes its outputs there: not from memory that
    work of the current stream, still to run, will write."""
    cache = w8.kv_cache(64, 2, 64, 64)
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    table, lens = i32([list(range(64))]), i32([4096])
    x = torch.randn(4096, 2, 64, device="cuda").bfloat16()
    q = torch.randn(4096, 4, 64, device="cuda").bfloat16()[:, :, ::1]
    pos, rt = torch.arange(4096, dtype=torch.int32, device="cuda"), w8.rope_table(4096, 64)
    w8.kv_append(cache, x, x, table, lens, table=rt)
    torch.cuda.synchronize()
    calls = [lambda s: [w8.rope(q, rt, pos, stream=s)],
             lambda s: [w8.kv_append(cache, x, x, table, lens, table=rt, q=q, stream=s)],
             lambda s: list(w8.kv_attention(q, cache, table, lens, return_lse=True, stream=s)),
             lambda s: [w8.rope_table(2048, 512, stream=s)]]
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        got = call(side)
        torch.cuda.synchronize()
        del got
        # memory of the outputs' sizes, freed while the current stream has
        # still to write it
        held = [torch.empty_like(w) for w in want]
        torch.cuda._sleep(200_000_000)
        for h in held:
            h.fill_(3.0)
        del h, held
        got = call(side)
        side.synchronize()
        assert not main.query()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("at,dtype", [(0, "float8_e5m2"), (1, "float8_e4m3fnuz"), (0, "int8"), (1, "bool"),
                                      (2, "float8_e4m3fn"), (3, "int8"), (0, "float8_e8m0fnu")])
def test_cache_types_are_checked(at, dtype):
    cache = list(w8mod.kv_cache(2, 1, 32, 16, device="cpu"))
    cache[at] = cache[at].view(getattr(torch, dtype))
    one, i = torch.zeros(1, 1, 16), torch.zeros(1, 1, dtype=torch.int32)
    for call in (lambda: w8mod.kv_append(cache, one, one, i, i[0]),
                 lambda: w8mod.kv_attention(one.bfloat16(), cache, i, i[0])):
        with pytest.raises(ValueError, match="float8_e4m3fn"):
            call()


@pytest.mark.parametrize("strides", [(0, 64), (256, 0), (63, 1000), (256, -63), (-1, 64)])
def test_outputs_that_overlap_themselves_are_refused(strides):
    lib = w8mod.library()
    c, s, ap, at = _descs(at__out_token_stride=strides[0], at__out_head_stride=strides[1],
                          ap__q_out_token_stride=strides[0], ap__q_out_head_stride=strides[1])
    assert lib.w8a16_kv_attention(c, s, at, 0) == w8mod.ERR_SHAPE and "overlap" in w8mod.last_error()
    assert lib.w8a16_kv_append(c, s, ap, 0) == w8mod.ERR_SHAPE and "overlap" in w8mod.last_error()
    assert lib.w8a16_rope(16, 256, 64, 16, strides[0], strides[1], 1, 4, 4, 64, 16, 8, 64, 16, 0, 0,
                          0) == w8mod.ERR_SHAPE and "overlap" in w8mod.last_error()
