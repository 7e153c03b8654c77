"""Attention where its number ranges and its callers' shapes end: weights far
below a row's largest, blocks of very unlike scale, blocks hidden from some
rows, tokens of no sequence, and refusals."""

import ctypes
import math

import numpy as np
import pytest

import attention_ref as ref
import block_scaled_fp8_w8a16_amd as w8mod
from test_attention import HALF_ULP, DT, _descs, check_attention, cuda, i32, rounded, w8  # noqa: F401

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
