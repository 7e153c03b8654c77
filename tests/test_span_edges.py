"""Attention and its cache where callers' shapes end: slots without tokens
beside a shared prefix, caches of one page."""

import numpy as np
import pytest

import attention_ref as ref
import block_scaled_fp8_w8a16_amd as w8mod
from test_attention import DT, cuda, i32, rounded
from test_kv_span import own_plan, w8  # noqa: F401

torch = pytest.importorskip("torch")


def served(rng, new, totals, shared, spare, hq, hkv, dim, page):
    """A cache of the sequences behind `shared` common tokens, `spare` pages
    of other tokens, block table rows of both, and queries."""
    common, own = shared // page, [-(-max(0, t - shared) // page) for t in totals]
    width = common + max(own + [1])
    pages = common + sum(own) + spare
    cache = ref.Cache(pages, hkv, page, dim, rng)
    for h in range(hkv):
        for is_v in (False, True):
            cache.append(None, is_v, h, np.arange(pages), 0, pages * page, rng.normal(size=(pages * page, dim)))
    table, at = np.zeros((len(totals), width), np.int64), common
    for b, n in enumerate(own):
        table[b, :common] = np.arange(common)
        table[b, common:common + n] = np.arange(at, at + n)
        at += n
    return cache, table, np.resize(np.arange(at, pages), width), rounded(rng.normal(size=(sum(new), hq, dim)), "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("slot", ["empty", "decreasing", "past the end"])
@pytest.mark.parametrize("longest", [False, True])
@pytest.mark.parametrize("new", [[1, 2, 1], [40, 3, 50], [1] * 40])
def test_slots_without_tokens_do_not_lead_to_the_prefix(w8, slot, longest, new):
    """A slot that brings no tokens (its offsets agree, decrease or end past
    the token axis) says nothing, whatever length and pages it is left with:
    the bits are those without it."""
    rng = np.random.default_rng(len(new))
    shared, hq, hkv, dim, page = 96, 4, 2, 64, 16
    # longest: no sequence holds all of the prefix
    totals = [max(n, 50 + 7 * i % 40) if longest else shared + n + 5 * i for i, n in enumerate(new)]
    cache, table, other, q = served(rng, new, totals, shared, 12, hq, hkv, dim, page)
    dev, qd = cache.to(w8), cuda(q, DT["bf16"])
    cu = [0] + np.cumsum(new).tolist()
    kw = dict(max_new=max(new), shared=shared, return_lse=True)

    def run(table, totals, cu, plan):
        return w8.kv_attention(qd, dev, cuda(table.astype(np.int32)), i32(totals), cu_seqlens=i32(cu), plan_=plan,
                               **kw)
    front, lens = np.r_[other[None], table], [150] + totals
    stale = {"empty": (front, lens, [0] + cu), "decreasing": (front, lens, [cu[-1]] + cu),
             "past the end": (np.r_[table, other[None]], totals + [150], cu + [cu[-1] + 3])}
    for plan in (own_plan(w8, new, 2, chunk=1), own_plan(w8, new, 2, chunk=50)):
        want = run(table, totals, cu, plan)
        got = run(*stale[slot], plan)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("pitch", [0, 3, 8])
def test_caches_of_one_page(w8, pitch):
    """The pitch of a single page says nothing."""
    heads, page, dim, tokens = 2, 32, 64, 20
    plain = w8.kv_cache(1, heads, page, dim)
    odd = w8.KVCache(*(t.clone().as_strided(t.shape, (t.stride(0) + pitch,) + t.stride()[1:]) for t in plain))
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v, q = (torch.randn(tokens, heads, dim, generator=g, device="cuda").bfloat16() for _ in range(3))
    bt, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), i32([tokens])
    out = []
    for cache in (plain, odd):
        w8.kv_append(cache, k, v, bt, lens)
        out.append(w8.kv_attention(q, cache, bt, lens))
    assert torch.equal(*out) and all(torch.equal(a, b) for a, b in zip(plain, odd))
