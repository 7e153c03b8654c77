"""Timing cases of the attention operators: rotary positions, appending to the
paged FP8 cache, and attention over that cache.

Cache layout (shared by both forms): blocks of 16 tokens inside pages.
    k        E4M3 codes [pages, kv_heads, page_size, head_dim]
    v        E4M3 codes [pages, kv_heads, page_size / 16, head_dim, 16]
    k_scale  E8M0 bytes [pages, kv_heads, page_size / 16]: a code stands for
    v_scale  code * 2^(byte - 127)
block_table[b, i] is the page of sequence b's tokens i * page_size onwards,
kv_lens[b] the tokens sequence b holds with the new ones counted, and
cu_seqlens the offsets of the sequences' new tokens in the flat token axis.

``own`` False computes the operators with elementary torch operations in
FP32; True calls the package.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 16


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a small batch: a few rows, pure call latency
        dict(name="rope_decode", op="rope", dtype="bf16", tokens=8, heads=32, head_dim=128,
             rot=128, layout="half", inverse=False, pitch=0),
        # the queries of a long prefill chunk, read out of fused QKV rows
        # (32 + 2 * 8 heads of 128), an odd number of tokens
        dict(name="rope_prefill_strided", op="rope", dtype="bf16", tokens=16381, heads=32,
             head_dim=128, rot=128, layout="half", inverse=False, pitch=6144),
        # gradient of a rotation of part of the head, adjacent pairs
        dict(name="rope_grad_partial", op="rope", dtype="fp16", tokens=4097, heads=40,
             head_dim=96, rot=64, layout="interleaved", inverse=True, pitch=0),
        # one decode step of four sequences, queries rotated in the same call
        dict(name="append_decode_4", op="append", dtype="bf16", seqs=4, new=1, ragged=False,
             past=1023, q_heads=32, kv_heads=8, head_dim=128, page=64, rot=128, layout="half"),
        # one decode step of a full serving batch, small pages, partial rotation
        dict(name="append_decode_256", op="append", dtype="bf16", seqs=256, new=1, ragged=True,
             past=2047, q_heads=40, kv_heads=8, head_dim=128, page=16, rot=64,
             layout="interleaved"),
        # ragged prompts joining a batch, some of them continuing inside a block
        dict(name="append_prefill", op="append", dtype="bf16", seqs=6, new=4099, ragged=True,
             past=777, q_heads=32, kv_heads=8, head_dim=128, page=64, rot=128, layout="half"),
        # short continuations (a draft's accepted tokens) without a rotation
        dict(name="append_short_fp16", op="append", dtype="fp16", seqs=48, new=7, ragged=True,
             past=501, q_heads=16, kv_heads=16, head_dim=80, page=32, rot=0, layout="half"),
        # first tokens of one conversation: call latency
        dict(name="attend_single_300", op="attend", dtype="bf16", seqs=1, new=1, ragged=False,
             past=299, q_heads=32, kv_heads=8, head_dim=128, page=64, window=0, causal=True),
        # decode step of a serving batch with mixed lengths: bandwidth
        dict(name="attend_decode_64", op="attend", dtype="bf16", seqs=64, new=1, ragged=True,
             past=8191, q_heads=32, kv_heads=8, head_dim=128, page=64, window=0, causal=True),
        # one long document, one token at a time: the cache split over the chip
        dict(name="attend_long_131k", op="attend", dtype="bf16", seqs=1, new=1, ragged=False,
             past=131071, q_heads=64, kv_heads=8, head_dim=128, page=128, window=0, causal=True),
        # drafts checked five at a time, sliding window, small pages, odd lengths
        dict(name="attend_draft_window", op="attend", dtype="fp16", seqs=24, new=5, ragged=True,
             past=3001, q_heads=40, kv_heads=8, head_dim=64, page=16, window=1024, causal=True),
        # a chunk of a long prompt against what is cached before it: compute
        dict(name="attend_prefill_chunk", op="attend", dtype="bf16", seqs=2, new=2048,
             ragged=False, past=6144, q_heads=32, kv_heads=8, head_dim=128, page=64, window=0,
             causal=True),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(hi, max(lo, n))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["rope", "append", "append", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    head_dim = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
    group = rng.choice([1, 2, 4, 4, 5, 8])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    layout = rng.choice(["half", "interleaved"])
    if op == "rope":
        heads = kv_heads * group
        tokens = min(_log_int(rng, 1, 16000), (1 << 26) // (heads * head_dim))
        return dict(op=op, dtype=rng.choice([dtype, "fp32"]), tokens=tokens, heads=heads,
                    head_dim=head_dim, rot=rng.choice([head_dim, head_dim // 2]), layout=layout,
                    inverse=rng.random() < 0.4,
                    pitch=rng.choice([0, 0, heads * head_dim + 16 * rng.randint(1, 64)]))
    if op == "append":
        seqs = _log_int(rng, 1, 256)
        new = rng.choice([1, 1, _log_int(rng, 2, 4000)])
        new = max(1, min(new, 24000 // seqs))
        return dict(op=op, dtype=dtype, seqs=seqs, new=new, ragged=rng.random() < 0.7,
                    past=_log_int(rng, 1, 2047), q_heads=kv_heads * group, kv_heads=kv_heads,
                    head_dim=head_dim, page=page, rot=rng.choice([0, head_dim // 2, head_dim]),
                    layout=layout)
    kind = rng.choice(["decode", "decode", "long", "draft", "prefill"])
    window = rng.choice([0, 0, 0, _log_int(rng, 100, 4000)])
    causal = True
    if kind == "decode":
        seqs, new, past = _log_int(rng, 1, 128), 1, _log_int(rng, 1, 8000)
    elif kind == "long":
        seqs, new, past = rng.randint(1, 3), 1, _log_int(rng, 9000, 131071)
    elif kind == "draft":
        seqs, new, past = _log_int(rng, 1, 48), rng.randint(2, 9), _log_int(rng, 1, 8000)
        causal = rng.random() < 0.9
    else:
        seqs, new, past = rng.randint(1, 3), _log_int(rng, 17, 2048), _log_int(rng, 1, 6000)
    # at most the largest listed cases' cache and products
    per = max(1, kv_heads * group * head_dim)
    if kind == "prefill":
        while seqs * new * (past + new) * per > 2 * 2048 * 8192 * 4096:
            new = max(1, new // 2)
    while seqs > 1 and seqs * (past + new) * kv_heads * head_dim > 64 * 8192 * 1024:
        seqs //= 2
    while seqs > 1 and seqs * new * (past + new) * kv_heads * group > 2 * 2048 * 8192 * 32:
        seqs //= 2
    return dict(op=op, dtype=dtype, seqs=seqs, new=new, ragged=rng.random() < 0.7, past=past,
                q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, page=page,
                window=window, causal=causal)


def _lengths(case):
    """(new tokens, tokens held with them) of each sequence, as lists."""
    new, total = [], []
    for b in range(case["seqs"]):
        f = 1.0 - 0.75 * ((0.6180339887 * b) % 1.0) if case["ragged"] else 1.0
        g = 1.0 - 0.5 * ((0.4142135624 * b) % 1.0) if case["ragged"] else 1.0
        n = max(1, int(round(case["new"] * g)))
        new.append(n)
        total.append(n + int(round(case["past"] * f)))
    return new, total


def _visible(case):
    """(query, key) pairs that see each other, and keys that some query sees."""
    pairs = keys = 0
    for n, t in zip(*_lengths(case)):
        w = case["window"] or t
        first = t
        for p in range(t - n, t):
            hi = p if case["causal"] else t - 1
            lo = max(0, p - w + 1)
            pairs += hi - lo + 1
            first = min(first, lo)
        keys += t - first
    return pairs, keys


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    d = case["head_dim"]
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * d
        return {"bytes": 2 * n * size + case["tokens"] * (case["rot"] * 4 + 4),
                "flops": 3 * case["tokens"] * case["heads"] * case["rot"]}
    new, total = _lengths(case)
    tokens, kvd = sum(new), case["kv_heads"] * d
    if case["op"] == "append":
        rot = case["rot"]
        by = tokens * (2 * kvd * size + 2 * kvd + rot * 4)      # k, v in; codes out; table
        by += 2 * tokens * case["q_heads"] * d * size if rot else 0
        return {"bytes": by, "flops": tokens * (3 * rot * (case["q_heads"] + case["kv_heads"]) + 4 * kvd)}
    pairs, keys = _visible(case)
    by = keys * (2 * kvd + 2 * case["kv_heads"] / BLOCK)
    by += tokens * case["q_heads"] * (2 * d * size + 4) + 4 * sum(-(-t // case["page"]) for t in total)
    return {"bytes": by, "flops": 4 * d * case["q_heads"] * pairs}


# ------------------------------------------------------------------ inputs

def _table(positions, rot, base=500000.0):
    """[positions, rot / 2, 2] FP32 cosines and sines."""
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack((a.cos(), a.sin()), dim=-1).float()


def _codes(x):
    """E4M3 codes and E8M0 bytes of blocks x [..., 16, head_dim]."""
    amax = x.abs().amax(dim=(-1, -2))
    byte = (((amax.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=1)
    code = (x * _power(254 - byte)[..., None, None]).to(torch.float8_e4m3fn)
    return code, byte.to(torch.uint8)


def _power(field):
    """2^(field - 127) in FP32 of exponent fields 1..254 (0 below them)."""
    return (field.int().clamp(min=0) << 23).view(torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = _DTYPES[case["dtype"]]
    d = case["head_dim"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] == "rope":
        t, h = case["tokens"], case["heads"]
        pitch = case["pitch"] or h * d
        x = randn(t, pitch).to(dtype)[:, :h * d].view(t, h, d) if not case["pitch"] else \
            randn(t, pitch).to(dtype)[:, :h * d].unflatten(1, (h, d))
        start = int(torch.randint(0, 1000, (1,), generator=gen, device="cuda"))
        pos = (torch.arange(t, device="cuda") + start).to(torch.int32)
        return dict(case=case, x=x, pos=pos, table=_table(t + 1000, case["rot"]))

    new, total = _lengths(case)
    order = torch.randperm(case["seqs"], generator=gen, device="cuda").tolist()
    new, total = [new[i] for i in order], [total[i] for i in order]
    seqs, hq, hkv, page = case["seqs"], case["q_heads"], case["kv_heads"], case["page"]
    need = [-(-t // page) for t in total]
    width = max(need)
    pages = sum(need) + max(4, sum(need) // 16)
    perm = torch.randperm(pages, generator=gen, device="cuda")
    used = torch.tensor(need, device="cuda")
    first = used.cumsum(0) - used
    col = torch.arange(width, device="cuda")
    at = (first[:, None] + col).clamp(max=pages - 1)
    table = torch.where(col < used[:, None], perm[at], torch.zeros_like(at)).to(torch.int32)
    # keys and values as a trained model's: channels and heads of unlike size
    blocks = page // BLOCK
    k = randn(pages, hkv, blocks, BLOCK, d) * (1.0 + randn(hkv, 1, 1, d).abs())
    k, k_scale = _codes(k)
    v = randn(pages, hkv, blocks, BLOCK, d) * torch.exp(0.5 * randn(pages, hkv, blocks, 1, 1))
    v, v_scale = _codes(v)
    v = v.view(torch.uint8).transpose(-1, -2).contiguous().view(torch.float8_e4m3fn)
    state = dict(case=case, k=k.view(pages, hkv, page, d), v=v, k_scale=k_scale, v_scale=v_scale,
                 block_table=table, kv_lens=torch.tensor(total, dtype=torch.int32, device="cuda"),
                 max_new=max(new), max_kv=max(total))
    lens = torch.tensor(new, dtype=torch.int32, device="cuda")
    cu = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    cu[1:] = lens.cumsum(0)
    state["cu"] = cu
    state["uniform"] = min(new) == max(new)
    tokens = sum(new)
    if case["op"] == "attend":
        q = randn(tokens, hq, d) * 0.6
        state["q"] = q.to(dtype)
        return state
    # one fused row per token, as the projections leave it
    qkv = randn(tokens, (hq + 2 * hkv) * d).to(dtype)
    state["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
    state["kn"] = (qkv[:, hq * d:(hq + hkv) * d]).unflatten(1, (hkv, d))
    state["vn"] = (qkv[:, (hq + hkv) * d:]).unflatten(1, (hkv, d))
    state["table"] = _table(max(total), case["rot"]) if case["rot"] else None
    return state


# -------------------------------------------------------------- plain form

def _rotate(x, cs, rot, layout, inverse=False):
    """x FP32 [tokens, heads, d] rotated by cs [tokens, rot / 2, 2]."""
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    if inverse:
        s = -s
    r = x[..., :rot]
    if layout == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
    else:
        a, b = r[..., 0::2], r[..., 1::2]
    ya, yb = a * c - b * s, b * c + a * s
    y = torch.cat((ya, yb), -1) if layout == "half" else torch.stack((ya, yb), -1).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _places(state, tokens):
    """Sequence and position of each new token."""
    cu, lens = state["cu"].long(), state["kv_lens"].long()
    t = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b + 1] + lens[b]


def _plain_append(state):
    case = state["case"]
    page, rot = case["page"], case["rot"]
    kn, vn, q = state["kn"].float(), state["vn"].float(), state["q"]
    tokens, hkv, d = kn.shape
    if rot:
        _, pos = _places(state, tokens)
        cs = state["table"][pos]
        kn = _rotate(kn, cs, rot, case["layout"])
        q = _rotate(q.float(), cs, rot, case["layout"]).to(q.dtype)
    cu, lens = state["cu"].long(), state["kv_lens"].long()
    start = lens - (cu[1:] - cu[:-1])
    # every block a sequence's new tokens may lie in, its 16 slots' positions
    blk = start[:, None] // BLOCK + torch.arange(state["max_new"] // BLOCK + 2, device="cuda")
    b, i = torch.nonzero(blk * BLOCK < lens[:, None], as_tuple=True)
    blk = blk[b, i]
    p = blk[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    is_new = (p >= start[b, None]) & (p < lens[b, None])
    is_old = p < start[b, None]
    src = (cu[b, None] + p - start[b, None]).clamp(0, tokens - 1)
    pg = state["block_table"].long()[b, blk * BLOCK // page]
    sb = blk % (page // BLOCK)
    pools = ((state["k"].view(-1, hkv, page // BLOCK, BLOCK, d), state["k_scale"], kn),
             (state["v"].transpose(-1, -2), state["v_scale"], vn))
    _store_blocks(*pools[0], pg, sb, src, is_new, is_old)
    _store_blocks(*pools[1], pg, sb, src, is_new, is_old)
    out = [state["k"], state["v"], _scale_values(state["k_scale"]), _scale_values(state["v_scale"])]
    return out + [q] if rot else out


def _scale_values(byte):
    return byte.view(torch.float8_e8m0fnu)


def _store_blocks(pool, scale, x, pg, sb, src, is_new, is_old):
    """Quantise the new tokens of blocks (pg, sb) beside the tokens they hold."""
    codes = pool.view(torch.uint8)[pg, :, sb]                    # [n, heads, 16, d]
    old_byte = scale[pg, :, sb].int()                            # [n, heads]
    new = is_new[:, None, :, None]
    old = is_old[:, None, :, None]
    xs = x[src].transpose(1, 2)                                  # [n, heads, 16, d]
    amax = torch.where(new & xs.isfinite(), xs.abs(), 0.0).amax(dim=(-1, -2))
    byte = (((amax.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=1)
    byte = torch.where(is_old.any(-1)[:, None], torch.maximum(byte, old_byte), byte)
    held = codes.view(torch.float8_e4m3fn).float() * _power(127 + old_byte - byte)[..., None, None]
    y = torch.where(old, held, xs * _power(254 - byte)[..., None, None])
    y = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    pool.view(torch.uint8)[pg, :, sb] = torch.where(new | old, y, codes)
    scale[pg, :, sb] = byte.to(torch.uint8)


def _plain_attend(state):
    case = state["case"]
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    g, seqs, nq = hq // hkv, case["seqs"], state["max_new"]
    q, cu, lens = state["q"], state["cu"].long(), state["kv_lens"].long()
    tokens = q.shape[0]
    pg = state["block_table"].long()[:, :-(-state["max_kv"] // page)]
    s_len = pg.shape[1] * page
    ks, vs = _power(state["k_scale"][pg]), _power(state["v_scale"][pg])  # [seqs, n, heads, blocks]
    k = state["k"].view(torch.uint8)[pg].view(torch.float8_e4m3fn).float()
    k = (k.unflatten(3, (-1, BLOCK)) * ks[..., None, None]).transpose(1, 2).reshape(seqs, hkv, s_len, d)
    v = state["v"].view(torch.uint8)[pg].view(torch.float8_e4m3fn).float()
    v = (v * vs[..., None, None]).transpose(-1, -2).transpose(1, 2).reshape(seqs, hkv, s_len, d)
    n_new = cu[1:] - cu[:-1]
    i = torch.arange(nq, device="cuda")
    at = (cu[:-1, None] + i).clamp(max=tokens - 1)
    qp = q.float()[at].view(seqs, nq, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(seqs, hkv, g * nq, d)
    s = (qp @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(seqs, hkv, g, nq, s_len)
    j = torch.arange(s_len, device="cuda")
    pos = (lens - n_new)[:, None] + i
    see = j < lens[:, None, None]
    if case["causal"]:
        see = see & (j <= pos[..., None])
    if case["window"]:
        see = see & (j > pos[..., None] - case["window"])
    s.masked_fill_(~see[:, None, None].expand_as(s), -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    v = torch.where((j < lens[:, None])[:, None, :, None], v, 0.0)
    o = (p.view(seqs, hkv, g * nq, s_len) @ v).view(seqs, hkv, g, nq, d) / l
    lse = (m + l.log())[..., 0]
    b, _ = _places(state, tokens)
    r = torch.arange(tokens, device="cuda") - cu[b]
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs, nq, hq, d)[b, r]
    lse = lse.permute(0, 3, 1, 2).reshape(seqs, nq, hq)[b, r]
    return [o.to(q.dtype), lse]


def _plain(state):
    case = state["case"]
    if case["op"] == "rope":
        x = state["x"]
        cs = state["table"][state["pos"].long()]
        return _rotate(x.float(), cs, case["rot"], case["layout"], case["inverse"]).to(x.dtype)
    return _plain_append(state) if case["op"] == "append" else _plain_attend(state)


# --------------------------------------------------------------------- run

def run(state):
    if not own:
        return _plain(state)
    import block_scaled_fp8_w8a16_amd as w8
    case = state["case"]
    if case["op"] == "rope":
        return w8.rope(state["x"], state["table"], state["pos"], layout=case["layout"],
                       inverse=case["inverse"])
    cache = w8.KVCache(state["k"], state["v"], state["k_scale"], state["v_scale"])
    cu = None if state["uniform"] else state["cu"]
    if case["op"] == "append":
        rot = case["rot"]
        q = w8.kv_append(cache, state["kn"], state["vn"], state["block_table"], state["kv_lens"],
                         cu_seqlens=cu, max_new=state["max_new"], table=state["table"],
                         layout=case["layout"], q=state["q"] if rot else None)
        out = [state["k"], state["v"], _scale_values(state["k_scale"]),
               _scale_values(state["v_scale"])]
        return out + [q] if rot else out
    out, lse = w8.kv_attention(state["q"], cache, state["block_table"], state["kv_lens"],
                               cu_seqlens=cu, max_new=state["max_new"], max_kv=state["max_kv"],
                               causal=case["causal"], window=case["window"], return_lse=True)
    return [out, lse]


# ----------------------------------------------------------- 64-bit values

def _exact_rotate(x, pos, table, rot, layout, sign=1.0):
    """Rotation as a product of complex numbers, FP64."""
    cs = torch.view_as_complex(table[pos.long()].double().contiguous())[:, None]
    cs = cs if sign > 0 else cs.conj()
    y = x.double().clone()
    if layout == "half":
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * cs
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:rot:2].contiguous(), y[..., 1:rot:2].contiguous()) * cs
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def _e4m3(x):
    """Nearest E4M3 value of FP64 x (ties to even), saturating at 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -200))).clamp(min=-6)
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=x.device), e - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    state = prepare(case, seed)
    two = torch.tensor(2.0, dtype=torch.float64, device="cuda")
    if case["op"] == "rope":
        return _exact_rotate(state["x"], state["pos"], state["table"], case["rot"],
                             case["layout"], -1.0 if case["inverse"] else 1.0)
    cu, lens = state["cu"].tolist(), state["kv_lens"].tolist()
    page, d, hkv = case["page"], case["head_dim"], case["kv_heads"]
    table = state["block_table"].tolist()
    if case["op"] == "append":
        pos = torch.cat([torch.arange(lens[b] - (cu[b + 1] - cu[b]), lens[b], device="cuda")
                         for b in range(case["seqs"])])
        kn, vn, q = state["kn"].double(), state["vn"].double(), state["q"].double()
        if case["rot"]:
            kn = _exact_rotate(kn, pos, state["table"], case["rot"], case["layout"])
            q = _exact_rotate(q, pos, state["table"], case["rot"], case["layout"])
        if sum(-(-(cu[b + 1] - cu[b]) // BLOCK) + 1 for b in range(case["seqs"])) > 4000:
            return None
        k = state["k"].double().view(-1, hkv, page // BLOCK, BLOCK, d)
        v = state["v"].double().transpose(-1, -2).contiguous()
        ks = torch.pow(two, state["k_scale"].double() - 127)
        vs = torch.pow(two, state["v_scale"].double() - 127)
        for b in range(case["seqs"]):
            start = lens[b] - (cu[b + 1] - cu[b])
            for blk in range(start // BLOCK, (lens[b] - 1) // BLOCK + 1):
                lo, hi = max(start, blk * BLOCK), min(lens[b], (blk + 1) * BLOCK)
                p, s, kept = table[b][blk * BLOCK // page], blk % (page // BLOCK), lo - blk * BLOCK
                for pool, scale, x in ((k, ks, kn), (v, vs, vn)):
                    fresh = x[cu[b] + lo - start:cu[b] + hi - start].transpose(0, 1)
                    top = fresh.abs().amax(dim=(1, 2)) / 448.0
                    top = torch.pow(two, torch.ceil(torch.log2(top.clamp(min=2.0 ** -126))))
                    if kept:
                        top = torch.maximum(top, scale[p, :, s])
                        held = pool[p, :, s, :kept] * scale[p, :, s, None, None]
                        pool[p, :, s, :kept] = _e4m3(held / top[:, None, None])
                    pool[p, :, s, kept:kept + hi - lo] = _e4m3(fresh / top[:, None, None])
                    scale[p, :, s] = top
        out = [k.view(-1, hkv, page, d), v.transpose(-1, -2).contiguous(), ks, vs]
        return out + [q] if case["rot"] else out
    g = case["q_heads"] // hkv
    outs, sums = [], []
    for b in range(case["seqs"]):
        n, t = cu[b + 1] - cu[b], lens[b]
        pg = state["block_table"][b, :-(-t // page)].long()
        k = state["k"][pg].double() * torch.pow(two, state["k_scale"][pg].double() - 127) \
            .repeat_interleave(BLOCK, -1)[..., None]
        v = state["v"][pg].double() * torch.pow(two, state["v_scale"][pg].double() - 127)[..., None, None]
        k = k.transpose(0, 1).reshape(hkv, -1, d)[:, :t]
        v = v.permute(1, 0, 2, 4, 3).reshape(hkv, -1, d)[:, :t]
        pos = torch.arange(t - n, t, device="cuda")[:, None]
        j = torch.arange(t, device="cuda")
        hide = (j > pos) if case["causal"] else torch.zeros(n, t, dtype=torch.bool, device="cuda")
        if case["window"]:
            hide = hide | (j <= pos - case["window"])
        q = state["q"][cu[b]:cu[b + 1]].double()
        o = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
        for h in range(case["q_heads"]):
            s = (q[:, h] @ k[h // g].t()) / math.sqrt(d)
            s[hide] = -math.inf
            lse[:, h] = torch.logsumexp(s, -1)
            o[:, h] = torch.exp(s - lse[:, h, None]) @ v[h // g]
        outs.append(o)
        sums.append(lse)
    return [torch.cat(outs), torch.cat(sums)]
