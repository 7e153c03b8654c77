"""Timing cases of: matrix products with an epilogue (bias, activation, gate,
residual), rotary positions of several axes (alone and while appending to the
paged FP8 cache), attention with a window and sinks, and attention of a batch
over a prefix that all of its sequences share.

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
        # a decode step's output projection with the residual added: latency
        dict(name="gemm_decode_residual", op="gemm", m=8, n=4096, k=4096, bias=None, act=None,
             gate=False, residual="bf16", out="bf16", pitch=0),
        # the gate half of a gated MLP, 16 tokens: silu(x Wg) * up
        dict(name="gemm_gated_16", op="gemm", m=16, n=12288, k=5120, bias=None, act="silu",
             gate=True, residual=None, out="bf16", pitch=0),
        # a chunk of a prompt through an MLP with biases, rows out of wider
        # ones, into an FP32 residual stream
        dict(name="gemm_chunk_gelu", op="gemm", m=123, n=8190, k=8192, bias="fp32", act="gelu_tanh",
             gate=False, residual="fp32", out="fp32", pitch=8448),
        # one decode step of a serving batch of multimodal conversations
        dict(name="append3_decode_64", op="append", dtype="bf16", seqs=64, new=1, ragged=True,
             past=4095, q_heads=32, kv_heads=8, head_dim=128, page=64, sections="16,24,24",
             order="split", layout="half"),
        # prompts with images joining a batch, some inside a block
        dict(name="append3_prefill", op="append", dtype="bf16", seqs=6, new=4099, ragged=True,
             past=777, q_heads=32, kv_heads=8, head_dim=128, page=64, sections="24,20,20",
             order="turns", layout="half"),
        # gradient of a vision tower's rotation by row and column
        dict(name="rope2_grad_vision", op="rope", dtype="fp16", tokens=4097, heads=16, head_dim=80,
             sections="20,20", order="own", layout="half", inverse=True, pitch=0),
        # decode step of a serving batch with mixed lengths: a window and sinks
        dict(name="sinks_decode_32", op="attend", dtype="bf16", seqs=32, new=1, ragged=True,
             past=8191, q_heads=32, kv_heads=8, head_dim=128, page=64, window=1024, sinks=4,
             shared=0, causal=True),
        # drafts of one long stream each, small pages, odd lengths
        dict(name="sinks_draft_12", op="attend", dtype="fp16", seqs=12, new=5, ragged=True,
             past=20011, q_heads=40, kv_heads=8, head_dim=64, page=16, window=509, sinks=67,
             shared=0, causal=True),
        # chunks of long prompts
        dict(name="sinks_prefill", op="attend", dtype="bf16", seqs=2, new=1501, ragged=False,
             past=4000, q_heads=32, kv_heads=8, head_dim=128, page=64, window=1024, sinks=4,
             shared=0, causal=True),
        # a few conversations under one system prompt
        dict(name="shared_decode_6", op="attend", dtype="bf16", seqs=6, new=1, ragged=True,
             past=333, q_heads=32, kv_heads=8, head_dim=128, page=64, window=0, sinks=0,
             shared=1984, causal=True),
        # a serving batch under one long document
        dict(name="shared_decode_64", op="attend", dtype="bf16", seqs=64, new=1, ragged=True,
             past=511, q_heads=32, kv_heads=8, head_dim=128, page=64, window=0, sinks=0,
             shared=8192, causal=True),
        # candidates of one context, four drafted tokens each
        dict(name="shared_draft_24", op="attend", dtype="fp16", seqs=24, new=4, ragged=False,
             past=101, q_heads=64, kv_heads=8, head_dim=128, page=32, window=0, sinks=0,
             shared=30016, causal=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sections(rng, pairs):
    """Pairs of two to four axes, and how they take turns."""
    count = rng.choice([2, 3, 3, 4])
    order = rng.choice(["split", "split", "turns", "own"])
    if order == "own":
        return "%d,%d" % (pairs // 2, pairs - pairs // 2), order
    rest = [max(1, pairs // (count + rng.randint(0, 1))) for _ in range(count - 1)]
    if order == "split":
        rest = [max(1, r - rng.randint(0, r // 3)) for r in rest]
    # in turns, axis a needs the pairs a, a + count, ... to exist
    rest = [min(r, (pairs - 1 - a - 1) // count + 1) for a, r in enumerate(rest)]
    return ",".join(map(str, [pairs - sum(rest)] + rest)), order


def _pairs(case):
    """Pairs of each axis."""
    return tuple(map(int, case["sections"].split(",")))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "rope", "append", "attend", "attend", "attend", "attend"])
    if op == "gemm":
        m, n, k = _log_int(rng, 1, 512), _log_int(rng, 100, 12288), 128 * _log_int(rng, 2, 64)
        while m * n * k > 123 * 8190 * 8192:
            m = (m + 1) // 2
        gate = rng.random() < 0.4
        return dict(op=op, m=m, n=n, k=k, bias=rng.choice([None, "bf16", "fp32"]),
                    act=rng.choice([None, "relu", "silu", "gelu", "gelu_tanh"]), gate=gate,
                    residual=rng.choice([None, "bf16", "fp32"]), out=rng.choice(["bf16", "bf16", "fp32"]),
                    pitch=rng.choice([0, 0, k + 8 * rng.randint(1, 64)]))
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    head_dim = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
    group = rng.choice([1, 2, 4, 4, 5, 8])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    layout = rng.choice(["half", "interleaved"])
    if op in ("rope", "append"):
        sections, order = _sections(rng, rng.choice([head_dim, head_dim, head_dim // 2]) // 2)
    if op == "rope":
        heads = kv_heads * group
        tokens = min(_log_int(rng, 1, 16000), 48000000 // (heads * head_dim))
        return dict(op=op, dtype=rng.choice([dtype, "fp32"]), tokens=tokens, heads=heads,
                    head_dim=head_dim, sections=sections, order=order, layout=layout,
                    inverse=rng.random() < 0.4,
                    pitch=rng.choice([0, 0, heads * head_dim + 16 * rng.randint(1, 64)]))
    if op == "append":
        seqs = _log_int(rng, 1, 256)
        new = rng.choice([1, 1, _log_int(rng, 2, 4000)])
        new = max(1, min(new, 24000 // seqs, 90000000 // (kv_heads * (group + 3) * head_dim * seqs)))
        return dict(op=op, dtype=dtype, seqs=seqs, new=new, ragged=rng.random() < 0.7,
                    past=_log_int(rng, 1, 4095), q_heads=kv_heads * group, kv_heads=kv_heads,
                    head_dim=head_dim, page=page, sections=sections, order=order, layout=layout)
    window = sinks = shared = 0
    kind = rng.choice(["decode", "decode", "draft", "prefill"])
    if rng.random() < 0.5:
        window, sinks = _log_int(rng, 16, 4000), _log_int(rng, 1, 200)
        if kind == "decode":
            seqs, new, past = _log_int(rng, 1, 128), 1, _log_int(rng, 1, 20000)
        elif kind == "draft":
            seqs, new, past = _log_int(rng, 1, 48), rng.randint(2, 9), _log_int(rng, 1, 20000)
        else:
            seqs, new, past = rng.randint(1, 3), _log_int(rng, 17, 1500), _log_int(rng, 1, 6000)
    else:
        shared = page * max(1, _log_int(rng, 64, 30000) // page)
        if kind == "decode":
            seqs, new, past = _log_int(rng, 2, 128), 1, _log_int(rng, 1, 2000)
        elif kind == "draft":
            seqs, new, past = _log_int(rng, 2, 48), rng.randint(2, 9), _log_int(rng, 1, 1000)
        else:
            seqs, new, past = _log_int(rng, 2, 16), _log_int(rng, 10, 300), _log_int(rng, 1, 300)
    heads = kv_heads * group
    case = dict(op=op, dtype=dtype, seqs=seqs, new=new, ragged=rng.random() < 0.7, past=past,
                q_heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page, window=window,
                sinks=sinks, shared=shared, causal=rng.random() < 0.9)
    # at most the largest listed cases' products and held keys
    while case["seqs"] > 1 and case["seqs"] * (case["past"] + new + shared) * kv_heads * head_dim > \
            32 * 33000 * 1024:
        case["seqs"] //= 2
    while case["seqs"] * case["new"] * (case["past"] + case["new"] + shared) * heads * head_dim > \
            24 * 4 * 30121 * 64 * 128 and case["seqs"] * case["new"] > 1:
        if case["new"] > 1:
            case["new"] //= 2
        else:
            case["seqs"] //= 2
    return case


def _lengths(case):
    """(new tokens, tokens held with them) of each sequence, as lists."""
    new, total = [], []
    for b in range(case["seqs"]):
        f = 1.0 - 0.75 * ((0.6180339887 * b) % 1.0) if case["ragged"] else 1.0
        g = 1.0 - 0.5 * ((0.4142135624 * b) % 1.0) if case["ragged"] else 1.0
        n = max(1, int(round(case["new"] * g)))
        new.append(n)
        total.append(case.get("shared", 0) + n + int(round(case["past"] * f)))
    return new, total


def _visible(case):
    """(query, key) pairs that see each other, and keys to be read (those of
    the shared prefix once)."""
    pairs = keys = 0
    window, sinks, shared = case["window"], case["sinks"], case["shared"]
    for n, t in zip(*_lengths(case)):
        first = t
        for p in range(t - n, t):
            hi = p + 1 if case["causal"] else t
            lo = max(0, p - window + 1) if window else 0
            pairs += hi - lo + min(lo, sinks)
            first = min(first, lo)
        keys += t - first + min(first, sinks) - shared
    return pairs, keys + shared


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        by = 2 * m * k + n * k + 4 * -(-n // 128) * (k // 128) + m * n * size[case["out"]]
        by += n * size[case["bias"]] if case["bias"] else 0
        by += 2 * m * n if case["gate"] else 0
        by += m * n * size[case["residual"]] if case["residual"] else 0
        return {"bytes": by, "flops": 2 * m * n * k}
    d, el = case["head_dim"], size[case["dtype"]]
    if case["op"] == "attend":
        new, total = _lengths(case)
        tokens, kvd = sum(new), case["kv_heads"] * d
        pairs, keys = _visible(case)
        by = keys * (2 * kvd + 2 * case["kv_heads"] / BLOCK)
        by += tokens * case["q_heads"] * (2 * d * el + 4) + 4 * sum(-(-t // case["page"]) for t in total)
        return {"bytes": by, "flops": 4 * d * case["q_heads"] * pairs}
    rot, axes = 2 * sum(_pairs(case)), len(_pairs(case))
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * d
        return {"bytes": 2 * n * el + case["tokens"] * (rot * 4 + 4 * axes),
                "flops": 3 * case["tokens"] * case["heads"] * rot}
    tokens, kvd = sum(_lengths(case)[0]), case["kv_heads"] * d
    by = tokens * (2 * kvd * el + 2 * kvd + rot * 4 + 4 * axes)      # k, v in; codes out; table
    by += 2 * tokens * case["q_heads"] * d * el
    return {"bytes": by, "flops": tokens * (3 * rot * (case["q_heads"] + case["kv_heads"]) + 4 * kvd)}


# ------------------------------------------------------------------ inputs

def _table(positions, rot, base=500000.0):
    """[positions, rot / 2, 2] FP32 cosines and sines."""
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack((a.cos(), a.sin()), dim=-1).float()


def _axes_table(case, positions):
    s = _pairs(case)
    return _table(positions, 2 * (max(s) if case["order"] == "own" else sum(s)))


def _axes_positions(case, pos, start):
    """int32 [axes, tokens] of tokens at places `pos` of pictures in rows of
    41 patches: the frame, the row, the column, and the place again."""
    rows = [pos // 1681 + start, pos // 41 % 41 + start, pos % 41 + start, pos + start]
    axes = len(_pairs(case))
    return torch.stack(rows[1:3] if axes == 2 else rows[:axes]).to(torch.int32)


def _codes(x):
    """E4M3 codes and E8M0 bytes of blocks x [..., 16, head_dim]."""
    amax = x.abs().amax(dim=(-1, -2))
    byte = (((amax.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=1)
    code = (x * _power(254 - byte)[..., None, None]).to(torch.float8_e4m3fn)
    return code, byte.to(torch.uint8)


def _power(field):
    """2^(field - 127) in FP32 of exponent fields 1..254 (0 below them)."""
    return (field.int().clamp(min=0) << 23).view(torch.float32)


def _prepare_gemm(case, randn):
    m, n, k = case["m"], case["n"], case["k"]
    state = dict(case=case)
    pitch = case["pitch"] or k
    state["a"] = randn(m, pitch).to(torch.bfloat16)[:, :k]
    rows = -(-n // 128) * 128
    w = randn(rows, k) * (1.0 + randn(rows, 1).abs()) * k ** -0.5
    blocks = w.view(rows // 128, 128, k // 128, 128)
    s = blocks.abs().amax((1, 3)) / 448.0
    codes = (blocks / s[:, None, :, None]).view(rows, k)[:n].to(torch.float8_e4m3fn)
    state["w"], state["scale"] = codes.contiguous(), s
    state["bias"] = randn(n).to(_DTYPES[case["bias"]]) if case["bias"] else None
    state["gate"] = randn(m, n).to(torch.bfloat16) if case["gate"] else None
    state["residual"] = (2.0 * randn(m, n)).to(_DTYPES[case["residual"]]) if case["residual"] else None
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] == "gemm":
        return _prepare_gemm(case, randn)
    dtype, d = _DTYPES[case["dtype"]], case["head_dim"]
    start = int(torch.randint(0, 1000, (1,), generator=gen, device="cuda"))
    if case["op"] == "rope":
        t, h = case["tokens"], case["heads"]
        pitch = case["pitch"] or h * d
        x = randn(t, pitch).to(dtype)[:, :h * d].unflatten(1, (h, d))
        pos = _axes_positions(case, torch.arange(t, device="cuda"), start)
        return dict(case=case, x=x, pos=pos, table=_axes_table(case, t + 1041))

    new, total = _lengths(case)
    order = torch.randperm(case["seqs"], generator=gen, device="cuda").tolist()
    new, total = [new[i] for i in order], [total[i] for i in order]
    seqs, hq, hkv, page = case["seqs"], case["q_heads"], case["kv_heads"], case["page"]
    common = case.get("shared", 0) // page          # pages that all sequences hold
    need = [-(-t // page) - common for t in total]
    width = max(need)
    pages = common + sum(need) + max(4, sum(need) // 16)
    perm = torch.randperm(pages, generator=gen, device="cuda")
    used = torch.tensor(need, device="cuda")
    first = common + used.cumsum(0) - used
    col = torch.arange(width, device="cuda")
    at = (first[:, None] + col).clamp(max=pages - 1)
    table = torch.where(col < used[:, None], perm[at], torch.zeros_like(at))
    table = torch.cat((perm[:common].expand(seqs, common), table), 1).to(torch.int32)
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
    cu = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    cu[1:] = torch.tensor(new, dtype=torch.int32, device="cuda").cumsum(0)
    state["cu"] = cu
    state["uniform"] = min(new) == max(new)
    tokens = sum(new)
    if case["op"] == "attend":
        state["q"] = (randn(tokens, hq, d) * 0.6).to(dtype)
        return state
    # one fused row per token, as the projections leave it
    qkv = randn(tokens, (hq + 2 * hkv) * d).to(dtype)
    state["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
    state["kn"] = (qkv[:, hq * d:(hq + hkv) * d]).unflatten(1, (hkv, d))
    state["vn"] = (qkv[:, (hq + hkv) * d:]).unflatten(1, (hkv, d))
    _, pos = _places(state, tokens)
    state["pos"] = _axes_positions(case, pos, start)
    state["table"] = _axes_table(case, max(total) + 1041)
    return state


# -------------------------------------------------------------- plain form

def _plain_gemm(state):
    case = state["case"]
    n, k = state["w"].shape
    w = state["w"].float().view(n, k // 128, 128)
    w = (w * state["scale"].repeat_interleave(128, 0)[:n, :, None]).view(n, k)
    y = state["a"].float() @ w.t()
    if case["bias"]:
        y = y + state["bias"].float()
    if case["act"] == "relu":
        y = y.clamp(min=0.0)
    elif case["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    elif case["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    elif case["act"] == "gelu_tanh":
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    if case["gate"]:
        y = y * state["gate"].float()
    if case["residual"]:
        y = y + state["residual"].float()
    return y.to(_DTYPES[case["out"]])


def _pair_axes(case):
    """The axis and the table's column of every pair."""
    s, order = _pairs(case), case["order"]
    if order == "turns":
        n = len(s)
        axis = [i % n if i % n and i < n * s[i % n] else 0 for i in range(sum(s))]
        return axis, list(range(sum(s)))
    axis = [a for a, c in enumerate(s) for _ in range(c)]
    if order == "own":
        return axis, [i for c in s for i in range(c)]
    return axis, list(range(sum(s)))


def _angles(case, table, pos):
    """[tokens, pairs, 2] of positions [axes, tokens]."""
    axis, col = _pair_axes(case)
    axis = torch.tensor(axis, device="cuda")
    return table[pos.long()[axis].t(), torch.tensor(col, device="cuda")]


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
    page, rot = case["page"], 2 * sum(_pairs(case))
    kn, vn, q = state["kn"].float(), state["vn"].float(), state["q"]
    tokens, hkv, d = kn.shape
    cs = _angles(case, state["table"], state["pos"])
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
    return [state["k"], state["v"], _scale_values(state["k_scale"]), _scale_values(state["v_scale"]), q]


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
    see = (j < lens[:, None, None]).expand(seqs, nq, s_len)
    if case["causal"]:
        see = see & (j <= pos[..., None])
    if case["window"]:
        see = see & ((j > pos[..., None] - case["window"]) | (j < case["sinks"]))
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
    if case["op"] == "gemm":
        return _plain_gemm(state)
    if case["op"] == "rope":
        x = state["x"]
        cs = _angles(case, state["table"], state["pos"])
        return _rotate(x.float(), cs, 2 * sum(_pairs(case)), case["layout"], case["inverse"]).to(x.dtype)
    return _plain_append(state) if case["op"] == "append" else _plain_attend(state)


# --------------------------------------------------------------------- run

def run(state):
    if not own:
        return _plain(state)
    import block_scaled_fp8_w8a16_amd as w8
    case = state["case"]
    if case["op"] == "gemm":
        return w8.gemm_epilogue(state["a"], state["w"], state["scale"], bias=state["bias"],
                                activation=case["act"], gate=state["gate"],
                                residual=state["residual"], out_dtype=_DTYPES[case["out"]])
    if case["op"] == "rope":
        return w8.rope(state["x"], state["table"], state["pos"], layout=case["layout"],
                       inverse=case["inverse"], sections=_pairs(case), order=case["order"])
    cache = w8.KVCache(state["k"], state["v"], state["k_scale"], state["v_scale"])
    cu = None if state["uniform"] else state["cu"]
    if case["op"] == "append":
        q = w8.kv_append(cache, state["kn"], state["vn"], state["block_table"], state["kv_lens"],
                         cu_seqlens=cu, max_new=state["max_new"], table=state["table"],
                         layout=case["layout"], q=state["q"], positions=state["pos"],
                         sections=_pairs(case), order=case["order"])
        return [state["k"], state["v"], _scale_values(state["k_scale"]),
                _scale_values(state["v_scale"]), q]
    out, lse = w8.kv_attention(state["q"], cache, state["block_table"], state["kv_lens"],
                               cu_seqlens=cu, max_new=state["max_new"], max_kv=state["max_kv"],
                               causal=case["causal"], window=case["window"], sinks=case["sinks"],
                               shared=case["shared"], return_lse=True)
    return [out, lse]


# ----------------------------------------------------------- 64-bit values

def _exact_rotate(x, pos, table, case, sign=1.0):
    """Rotation as a product of complex numbers, FP64, axis by axis."""
    y = x.double().clone()
    axes, cols = _pair_axes(case)
    half = len(axes)
    for i, (a, c) in enumerate(zip(axes, cols)):
        z = torch.view_as_complex(table[pos[a].long(), c].double().contiguous())[:, None]
        z = z if sign > 0 else z.conj()
        i0, i1 = (i, i + half) if case["layout"] == "half" else (2 * i, 2 * i + 1)
        w = torch.complex(y[..., i0].clone(), y[..., i1].clone()) * z
        y[..., i0], y[..., i1] = w.real, w.imag
    return y


def _e4m3(x):
    """Nearest E4M3 value of FP64 x (ties to even), saturating at 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -200))).clamp(min=-6)
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=x.device), e - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_gemm(state):
    case = state["case"]
    a, codes, scale = state["a"].double(), state["w"], state["scale"].double()
    n, k = codes.shape
    y = torch.zeros(a.shape[0], n, dtype=torch.float64, device="cuda")
    for r in range(0, n, 128):
        rows = codes[r:r + 128].double()
        y[:, r:r + 128] = a @ (rows * scale[r // 128].repeat_interleave(128)).t().contiguous()
    if case["bias"]:
        y += state["bias"].double()
    act = case["act"]
    if act == "relu":
        y = torch.where(y > 0, y, torch.zeros_like(y))
    elif act == "silu":
        y = y * torch.special.expit(y)
    elif act == "gelu":
        y = y * 0.5 * torch.special.erfc(-y / math.sqrt(2.0))
    elif act == "gelu_tanh":
        y = y * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3))
    if case["gate"]:
        y = y * state["gate"].double()
    return y + state["residual"].double() if case["residual"] else y


def exact(case, seed):
    state = prepare(case, seed)
    two = torch.tensor(2.0, dtype=torch.float64, device="cuda")
    if case["op"] == "gemm":
        return _exact_gemm(state)
    if case["op"] == "rope":
        return _exact_rotate(state["x"], state["pos"], state["table"], case,
                             -1.0 if case["inverse"] else 1.0)
    cu, lens = state["cu"].tolist(), state["kv_lens"].tolist()
    page, d, hkv = case["page"], case["head_dim"], case["kv_heads"]
    table = state["block_table"].tolist()
    if case["op"] == "append":
        if sum(-(-(cu[b + 1] - cu[b]) // BLOCK) + 1 for b in range(case["seqs"])) > 4000:
            return None
        kn, vn, q = state["kn"], state["vn"].double(), state["q"]
        kn = _exact_rotate(kn, state["pos"], state["table"], case)
        q = _exact_rotate(q, state["pos"], state["table"], case)
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
        return [k.view(-1, hkv, page, d), v.transpose(-1, -2).contiguous(), ks, vs, q]
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
            hide = hide | ((j <= pos - case["window"]) & (j >= case["sinks"]))
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
