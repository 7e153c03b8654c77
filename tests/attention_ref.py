"""Plain references of the attention operators, on the CPU: the rotation in
FP32 with every product and sum rounded by itself (the operators' stated
arithmetic, so results are compared bit for bit), E4M3 coding by search in
the table of its values, and attention in FP64 with its error bounds."""

import math

import numpy as np
import torch

BLOCK = 16
NAN_CODE = 0x7F


def e4m3_values():
    """The 256 codes' values (NaN for 0x7f and 0xff)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


VALUES = e4m3_values()
_POS = VALUES[:127]                       # 0 .. 448, ascending
_MID = (_POS[1:] + _POS[:-1]) / 2


def encode(x):
    """Codes of float64 x: nearest, ties to the even code, saturated; NaN 0x7f."""
    a = np.abs(x)
    i = np.searchsorted(_MID, a, side="left")     # a <= mid: lower code
    tie = (i < len(_MID)) & (a == _MID[np.minimum(i, len(_MID) - 1)])
    i = np.where(tie & (i % 2 == 1), i + 1, i)
    code = np.where(np.signbit(x), i | 128, i)
    return np.where(np.isnan(x), NAN_CODE, code).astype(np.uint8)


def scale_byte(amax):
    """Smallest b >= 1 with amax <= 448 * 2^(b - 127)."""
    b = 1
    while amax > 448.0 * 2.0 ** (b - 127):
        b += 1
    return b


def table64(positions, rot, base=10000.0, scaling=None, factor=1.0, original=0.0, low=1.0,
            high=4.0, magnitude=1.0):
    out = np.empty((positions, rot // 2, 2))
    b = base * factor ** (rot / (rot - 2.0)) if scaling == "base" else base
    for i in range(rot // 2):
        f = b ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "bands":
            turns = original * f / (2 * math.pi)
            w = min(1.0, max(0.0, (turns - low) / (high - low)))
            f *= w + (1 - w) / factor
        a = np.arange(positions) * f
        out[:, i, 0], out[:, i, 1] = magnitude * np.cos(a), magnitude * np.sin(a)
    return out


def rotate32(x, table, pos, layout, inverse=False):
    """x float32 [tokens, heads, d], table float32, pos ints (outside the
    table: NaN).  Returns float32."""
    x = x.astype(np.float32)
    y = x.copy()
    half = table.shape[1]
    for t, p in enumerate(pos):
        inside = 0 <= p < table.shape[0]
        c = table[p, :, 0] if inside else np.full(half, np.nan, np.float32)
        s = table[p, :, 1] if inside else np.full(half, np.nan, np.float32)
        s = -s if inverse else s
        i0 = np.arange(half) if layout == "half" else 2 * np.arange(half)
        i1 = i0 + half if layout == "half" else i0 + 1
        a, b = x[t][:, i0], x[t][:, i1]
        y[t][:, i0] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
        y[t][:, i1] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return y


class Cache:
    """A cache on the host: codes and bytes as numpy arrays."""

    def __init__(self, pages, heads, page, dim, rng=None):
        blocks = page // BLOCK
        shape_k, shape_v = (pages, heads, page, dim), (pages, heads, blocks, dim, BLOCK)
        if rng is None:
            self.k, self.v = np.zeros(shape_k, np.uint8), np.zeros(shape_v, np.uint8)
            self.ks = np.zeros((pages, heads, blocks), np.uint8)
            self.vs = self.ks.copy()
        else:      # whatever an earlier user of the pages left, NaN codes among it
            self.k = rng.integers(0, 256, shape_k, dtype=np.uint8)
            self.v = rng.integers(0, 256, shape_v, dtype=np.uint8)
            self.ks = rng.integers(0, 256, (pages, heads, blocks), dtype=np.uint8)
            self.vs = rng.integers(0, 256, (pages, heads, blocks), dtype=np.uint8)
        self.pages, self.heads, self.page, self.dim = pages, heads, page, dim

    def parts(self, page, head, block):
        """Views of one block: K codes [16, d], V codes [16, d] and setters."""
        return self.k[page, head, block * BLOCK:(block + 1) * BLOCK], self.v[page, head, block].T

    def to(self, w8, pad_pages=False):
        """Device copy; pad_pages: pages further apart than their size."""
        def dev(x):
            t = torch.from_numpy(x.copy()).cuda()
            if pad_pages:
                big = torch.full((t.shape[0], 2) + tuple(t.shape[1:]), 0xAB, dtype=torch.uint8,
                                 device="cuda")
                big[:, 1] = t
                return big[:, 1]
            return t
        return w8.KVCache(dev(self.k), dev(self.v), dev(self.ks), dev(self.vs))

    def append(self, x, is_v, head, table_row, start, stop, values):
        """Store float32 values [stop - start, d] at positions start..stop-1
        of one sequence (pages: table_row)."""
        for blk in range(start // BLOCK, (stop + BLOCK - 1) // BLOCK):
            lo, hi = max(start, blk * BLOCK), min(stop, (blk + 1) * BLOCK)
            if lo >= hi:
                continue
            col = blk * BLOCK // self.page
            if col >= len(table_row) or not 0 <= table_row[col] < self.pages:
                continue
            pg, b = table_row[col], blk % (self.page // BLOCK)
            kc, vc = self.parts(pg, head, b)
            codes = vc if is_v else kc
            scales = self.vs if is_v else self.ks
            new = values[lo - start:hi - start].astype(np.float64)
            fin = np.abs(new[np.isfinite(new)])
            byte, s0 = scale_byte(fin.max() if fin.size else 0.0), lo - blk * BLOCK
            if s0 > 0:
                old = int(scales[pg, head, b])
                byte = max(byte, old)
                if byte > old:
                    codes[:s0] = encode(VALUES[codes[:s0]] * 2.0 ** (old - byte))
            codes[s0:s0 + hi - lo] = encode(new * 2.0 ** (127 - byte))
            scales[pg, head, b] = byte

    def read(self, head, table_row, length):
        """float64 K and V [length, d] of one sequence."""
        k, v = np.empty((length, self.dim)), np.empty((length, self.dim))
        for p in range(length):
            pg, b = table_row[p // self.page], p % self.page // BLOCK
            kc, vc = self.parts(pg, head, b)
            ks, vs = int(self.ks[pg, head, b]), int(self.vs[pg, head, b])
            k[p] = VALUES[kc[p % BLOCK]] * (2.0 ** (ks - 127) if 0 < ks < 255 else np.nan)
            v[p] = VALUES[vc[p % BLOCK]] * (2.0 ** (vs - 127) if 0 < vs < 255 else np.nan)
        return k, v


def attention64(q, cache, table, lens, new, group, scale, causal, window):
    """FP64 attention of q float64 [tokens, q_heads, d].  Returns out, lse,
    and the bounds of their FP32/FP16 arithmetic's error.

    With D channels and FP32 sums, a score is off by at most
    (D + 4) 2^-24 sum|q k| scale =: e (products of 8- or 11-bit queries with
    4-bit codes are exact), so a weight is off by a factor 1 + 2 e, and by
    2^-20 for the exponential; rounding to FP16 adds 2^-11, or 2^-25 of the
    largest weight below FP16's normal range; FP32 sums over N keys add
    N 2^-24.  All of it multiplies sum p |v|."""
    out = np.zeros(q.shape)
    lse = np.full(q.shape[:2], -np.inf)
    tol_o, tol_l = np.zeros(q.shape), np.zeros(q.shape[:2])
    first, d = 0, q.shape[2]
    for b, (n, t) in enumerate(zip(new, lens)):
        for h in range(cache.heads):
            k, v = cache.read(h, table[b], t)
            for i in range(n):
                p = t - n + i
                if p < 0:
                    continue
                hi = min(t, p + 1) if causal else t
                lo = max(0, p - window + 1) if window else 0
                kk, vv = k[lo:hi], v[lo:hi]
                for g in range(group):
                    qq = q[first + i, h * group + g]
                    s = kk @ qq * scale
                    e = float(np.max(np.abs(kk) @ np.abs(qq))) * scale * (d + 4) * 2.0 ** -24
                    m = s.max()
                    w = np.exp(s - m)
                    l = w.sum()
                    out[first + i, h * group + g] = w @ vv / l
                    lse[first + i, h * group + g] = m + math.log(l)
                    rel = 4 * e + 2.0 ** -20 + 2.0 ** -11 + 2 * (hi - lo) * 2.0 ** -24
                    tol_o[first + i, h * group + g] = rel * (w @ np.abs(vv)) / l + \
                        2.0 ** -25 * np.abs(vv).sum(0) / l
                    tol_l[first + i, h * group + g] = 2 * e + 2.0 ** -19 + (hi - lo) * 2.0 ** -24 + \
                        2.0 ** -21 * abs(m)
        first += n
    return out, lse, tol_o, tol_l
