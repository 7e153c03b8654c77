"""The W8A16 product with bias, activation, gate and residual.

Operands are chosen so that the product's FP32 sum is exact in any order
(small whole A, a few-bit weights, power-of-two scales); what the epilogue
makes of it is compared with FP64, within the FP32 roundings counted in
``expected``."""

import ctypes
import math

import numpy as np
import pytest

import block_scaled_fp8_w8a16_amd as w8mod

torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def w8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w8mod.library()
    return w8mod


# ---------------------------------------------------------------- CPU side

def raw(m=1, n=16, k=128, ars=128, crs=16, a=16, w=16, s=16, c=16, null=False, **kw):
    e = w8mod.Epilogue(**dict(dict(out_dtype=1), **kw))
    return w8mod.library().w8a16_gemm_epilogue(a, ars, w, s, c, crs, m, n, k, None if null else e, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(m=0), w8mod.ERR_M_ZERO), (dict(k=100), w8mod.ERR_K_NOT_MULT_128),
    (dict(crs=15), w8mod.ERR_PITCH_TOO_SHORT), (dict(ars=132), w8mod.ERR_A_STRIDE_ALIGN),
    (dict(n=0), w8mod.ERR_N_ZERO), (dict(a=0), w8mod.ERR_NULL_PTR), (dict(c=0), w8mod.ERR_NULL_PTR),
    (dict(null=True), w8mod.ERR_NULL_PTR), (dict(activation=5), w8mod.ERR_SHAPE),
    (dict(out_dtype=0), w8mod.ERR_SHAPE), (dict(out_dtype=2), w8mod.ERR_SHAPE),
    (dict(bias=16, bias_dtype=2), w8mod.ERR_SHAPE), (dict(bias=16), w8mod.ERR_SHAPE),
    (dict(residual=16, residual_dtype=2, residual_row_stride=16), w8mod.ERR_SHAPE),
    (dict(residual=16, residual_dtype=1, residual_row_stride=15), w8mod.ERR_PITCH_TOO_SHORT),
    (dict(gate=16, gate_row_stride=15), w8mod.ERR_PITCH_TOO_SHORT)])
def test_refusals(kw, want):
    assert raw(**kw) == want
    assert w8mod.last_error().startswith("w8a16_gemm_epilogue: ")


def test_python_side_refusals():
    t = torch.zeros
    a, w, s = t(2, 128, dtype=BF16), t(8, 128, dtype=torch.uint8), t(1, 1)
    for kw in (dict(activation="swish"), dict()):                   # the last: no GPU tensors
        with pytest.raises(ValueError):
            w8mod.gemm_epilogue(a, w, s, **kw)
    with pytest.raises(ValueError):
        w8mod.gemm_epilogue(a, w[:, :64], s)


# ---------------------------------------------------------------- GPU side

def operands(m, n, k, seed, pitch=0):
    """a, w, scale on the GPU and the exact sums in FP64."""
    g = torch.Generator().manual_seed(seed)
    a = torch.randint(-2, 3, (m, pitch or k), generator=g).to(BF16).cuda()[:, :k]
    # codes of magnitude below 3.75 (multiples of 2^-9), below 1/2 for long k
    top = 0x48 if k <= 1024 else 0x30
    w = torch.randint(0, top, (n, k), generator=g, dtype=torch.uint8) | \
        (torch.randint(0, 2, (n, k), generator=g, dtype=torch.uint8) << 7)
    w = w.cuda()
    s = torch.randint(0, 2, (-(-n // 128), k // 128), generator=g)
    s = (2.0 ** (s - (5 if k <= 1024 else 4))).float().cuda()
    # the largest sum 2 * 3.75 * 1024 / 16 = 480 < 2^24 units of 2^-9 * 2^-5
    full = w.view(torch.float8_e4m3fn).double() * \
        s.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
    return a, w, s, a.double() @ full.t().contiguous()


def expected(s, bias, act, gate, res, out):
    """FP64 outputs and the bound of the kernel's error.

    y = s + bias is rounded once.  expf is within an ulp (2 U), erfcf within 16
    ulp (32 U); a relative error r of an activation's argument x enters its
    value by at most (1 + |x|) r for SiLU (x sigmoid(x): 1 + |x| (1 -
    sigmoid)), (2 + x^2) r for GELU (its tail falls as e^(-x^2/2)), and for the
    hyperbolic form by 1 + 6 |u|, u its cubic (each factor of u is a rounding: 6
    of them, and 2 |u| the exponent)."""
    y = s if bias is None else s + bias.double()
    e = 0.0 if bias is None else U
    x = y.abs()
    if act == "relu":
        v, rel = y.clamp(min=0.0), e + 0 * x
    elif act == "silu":
        v, rel = y * torch.special.expit(y), (1 + x) * e + 4 * U
    elif act == "gelu":
        v, rel = y * 0.5 * torch.special.erfc(-y / math.sqrt(2)), (2 + x * x) * (e + 2 * U) + 34 * U
    elif act == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)
        v, rel = y * torch.special.expit(2 * u), (1 + 6 * u.abs()) * e + 12 * u.abs() * U + 4 * U
    else:
        v, rel = y, e + 0 * x
    tol = v.abs() * rel + 2.0 ** -126
    if gate is not None:
        v, tol = v * gate.double(), tol * gate.double().abs()
        tol = tol + v.abs() * U
    if res is not None:
        v = v + res.double()
        tol = tol + v.abs() * U
    return v, tol + v.abs() * (2.0 ** -8 if out == BF16 else U) + 2.0 ** -133


def check(got, s, bias, act, gate, res):
    want, tol = expected(s, bias, act, gate, res, got.dtype)
    # U U terms of the products of the bounds above
    bad = ~((got.double() - want).abs() <= tol * (1 + 2.0 ** -10))
    assert not bad.any(), "%d off, first %s: %r, want %r +- %r" % (
        int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item(), tol[bad][0].item())


SHAPES = [(1, 16, 128), (3, 515, 256), (8, 512, 1024), (8, 4096, 512), (16, 1000, 1024), (33, 777, 256),
          (64, 640, 512), (1, 1024, 8192), (5, 256, 8192), (16, 12288, 5120), (8, 12290, 4352),
          (48, 8192, 2176), (72, 8192, 2176), (123, 1030, 8192), (129, 515, 1024), (300, 2050, 512)]
FORMS = [(None, None, None, None, BF16), ("silu", None, BF16, None, BF16), (None, None, None, BF16, BF16),
         ("gelu_tanh", F32, None, F32, F32), ("gelu", BF16, BF16, BF16, F32), ("relu", BF16, BF16, F32, BF16)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_against_fp64(w8, shape, form):
    m, n, k = shape
    act, bt, gt, rt, out = FORMS[form]
    a, w, scale, s = operands(m, n, k, 10 * m + form, pitch=k + 8 * (form % 2))
    g = torch.Generator(device="cuda").manual_seed(form)

    def rows(t, pad):      # rows apart by `pad` more than n: whole pieces of four, or not
        x = torch.randn(m, n + pad, generator=g, device="cuda").to(t)
        return x[:, pad // 2:pad // 2 + n]
    pad = (0, 8 - n % 4, 5)[form % 3]
    bias = torch.randn(n, generator=g, device="cuda").to(bt) if bt else None
    gate = rows(gt, pad) if gt else None
    res = rows(rt, pad) if rt else None
    c = torch.full((m + 1, n + 7), float("nan"), dtype=out, device="cuda")
    got = w8.gemm_epilogue(a, w, scale, c[:m, 3:3 + n], bias=bias, activation=act, gate=gate, residual=res)
    check(got, s, bias, act, gate, res)
    assert c[m].isnan().all() and c[:, :3].isnan().all() and c[:, 3 + n:].isnan().all()
    # a new output, of rows aligned as the allocator does it: the same bits
    new = w8.gemm_epilogue(a, w, scale, bias=bias, activation=act, gate=gate, residual=res, out_dtype=out)
    assert torch.equal(new, got)
    if form == 0:
        assert torch.equal(new, w8.gemm(a, w, scale))


@pytest.mark.gpu
@pytest.mark.parametrize("t", [BF16, F32])
@pytest.mark.parametrize("shape", [(4, 260, 256), (1, 1024, 8192), (129, 515, 1024), (72, 8192, 2176)], ids=str)
def test_residual_in_place(w8, shape, t):
    m, n, k = shape
    a, w, scale, s = operands(m, n, k, 5)
    x = torch.randn(m, n, device="cuda").to(t)
    want = w8.gemm_epilogue(a, w, scale, activation="silu", residual=x, out_dtype=t)
    got = w8.gemm_epilogue(a, w, scale, x, activation="silu", residual=x)
    assert got is x and torch.equal(x, want)


@pytest.mark.gpu
def test_special_values(w8):
    a, w, scale, s = operands(3, 8, 128, 1)
    inf, nan = float("inf"), float("nan")
    bias = torch.tensor([inf, -inf, nan, 0, 0, 0, 0, -300.0], device="cuda")
    gate = torch.ones(3, 8, device="cuda", dtype=BF16)
    gate[:, 3], gate[:, 4] = inf, nan
    res = torch.zeros(3, 8, device="cuda")
    res[:, 5], res[:, 6] = -inf, nan
    y = s + bias.double()
    for act, f in (("relu", lambda v: torch.where(v < 0, 0 * v.abs().clamp(max=1), v)),
                   ("silu", lambda v: v / (1 + (-v).exp()))):
        got = w8.gemm_epilogue(a, w, scale, bias=bias, activation=act, gate=gate, residual=res,
                               out_dtype=F32).double()
        want = f(y) * gate.double() + res.double()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
        fin = want.isfinite()
        assert ((got - want)[fin].abs() <= want[fin].abs() * 16 * U * 400 + 2.0 ** -126).all()


@pytest.mark.gpu
def test_wide_rows_and_far_columns(w8):
    """Strides past 2^31 bytes from the base."""
    m, n, k = 3, 264, 128
    a, w, scale, s = operands(m, n, k, 3)
    pitch = (1 << 30) + 4
    big = torch.empty(2 * pitch + n, dtype=BF16, device="cuda")
    c = big.as_strided((m, n), (pitch, 1))
    c.copy_(torch.randn(m, n, device="cuda"))
    res = c.clone()
    w8.gemm_epilogue(a, w, scale, c, residual=c, gate=res)
    check(c, s, None, None, res, res)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(8, 512, 1024), (1, 1024, 8192), (72, 8192, 2176)], ids=str)
def test_captured_and_on_another_stream(w8, shape):
    m, n, k = shape
    a, w, scale, s = operands(m, n, k, 9)
    x = torch.randn(m, n, device="cuda").to(BF16)
    bias = torch.randn(n, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):       # workspaces grow before the capture
        w8.gemm_epilogue(a, w, scale, bias=bias, activation="gelu", residual=x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        y = w8.gemm_epilogue(a, w, scale, bias=bias, activation="gelu", residual=x)
    for _ in range(3):
        x.copy_(torch.randn(m, n, device="cuda").to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        want = w8.gemm_epilogue(a, w, scale, bias=bias, activation="gelu", residual=x, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.gpu
def test_refusals_of_tensors(w8):
    a, w, scale, _ = operands(2, 24, 128, 1)
    ok = torch.zeros(2, 24, dtype=BF16, device="cuda")
    for kw in (dict(gate=ok.float()), dict(gate=ok[:1]), dict(residual=ok.half()), dict(residual=ok.cpu()),
               dict(bias=ok[0, :23]), dict(bias=ok[0].half()), dict(c=ok.half()), dict(c=ok.t()),
               dict(gate=torch.zeros(2, 48, dtype=BF16, device="cuda")[:, ::2]), dict(out_dtype=torch.float16),
               dict(c=ok, out_dtype=F32)):
        with pytest.raises(ValueError):
            w8.gemm_epilogue(a, w, scale, **kw)
    with pytest.raises(w8.W8A16Error):      # rows of the gate on top of each other
        w8.gemm_epilogue(a, w, scale, gate=ok[:1].expand(2, 24))


@pytest.mark.gpu
def test_rows_too_far_apart_are_refused(w8):
    _, w, scale, _ = operands(2, 24, 128, 1)
    far = torch.empty((1 << 32) + 128, dtype=BF16, device="cuda").as_strided((2, 128), (1 << 32, 1))
    with pytest.raises(ValueError, match="apart"):
        w8.gemm_epilogue(far, w, scale)


@pytest.mark.gpu
def test_two_threads(w8):
    """Threads on streams of their own get what one gets."""
    import threading

    a, w, scale, _ = operands(1, 1024, 8192, 6)      # cut along k: the streams' workspaces
    rows = [a * (i + 1) for i in range(4)]
    want = [w8.gemm_epilogue(x, w, scale, activation="silu") for x in rows]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    torch.cuda.synchronize()

    def work(i):
        for n in range(40):
            got[i].append(w8.gemm_epilogue(rows[(n + i) % 4], w, scale, activation="silu", stream=streams[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 40 and all(torch.equal(y, want[(n + i) % 4]) for n, y in enumerate(got[i]))
