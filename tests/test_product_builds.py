"""The product with an epilogue in every build that a default plan names for a
256-CU GPU, and its activations where they end."""

import math
import random

import pytest

import block_scaled_fp8_w8a16_amd as w8mod
from test_product_epilogue import BF16, F32, U, check, operands, w8  # noqa: F401

torch = pytest.importorskip("torch")

# A small product for each kernel, tile, ring depth, number of waves, flags,
# K splits or none, one row tile or several.
SHAPES = [
    (17, 9, 4096), (2, 9, 4096), (17, 570, 8192), (1, 1137, 8064), (17, 9, 128), (2, 9, 128), (17, 9, 2048),
    (2, 9, 2048), (17, 49, 2048), (2, 113, 2048), (17, 2049, 128), (2, 6114, 128), (33, 1365, 2048),
    (2, 6114, 2048), (17, 4097, 128), (2, 8193, 128), (65, 1647, 2048), (1, 8193, 2048), (33, 4097, 128),
    (1, 12289, 128), (65, 2730, 2048), (1, 12291, 2048), (33, 8223, 128), (81, 1346, 128), (85, 1347, 2048),
    (17, 715, 71168), (17, 1533, 32896), (33, 4082, 128), (17, 6146, 128), (81, 2025, 2048), (17, 6169, 2048),
    (33, 5443, 128), (17, 8194, 128), (97, 2323, 2048), (17, 8247, 2048), (65, 6543, 128), (33, 8193, 2048),
    (65, 3882, 4352), (33, 4374, 3840), (65, 8256, 2048), (33, 16411, 2048), (66, 4154, 4096), (33, 8220, 4096),
    (129, 9, 128), (129, 9, 256), (132, 8217, 2048), (130, 4099, 4096), (65, 16391, 2048), (65, 4152, 8192),
    (8, 775, 65920), (9, 5879, 8576), (8, 5962, 8448), (9, 6145, 65664), (9, 7711, 6528), (8, 7022, 7168),
    (9, 12685, 3968), (8, 12689, 3968), (17, 6051, 8320), (22, 6224, 65920), (17, 6901, 7296),
    (18, 12374, 66304), (17, 12686, 3968)]


def build_of(m, n, k):
    p = w8mod.plan(m, n, k, 256)
    return (p.kernel, p.m_blocks, p.n_blocks, p.depth, p.a_depth, p.waves, p.flags, p.splits > 1, p.m_tiles > 1)


def test_shapes_name_every_build():
    builds = {build_of(*s) for s in SHAPES}
    assert len(builds) == len(SHAPES)
    rng = random.Random(5)

    def log(lo, hi):
        return int(lo * (hi / lo) ** rng.random())
    for _ in range(20000):
        s = log(1, 1100), log(1, 70000), 128 * log(1, rng.choice([130, 1000]))
        assert build_of(*s) in builds, s


def test_default_plans_are_built():
    """With an epilogue the launchers know these variants only."""
    rng = random.Random(6)
    tiles = {(4, 4, 4, 6, 8), (8, 8, 3, 2, 8), (8, 4, 4, 2, 8), (8, 8, 3, 3, 8), (4, 8, 4, 4, 10)}
    for _ in range(20000):
        m, n, k = (int(hi ** rng.random()) for hi in (1100, 70000, 1000))
        p = w8mod.plan(m, n, 128 * k, rng.choice([256, rng.randint(1, 400)]))
        if p.kernel == w8mod.KERNEL_STREAM:
            assert p.depth == 1 and not p.flags & w8mod.FLAG_DIRECT and (p.m_blocks, p.n_blocks) != (2, 8)
        elif p.kernel == w8mod.KERNEL_RING:
            assert p.stage_steps == 4 and p.depth in (2, 3)
        else:
            assert (p.m_blocks, p.n_blocks, p.depth, p.a_depth, p.waves) in tiles


def sums(a, w, scale):
    """A @ dequant(W)^T in FP64, some columns at a time."""
    out = []
    for j in range(0, len(w), 1024):
        full = w[j:j + 1024].view(torch.float8_e4m3fn).double()
        s = scale[j // 128:(j + 1024) // 128].double()
        full *= s.repeat_interleave(128, 0)[:len(full)].repeat_interleave(128, 1)
        out.append(a.double() @ full.t().contiguous())
    return torch.cat(out, 1)


def big_operands(m, n, k, seed):
    """As operands(), made on the GPU.  Codes below 1/2, multiples of 2^-9, and
    scales of 1/16 and 1/8: sums are multiples of 2^-13, exact in FP32 in any
    order while they stay below 2^11, which is 200 standard deviations of a sum
    of 70000 such products."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def ints(lo, hi, *shape, **kw):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", **kw)
    a = ints(-2, 3, m, k).to(BF16)
    w = ints(0, 0x30, n, k, dtype=torch.uint8) | (ints(0, 2, n, k, dtype=torch.uint8) << 7)
    s = (2.0 ** (ints(0, 2, -(-n // 128), k // 128) - 4)).float()
    return a, w, s, sums(a, w, s)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_every_build(w8, shape):
    m, n, k = shape
    a, w, scale, s = operands(m, n, k, m + n) if n * k < 1 << 21 else big_operands(m, n, k, m + n)
    g = torch.Generator(device="cuda").manual_seed(k)

    def rows(t):
        return torch.randn(m, n, generator=g, device="cuda").to(t)
    bias, gate, res = rows(F32)[0].contiguous(), rows(BF16), rows(F32)
    got = w8.gemm_epilogue(a, w, scale, bias=bias, activation="silu", gate=gate, residual=res, out_dtype=F32)
    check(got, s, bias, "silu", gate, res)
    res = rows(BF16)
    c = res.clone()
    w8.gemm_epilogue(a, w, scale, c, bias=bias, residual=c)
    check(c, s, bias, None, None, res)
    assert torch.equal(w8.gemm_epilogue(a, w, scale), w8.gemm(a, w, scale))


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
def test_gelu_of_special_values(w8, act):
    """Infinities, NaN, and arguments so large that a form's parts overflow."""
    n = 16
    a, w, scale, s = operands(3, n, 128, 1)
    inf, nan = float("inf"), float("nan")
    ends = [inf, -inf, nan, 3e38, -3e38, 1e20, -1e20, 300.0, -300.0, 20.0, -20.0, 0.0, -0.0, 1e-30, -1e-30, 0.0]
    bias = torch.tensor(ends, device="cuda")
    gate, res = torch.ones(3, n, device="cuda", dtype=BF16), torch.zeros(3, n, device="cuda")
    gate[:, 11], gate[:, 12], res[:, 13], res[:, 14] = inf, nan, -inf, nan
    y = s + bias.double()
    y = y.float().double()            # (the sum is rounded before the activation)
    if act == "gelu":
        v = 0.5 * y * torch.special.erfc(-y / math.sqrt(2))
    else:
        v = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    want = v * gate.double() + res.double()
    got = w8.gemm_epilogue(a, w, scale, bias=bias, activation=act, gate=gate, residual=res, out_dtype=F32).double()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
    fin = want.isfinite()
    # erfcf within 32 U, its argument rounded twice (2 U x^2 of the tail);
    # each factor of u is a rounding, 6 of them, and 2 |u| the exponent;
    # 1 + tanh(u) is rounded to FP64 by 2^-53 at the most; below FP32's normal
    # range erfcf and expf may give zeros
    x = y[fin].abs().clamp(max=20)
    tol = want[fin].abs() * U * (40 + (2 * x * x if act == "gelu" else 18 * (0.8 * x + 0.036 * x ** 3))) + 2.0 ** -50 * x
    assert ((got - want)[fin].abs() <= tol + 2.0 ** -122).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(40, 2304, 8192), (130, 4099, 4096), (65, 4152, 8192)], ids=str)
def test_captured_sums_of_tile_splits(w8, shape):
    """Two launches through the stream's workspace, replayed with eager calls
    of the same stream in between."""
    m, n, k = shape
    assert w8.plan(m, n, k).kernel == w8.KERNEL_TILE and w8.plan(m, n, k).splits > 1
    a, w, scale, s = big_operands(m, n, k, 3)
    x, bias = torch.randn(m, n, device="cuda").to(BF16), torch.randn(n, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):       # workspaces grow before the capture
        w8.gemm_epilogue(a, w, scale, bias=bias, residual=x)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            y = w8.gemm_epilogue(a, w, scale, bias=bias, residual=x)
        for _ in range(4):
            x.copy_(torch.randn(m, n, device="cuda"))
            y.zero_()
            graph.replay()
            eager = w8.gemm_epilogue(a, w, scale, bias=bias, residual=x)
            stream.synchronize()
            assert torch.equal(y, eager)
            check(y, s, bias, None, None, x)
