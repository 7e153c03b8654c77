"""Products on operands of one row, whose row stride says nothing."""

import pytest

import block_scaled_fp8_w8a16_amd as w8mod
from test_product_epilogue import BF16, F32, operands, w8  # noqa: F401

torch = pytest.importorskip("torch")


@pytest.mark.gpu
@pytest.mark.parametrize("pitch", [0, 1, 131, 4096 * (1 << 20), (1 << 33) + 3])
def test_one_row(w8, pitch):
    n, k = 24, 128
    a, w, scale, _ = operands(1, n, k, 1)
    g = torch.Generator(device="cuda").manual_seed(2)
    gate, res = (torch.randn(1, n, generator=g, device="cuda").to(t) for t in (BF16, F32))
    want = w8.gemm_epilogue(a, w, scale, activation="silu", gate=gate, residual=res, out_dtype=F32)

    def view(t):
        return t.as_strided(t.shape, (pitch, 1))
    c = torch.empty(1, n, device="cuda")
    got = w8.gemm_epilogue(view(a), w, scale, view(c), activation="silu", gate=view(gate), residual=view(res))
    assert torch.equal(got, want) and torch.equal(c, want)
    plain = torch.empty(1, n, device="cuda", dtype=BF16)
    assert torch.equal(w8.gemm(view(a), w, scale, view(plain)), w8.gemm(a, w, scale))
