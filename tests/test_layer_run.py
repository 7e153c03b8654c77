"""The operators together, as a served layer uses them: the example's whole
layer against plain arithmetic, its captured steps against eager ones, a
shared prefix against its copies, and a training step through the rotation."""

import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import decode_layer as ex  # noqa: E402

SMALL = dict(hidden=512, q_heads=8, kv_heads=2, head_dim=64, page_size=16)


def test_picture_positions():
    p = ex.picture_positions(2, 3, 2, 10)
    assert p.tolist() == [[10] * 6 + [13, 14], [10, 10, 10, 11, 11, 11, 13, 14], [10, 11, 12] * 2 + [13, 14]]


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.gpu
@pytest.mark.parametrize("prompts,kw", [
    ([130, 3, 1, 70], dict(prefix=96, chunk=64)), ([40, 17], dict(prefix=0, window=33, sinks=5)),
    ([5, 60, 61], dict(prefix=256, chunk=128)), ([90, 200], dict(prefix=48, window=50, sinks=64))])
def test_served_layer_matches_the_plain_one(gpu, prompts, kw):
    # keys and values are rounded to E4M3, by at most 2^-4 of each
    worst, _ = ex.run_layer(prompts, 6, **kw, **SMALL)
    assert worst < 2.0 ** -4


def make(prefix, prompts, steps, shared):
    """Layer, tables and inputs; without `shared` every sequence has the
    prefix on pages of its own."""
    g = torch.Generator().manual_seed(5)
    common = torch.randn(prefix, 512, generator=g).to(torch.bfloat16).cuda()
    xs = [torch.randn(n + steps, 512, generator=g).to(torch.bfloat16).cuda() for n in prompts]
    if shared:
        table, pages = ex.share_pages([n + steps for n in prompts], prefix, 16)
    else:
        table, pages = ex.lay_out_pages([prefix + n + steps for n in prompts], 16)
    layer = ex.DecoderLayer(512, 8, 2, 64, pages, 16, prefix + max(prompts) + steps, seed=3,
                            sections=[16, 8, 8], shared=prefix if shared else 0)
    at = torch.arange(prefix, dtype=torch.int32).expand(3, -1).contiguous().cuda()
    for row in range(1 if shared else len(prompts)):
        ex.prefill(layer, [common], table[row:row + 1], 64, positions=[at])
    places = [ex.picture_positions(3, 4, n, prefix)[:, :n].contiguous().cuda() for n in prompts]
    outs, lens = ex.prefill(layer, [x[:n] for x, n in zip(xs, prompts)], table, 32, prefix, places)
    last = torch.stack([p[:, -1] for p in places], 1).contiguous()
    return layer, table, xs, outs, lens, last


@pytest.mark.gpu
def test_captured_steps_are_the_eager_ones(gpu):
    prompts, steps = [20, 1, 33, 16, 7, 50, 3, 9, 80, 2, 12, 31], 8
    layer, table, xs, _, lens, last = make(512, prompts, steps, True)
    other, _, _, _, elens, elast = make(512, prompts, steps, True)
    graph = ex.DecodeGraph(layer, table, lens, 512, last)
    for i in range(steps):
        x = torch.stack([x[n + i] for x, n in zip(xs, prompts)])
        got = graph.step(x).clone()
        elens += 1
        elast += 1
        want = other(x, table, elens, positions=elast)
        torch.cuda.synchronize()
        assert torch.equal(got, want), i
    assert torch.equal(lens, elens) and torch.equal(last, elast)
    for a, b in zip(layer.cache, other.cache):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_shared_prefix_is_its_copies(gpu):
    """Held once or by every sequence: the same tokens give the same keys and
    values, so outputs differ by the order of the softmax's sums alone, that
    is by roundings to bfloat16 that fall to the other side."""
    prompts, steps = [20, 1, 33, 16, 7, 50, 3, 9], 4
    layer, table, xs, outs, lens, last = make(256, prompts, steps, True)
    copies, ctable, _, couts, clens, clast = make(256, prompts, steps, False)
    for a, b in zip(outs, couts):
        torch.testing.assert_close(a, b, rtol=2.0 ** -4, atol=2.0 ** -4)
    for i in range(steps):
        x = torch.stack([x[n + i] for x, n in zip(xs, prompts)])
        for t in (lens, last, clens, clast):
            t += 1
        a, b = layer(x, table, lens, positions=last), copies(x, ctable, clens, positions=clast)
        # (a rounding of the attention's outputs, 2^-8 of one, passes two
        # products whose weights keep the size of their inputs)
        torch.testing.assert_close(a, b, rtol=2.0 ** -4, atol=2.0 ** -4)


class Turned(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, table, positions, sections):
        ctx.save_for_backward(table, positions)
        ctx.sections = sections
        return ex.w8.rope(x, table, positions, sections=sections)

    @staticmethod
    def backward(ctx, dy):
        table, positions = ctx.saved_tensors
        return ex.w8.rope(dy.contiguous(), table, positions, sections=ctx.sections, inverse=True), None, None, None


@pytest.mark.gpu
def test_a_training_step_through_the_rotation(gpu):
    """Gradients of a weight in front of the rotation against FP64 (sums of 40 products of FP32 roundings, far below 1e-4)."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(40, 32, generator=g).cuda()
    w = (torch.randn(32, 4 * 32, generator=g) * 0.2).cuda().requires_grad_()
    target = torch.randn(40, 4, 32, generator=g).cuda()
    table = ex.w8.rope_table(64, 32)
    positions = ex.picture_positions(5, 6, 10).cuda()

    def loss(w):
        y = Turned.apply((x @ w).view(40, 4, 32), table, positions, [6, 5, 5])
        return ((y - target) ** 2).mean()
    grad, = torch.autograd.grad(loss(w), w)
    axis = torch.arange(3).repeat_interleave(torch.tensor([6, 5, 5])).cuda()
    turn = table.double()[positions[axis].long(), torch.arange(16, device="cuda")[:, None]].permute(2, 1, 0)[:, :, None]
    w64 = w.detach().double().requires_grad_()
    y = (x.double() @ w64).view(40, 4, 32)
    a, b = y[..., :16], y[..., 16:]
    y = torch.cat([a * turn[0] - b * turn[1], b * turn[0] + a * turn[1]], -1)
    want, = torch.autograd.grad(((y - target.double()) ** 2).mean(), w64)
    torch.testing.assert_close(grad.double(), want, rtol=1e-4, atol=1e-6)
