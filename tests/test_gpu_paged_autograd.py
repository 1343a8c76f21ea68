"""The rotation of token tensors under autograd: x.grad through backward() against the
transposed rotation in 64 bits and against differences."""
import numpy as np
import pytest
import torch

import sink_window_attention_b200 as swa
from oracle import tokens
from tests.test_gpu_tokens import f64, i32

pytestmark = pytest.mark.gpu
POS = [0, 1, 17, 4095, 100000, 7, 8]


def setup(layout, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, y = (torch.randn((7, 3, 64), generator=g, device="cuda").to(dtype) for _ in range(2))
    return x, y, i32(POS), swa.TokenRope(32, layout=layout, amplitude=1.5)


def bound(y, want, dtype):
    # a rotated element is within 1.5e-6 of 1.5 (|a| + |b|) of its pair (both below max|y|), then rounded
    u = 2.0**-8 if dtype == torch.bfloat16 else 2.0**-24
    return 2 * 1.5 * 1.5e-6 * np.abs(f64(y)).max() + u * np.abs(want)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("transpose", [False, True])
def test_gradient_through_backward(layout, dtype, transpose):
    x, y, pos, rope = setup(layout, dtype)
    plain = swa.token_rope_apply(x, pos, rope, transpose)
    x.requires_grad_()
    out = swa.token_rope_apply(x, pos, rope, transpose)
    assert out.requires_grad and torch.equal(out, plain)
    out.backward(y)
    want = tokens.rotate(f64(y), POS, tokens.frequencies(32), layout, 1.5, not transpose)
    assert x.grad.dtype == dtype and np.all(np.abs(f64(x.grad) - want) <= bound(y, want, dtype))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_against_differences(layout):
    """y . R(x) is linear in x, so a step of 1 is exact but for fp32's rounding of 64 terms."""
    x, y, pos, rope = setup(layout, torch.float32, 3)
    base = f64(swa.token_rope_apply(x, pos, rope))
    x.requires_grad_()
    (swa.token_rope_apply(x, pos, rope) * y).sum().backward()
    for d in range(64):
        step = x.detach().clone()
        step[:, :, d] += 1.0
        moved = f64(step[:, :, d]) - f64(x[:, :, d])
        diff = np.sum((f64(swa.token_rope_apply(step, pos, rope)) - base) * f64(y), axis=-1)
        assert np.abs(diff - f64(x.grad[:, :, d]) * moved).max() <= 64 * 4 * 1.5e-6


def test_gradients_of_a_fused_projection_and_of_a_shared_input():
    """Slices of one tensor (rows further apart), the same slice used twice, and incoming
    gradients that are expanded, permuted or off a 16-byte boundary."""
    _, _, pos, rope = setup("half", torch.float32)
    wide = torch.randn((7, 8, 64), device="cuda", requires_grad=True)
    a = swa.token_rope_apply(wide[:, :3], pos, rope)
    b = swa.token_rope_apply(wide[:, 2:7], pos, rope)
    (a.sum() + (b.transpose(0, 1) ** 2).sum() / 2).backward()
    w = tokens.frequencies(32)
    want = np.zeros((7, 8, 64))
    want[:, :3] += tokens.rotate(np.ones((7, 3, 64)), POS, w, "half", 1.5, True)
    turned = tokens.rotate(f64(wide[:, 2:7]), POS, w, "half", 1.5)
    want[:, 2:7] += tokens.rotate(turned, POS, w, "half", 1.5, True)
    assert np.abs(f64(wide.grad) - want).max() <= 1e-4
    x = wide.detach()[:, :3].clone().requires_grad_()
    odd = torch.randn(7 * 3 * 64 + 1, device="cuda")[1:].view(7, 3, 64)
    swa.token_rope_apply(x, pos, rope).backward(odd)
    assert np.abs(f64(x.grad) - tokens.rotate(f64(odd), POS, w, "half", 1.5, True)).max() <= 5e-5


def test_second_derivative():
    x, y, pos, rope = setup("interleaved", torch.float32)
    x.requires_grad_()
    y.requires_grad_()
    g, = torch.autograd.grad((swa.token_rope_apply(x, pos, rope) * y).sum(), x, create_graph=True)
    v = torch.randn_like(x)
    gy, = torch.autograd.grad((g * v).sum(), y)
    assert torch.equal(gy, swa.token_rope_apply(v, pos, rope))


def test_where_no_graph_is_made():
    x, _, pos, rope = setup("half", torch.float32)
    want = swa.token_rope_apply(x, pos, rope)
    x.requires_grad_()
    with torch.no_grad():
        out = swa.token_rope_apply(x, pos, rope)
        assert not out.requires_grad and torch.equal(out, want)
        buf = torch.empty_like(x)
        assert swa.token_rope_apply(x, pos, rope, out=buf) is buf
    empty = torch.zeros((0, 3, 64), device="cuda", requires_grad=True)
    swa.token_rope_apply(empty, i32([]), rope).sum().backward()
    assert empty.grad.shape == (0, 3, 64)
    # positions that are written before backward are noticed
    out = swa.token_rope_apply(x, pos, rope)
    pos.add_(1)
    with pytest.raises(RuntimeError, match="modified"):
        out.sum().backward()


def test_on_a_side_stream_and_captured():
    x, y, pos, rope = setup("half", torch.float32)
    want = swa.token_rope_apply(y, pos, rope, transpose=True)
    x.requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = swa.token_rope_apply(x, pos, rope, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    out.backward(y)
    assert torch.equal(x.grad, want)
    del out
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, = torch.autograd.grad(swa.token_rope_apply(x, pos, rope), x, y)
    for _ in range(2):
        with torch.no_grad():
            y.normal_()
        graph.replay()
        assert torch.equal(got, swa.token_rope_apply(y, pos, rope, transpose=True))
