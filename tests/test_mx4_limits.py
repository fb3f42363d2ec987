"""The MX4 operators at the ends of their types' ranges, where a factor, a product
of two or an expanded weight leaves float32 although the result does not.

Bounds are those of test_mx4_grad.py; where everything is a power of two, a small
integer or zero, nothing is rounded and results are compared for equality."""

import pytest
import torch

from oracle import mx4

pq2 = pytest.importorskip("gemm_pq2_w2a8_amd")

import test_mx4_grad as grad  # noqa: E402

TYPES, ACTS = grad.TYPES, grad.ACTS


def gated_grad(dh, gu, act, w):
    F = dh.shape[1]
    dx = torch.full((len(dh), 2 * w[0].shape[1]), 7.0, dtype=dh.dtype, device="cuda")
    dgu = torch.full((len(dh), 2 * F), 7.0, dtype=dh.dtype, device="cuda")
    pq2.pq2_mx4_gated_grad(dh, gu, *w, dx, dgu=dgu, act=act)
    return dx, dgu


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("ty", ["bf16", "f32"])
def test_slopes_of_gates_whose_square_is_infinite(ty, act):
    """Slopes are 0 and 1 and values 0 and g, to the last bit; dx of the same row
    is finite."""
    far = torch.tensor([1e10, 1e18, 1.8e19, 1.9e19, 4e19, 1e20, 1e30, 2.0 ** 127, 3.3e38])
    g = torch.cat([-far, far]).repeat(3).to(TYPES[ty]).cuda()
    F, t = len(g), 2.0 ** -20
    w = grad.weights(2 * F, 256, 1)
    gu = torch.cat([g, torch.ones_like(g)])[None].contiguous()
    dx, dgu = gated_grad(torch.full((1, F), t, dtype=TYPES[ty], device="cuda"), gu, act, w)
    assert torch.equal(dgu[0, :F].float(), torch.where(g > 0, t, 0.0))
    assert torch.equal(dgu[0, F:], torch.where(g > 0, g * t, torch.zeros_like(g)))
    assert torch.isfinite(dx).all()
    grad.check(dx, *grad.product(dgu, grad.decoded(*w), ty), ty)


@pytest.mark.gpu
@pytest.mark.parametrize("act,g", [("silu", -50.0), ("gelu", -10.0), ("gelu_tanh", -5.5)])
@pytest.mark.parametrize("ty", ["bf16", "f32"])
def test_slopes_near_zero_of_large_gradients(ty, act, g):
    """dh u is infinite in float32, times the slope it is not: the activation's
    relative (10 + 3 max(|z|, g^2)) 2^-23 of test_mx4_grad.py, |z| <= 21 and g^2 <=
    100 but for silu, which has no g^2, on a slope of two terms of which one is the
    other's g-fold: below 2^-13 in all. Slopes that are 0 give zeros."""
    F, big = 64, 1e20
    gates = torch.tensor([g, -1e3, -1e10, g]).repeat(F // 4).to(TYPES[ty]).cuda()
    dh = torch.full((2, F), big, dtype=TYPES[ty], device="cuda")
    dh[1] = -dh[0]
    gu = torch.cat([gates, torch.full_like(gates, big)]).repeat(2, 1)
    w = grad.weights(2 * F, 128, 1)
    dx, dgu = gated_grad(dh, gu, act, w)
    slope = torch.from_numpy(mx4.act(act, gates.double().cpu().numpy())[1]).cuda()
    want = dh.double() * gu[:, F:].double() * slope
    assert (dgu[:, :F][:, gates < -100] == 0).all()
    off = (dgu[:, :F].double() - want).abs()
    assert (off <= (2.0 ** -13 + grad.HALF[ty]) * want.abs()).all()
    grad.check(dx, *grad.product(dgu, grad.decoded(*w), ty), ty)
