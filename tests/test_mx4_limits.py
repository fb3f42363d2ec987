"""The MX4 operators at the ends of their types' ranges, where a factor, a product
of two or an expanded weight leaves float32 although the result does not.

Bounds are those of test_mx4_grad.py; where everything is a power of two, a small
integer or zero, nothing is rounded and results are compared for equality."""

import pytest
import torch

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
