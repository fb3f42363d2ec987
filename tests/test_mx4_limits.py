"""The MX4 operators at the ends of their types' ranges, where a factor, a product
of two or an expanded weight leaves float32 although the result does not.

Bounds are those of test_mx4_grad.py; where everything is a power of two, a small
integer or zero, nothing is rounded and results are compared for equality."""

import numpy as np
import pytest
import torch

from oracle import mx4

pq2 = pytest.importorskip("gemm_pq2_w2a8_amd")

import test_mx4_grad as grad  # noqa: E402

TYPES, ACTS = grad.TYPES, grad.ACTS


def test_workspace_query_at_the_width_limits():
    """A gated block's rows are both halves: the width a product still takes, and
    splits, is refused for it and taken at half."""
    f, K = pq2.lib.pq2_mx4_workspace_bytes, 1 << 14
    for rows in (1 << 20) + 128, (1 << 20) + 64:
        assert f(64, rows, K, 0) > 0 and f(64, rows, K, 1) == 0
        assert f(64, rows // 2, K, 1) == f(64, rows, K, 0)
    assert f(64, (1 << 21) + 1, K, 0) == 0


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


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(5, 64, 128), (33, 200, 256), (64, 5120, 256), (130, 1000, 512), (3100, 264, 4096),
                                   (2050, 100, 7040)])
def test_gradients_under_scales_of_every_size(M, N, K, ty):
    """Scale bytes 0, 1, 252, 253 and 254, in one row of the weights each. Their
    weights meet gradients that are 0, that take the product back among small
    integers, that are small integers themselves (products in and beyond float32's
    range), 2^127 (2^15 in float16) or infinite; nothing is rounded but the output."""
    ends = (0, 1, 252, 253, 254)
    codes, scales = grad.weights(N, K, 1, flat=True)
    g = torch.Generator(device="cuda").manual_seed(N)
    dy = torch.randint(-4, 5, (M, N), device="cuda", generator=g).double()
    kind = torch.arange(M, device="cuda") % 5
    dy[kind >= 2] = 0
    for i, byte in enumerate(ends):
        n = (N - 1) * i // 4
        own = torch.arange(K // 32, device="cuda") % 5 == i
        codes[n, ~own.repeat_interleave(16)] = 0
        scales[n, own] = byte
        v = torch.randint(1, 5, (M,), device="cuda", generator=g).double()
        v[torch.rand(M, device="cuda", generator=g) < 0.5] *= -1
        back = 0.0 if ty == "f16" else 2.0 ** (120 if byte < 2 else 127 - byte)
        most = 2.0 ** (15 if ty == "f16" else 127)
        size = torch.tensor([0.0, back, 1.0, most, torch.inf], dtype=torch.float64, device="cuda")[kind]
        dy[:, n] = torch.where(size >= most, size * v.sign(), size * v)
    dy = dy.to(TYPES[ty])
    dx = torch.full((M, K), 7.0, dtype=TYPES[ty], device="cuda")
    pq2.pq2_mx4_gemm_grad(dy, codes, scales, dx)
    # powers of two from the host: the device's power function is one step off at 2^125
    powers = torch.from_numpy(np.ldexp(1.0, scales.cpu().numpy().astype(np.int32) - 127)).cuda()
    values = grad.decoded(codes, torch.full_like(scales, 127)) * powers.repeat_interleave(32, 1)
    want = (dy.double() @ values).float().to(TYPES[ty])
    assert ((dx == want) | (dx.isnan() & want.isnan())).all()
    assert torch.isfinite(want[kind < 2]).all() and torch.isfinite(dx[kind < 2]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("byte", [127, 252])
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
def test_the_smallest_gradients(ty, byte):
    """One weight a column, 1 or 2^125: dx is dy itself, subnormals too. Of float32
    below 2^-110 (the three parts' last bit there: 2^(-110 - 23) = 2^-133) what lies
    below 2^-133 is cut off, and nothing else."""
    N = K = 128
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    for n in range(N):
        codes[n, n // 2] = 2 << (4 * (n % 2))            # 1.0
    scales = torch.full((N, K // 32), byte, dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(4)
    sign, frac, power = (torch.randint(0, n, (500, N), generator=g) for n in (2, 1 << 23, 24))
    if ty == "f32":
        dy = (frac | power << 23).to(torch.int32).view(torch.float32)
    else:
        dy = (frac & 0x3ff if ty == "f16" else frac & 0x7f | power << 7).to(torch.int16).view(TYPES[ty])
    dy = torch.where(sign == 1, -dy, dy)
    dx = torch.empty(500, K, dtype=TYPES[ty], device="cuda")
    pq2.pq2_mx4_gemm_grad(dy.cuda(), codes, scales, dx)
    want = dy.double()
    if ty == "f32":
        cut = torch.trunc(want * 2.0 ** 133) * 2.0 ** -133
        assert (cut == want)[want.abs() >= 2.0 ** -110].all() and (cut != want).any()
        want = cut
    assert torch.equal(dx.cpu(), (want * 2.0 ** (byte - 127)).to(TYPES[ty]))


@pytest.mark.parametrize("kw,want", [
    # rows of 13 columns: the elements' alignment (then the workspace is too small)
    (dict(dy=grad.P + 4, fmt=0, N=13), grad.ERR_SCRATCH), (dict(dy=grad.P + 2, fmt=1, N=13), grad.ERR_SCRATCH),
    (dict(dy=grad.P + 2, fmt=2, N=13), grad.ERR_SCRATCH), (dict(dy=grad.P + 2, fmt=0, N=13), grad.ERR_ALIGN),
    (dict(dy=grad.P + 1, fmt=1, N=13), grad.ERR_ALIGN), (dict(dy=grad.P + 4, fmt=0, N=16), grad.ERR_ALIGN),
])
def test_alignment_of_odd_rows(kw, want):
    assert grad.gemm_grad(size=0, **kw) == want
    assert grad.gated_grad(size=0, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(gu=grad.P + 4, N=13), grad.ERR_SCRATCH), (dict(gu=grad.P + 2, N=13), grad.ERR_ALIGN),
    (dict(dgu=grad.P + 4, N=13), grad.ERR_SCRATCH), (dict(dgu=grad.P + 2, N=13), grad.ERR_ALIGN),
    # 12 columns, and 24 of both halves
    (dict(dy=grad.P + 4, gu=grad.P + 4, N=12), grad.ERR_SCRATCH), (dict(dgu=grad.P + 4, N=12), grad.ERR_ALIGN),
])
def test_alignment_of_odd_rows_of_the_gated_block(kw, want):
    assert grad.gated_grad(fmt=0, size=0, **kw) == want


def off_by_one(t):
    """The same rows, one element past an aligned address."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    buf[1:] = t.flatten()
    return buf[1:].view(t.shape)


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 7, 128), (33, 100, 256), (130, 1411, 384), (3100, 260, 4096)])
def test_gradients_of_odd_rows_from_any_element(M, N, K, ty):
    w, dy = grad.weights(N, K, 1), grad.randn(M, N, ty, 1)
    dx, other = (torch.full((M, K), 7.0, dtype=TYPES[ty], device="cuda") for _ in range(2))
    pq2.pq2_mx4_gemm_grad(dy, *w, dx)
    pq2.pq2_mx4_gemm_grad(off_by_one(dy), *w, other)
    assert torch.equal(dx, other)


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,F,K", [(1, 7, 128), (33, 100, 256), (130, 1411, 384)])
def test_gated_gradients_of_odd_rows_from_any_element(M, F, K, ty):
    w, dh, gu = grad.weights(2 * F, K, 1), grad.randn(M, F, ty, 1), grad.randn(M, 2 * F, ty, 2)
    dx, dgu = gated_grad(dh, gu, "silu", w)
    other = torch.full_like(dx, 7.0)
    pq2.pq2_mx4_gated_grad(off_by_one(dh), off_by_one(gu), *w, other)
    assert torch.equal(dx, other)
    if F % 4:
        odd = off_by_one(gu)                             # and dgu in its place
        pq2.pq2_mx4_gated_grad(dh, odd, *w, other, dgu=odd)
        assert torch.equal(dx, other) and torch.equal(odd, dgu)
