"""pq2_mx4_gemm_grad and pq2_mx4_gated_grad: gradients through MX4 weights.

The reference is float64. The weights are exact in bfloat16, the incoming
gradient enters as one to three bfloat16 parts that add up to it, their products
are exact in float32, and a float32 sum of P N terms, whatever its order and
with additions that round or truncate, is within E = P N 2^-23 sum|terms| of the
exact one, with the parts' magnitudes adding up to the value's (all parts have
its sign). With integers and scales alike nothing is rounded anywhere. A stored
16-bit value adds half a step of its type.

The gated block's dg and du: a relative A = (10 + 3 max(|z|, g^2)) 2^-23 for the
activation (tests of the forward pass) and as much, of the size of the slope's
terms (at most 2.5 in sum), for its derivative, two products more, and half a
step. dx is checked against the exact product of the dgu returned.
"""

import numpy as np
import pytest
import torch

from oracle import mx4

pq2 = pytest.importorskip("gemm_pq2_w2a8_amd")

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}
PARTS = {"f32": 3, "bf16": 1, "f16": 2}
ACTS = ("silu", "gelu", "gelu_tanh")
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_HIP, ERR_ARG, ERR_SCRATCH = range(7)
P = 0x100000


# ------------------------------------------------------------------ refusals (CPU)

def gemm_grad(dy=P, w=P, ws=P, dx=P, fmt=1, M=1, N=8, K=128, work=P, size=1 << 40):
    return pq2.lib.pq2_mx4_gemm_grad(dy, w, ws, dx, fmt, M, N, K, work, size, None)


def gated_grad(dy=P, gu=P, act=0, w=P, ws=P, dgu=P, dx=P, fmt=1, M=1, N=8, K=128, work=P, size=1 << 40):
    return pq2.lib.pq2_mx4_gated_grad(dy, gu, act, w, ws, dgu, dx, fmt, M, N, K, work, size, None)


@pytest.mark.parametrize("call", [gemm_grad, gated_grad])
@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), ERR_NULL), (dict(w=None), ERR_NULL), (dict(ws=None), ERR_NULL),
    (dict(dx=None), ERR_NULL), (dict(M=-1), ERR_SHAPE), (dict(N=0), ERR_SHAPE),
    (dict(N=(1 << 21) + 1), ERR_SHAPE), (dict(K=0), ERR_SHAPE), (dict(K=192), ERR_SHAPE),
    (dict(K=(1 << 21) + 128), ERR_SHAPE), (dict(M=(1 << 26) + 1), ERR_SHAPE),
    (dict(M=1 << 26, N=1 << 15), ERR_SHAPE), (dict(M=1 << 26, K=1 << 15), ERR_SHAPE),
    (dict(fmt=3), ERR_ARG), (dict(fmt=-1), ERR_ARG), (dict(dy=P + 8), ERR_ALIGN),
    (dict(w=P + 8), ERR_ALIGN), (dict(ws=P + 2), ERR_ALIGN), (dict(dx=P + 1), ERR_ALIGN),
    (dict(dx=P + 2, fmt=0), ERR_ALIGN), (dict(work=P + 8), ERR_ALIGN),
    # the parts of one row of 64 columns, less a byte, or none at all
    (dict(fmt=0, size=3 * 64 * 2 - 1), ERR_SCRATCH), (dict(fmt=2, size=255), ERR_SCRATCH),
    (dict(fmt=0, work=None), ERR_SCRATCH), (dict(N=13, fmt=1, size=127), ERR_SCRATCH),
    (dict(M=0), OK), (dict(M=0, dy=None, work=None), OK),
])
def test_refusals(call, kw, want):
    assert call(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(gu=None), ERR_NULL), (dict(act=3), ERR_ARG), (dict(act=-1), ERR_ARG),
    (dict(gu=P + 8), ERR_ALIGN), (dict(dgu=P + 8), ERR_ALIGN), (dict(N=(1 << 20) + 1), ERR_SHAPE),
    (dict(N=1 << 20, K=1 << 15), ERR_SHAPE), (dict(dgu=None, size=31), ERR_SCRATCH),
    (dict(dgu=None, work=None), ERR_SCRATCH), (dict(N=7, size=127), ERR_SCRATCH),
])
def test_refusals_of_the_gated_block(kw, want):
    assert gated_grad(**kw) == want


def test_workspace_queries():
    f, g = pq2.lib.pq2_mx4_grad_workspace_bytes, pq2.lib.pq2_mx4_gated_grad_workspace_bytes
    assert f(0, 8, 128, 1) == 0 and f(1, 8, 100, 1) == 0 and f(1, 8, 128, 3) == 0
    assert g(0, 8, 128, 1, 1) == 0 and g(1, 8, 100, 1, 1) == 0 and g(1, 8, 128, 3, 1) == 0
    assert f(10, 100, 128, 0) >= 3 * 10 * 128 * 2 and f(10, 100, 128, 2) >= 2 * 10 * 128 * 2
    assert f(10, 100, 128, 1) >= 10 * 128 * 2       # 100 is no multiple of 8
    assert g(10, 100, 128, 1, 0) >= 10 * 200 * 2
    assert g(10, 100, 128, 1, 0) >= g(10, 100, 128, 1, 1)


# ------------------------------------------------------------------ GPU

def weights(N, K, seed, flat=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(121, 126, (N, K // 32), dtype=torch.uint8, device="cuda", generator=g)
    if flat:
        scales.fill_(127)
    return codes, scales


def decoded(codes, scales):
    table = torch.tensor(np.concatenate([mx4.VALUES, -mx4.VALUES]), device="cuda")
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(1).long()
    s = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), scales.int() - 127)
    return table[c] * torch.where(scales == 255, torch.nan, s).repeat_interleave(32, 1)


def randn(M, N, ty, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(M, N, device="cuda", generator=g).to(TYPES[ty])


def product(d, w, ty):
    return d.double() @ w, PARTS[ty] * d.shape[1] * 2.0 ** -23 * (d.double().abs() @ w.abs())


def check(got, want, bound, ty):
    tol = bound + HALF[ty] * (want.abs() + bound) + TINY[ty]
    off = (got.double() - want).abs()
    assert (off <= tol).all(), (off / tol).max().item()


SHAPES = [(1, 1, 128), (1, 8, 256), (2, 63, 384), (15, 64, 512), (16, 65, 128), (17, 136, 1024),
          (33, 256, 896), (64, 511, 128), (65, 1411, 640), (130, 300, 1152), (257, 72, 2176),
          (1, 5120, 640), (5, 2050, 5120), (300, 4104, 256)]
BIG = [(3100, 264, 4096), (2050, 100, 7040)]


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES + BIG)
def test_gemm_grad(M, N, K, ty):
    w, dy = weights(N, K, N + K), randn(M, N, ty, M + N)
    dx = torch.full((M, K), 7.0, dtype=TYPES[ty], device="cuda")
    pq2.pq2_mx4_gemm_grad(dy, *w, dx)
    check(dx, *product(dy, decoded(*w), ty), ty)


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES + BIG + [(40, 17408, 512)])
def test_gemm_grad_exact(M, N, K, ty):
    """Small integers and scales alike: no rounding but the output's."""
    w = weights(N, K, 1, flat=True)
    dy = torch.randint(-4, 5, (M, N), device="cuda").to(TYPES[ty])
    dx = torch.empty(M, K, dtype=TYPES[ty], device="cuda")
    pq2.pq2_mx4_gemm_grad(dy, *w, dx)
    assert torch.equal(dx, (dy.double() @ decoded(*w)).float().to(TYPES[ty]))


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 17408, 1024), (33, 5120, 17408), (300, 5120, 6144), (1000, 2048, 17408),
                                   (2048, 2048, 8704), (4000, 1000, 5120), (32, 34816, 1024), (17, 1000, 17408)])
def test_plans_agree(M, N, K, ty):
    """Both tiles, whole and split along N in any workspace: small integers, no
    rounding but the output's, so the same bits; some rows against float64."""
    w = weights(N, K, 1, flat=True)
    dy = torch.randint(-4, 5, (M, N), device="cuda").to(TYPES[ty])
    dx, other = (torch.full((M, K), 7.0, dtype=TYPES[ty], device="cuda") for _ in range(2))
    pq2.pq2_mx4_gemm_grad(dy, *w, dx)
    least = 0 if ty == "bf16" and N % 8 == 0 else (PARTS[ty] * M * ((N + 63) // 64 * 64) * 2 + 255) // 256 * 256
    most = pq2.mx4_grad_workspace_bytes(M, N, K, TYPES[ty])
    for n in {least, (least + most) // 2, least + (most - least) // 7}:
        work = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")[:n]
        pq2.pq2_mx4_gemm_grad(dy, *w, other, workspace=work if n else None)
        assert torch.equal(dx, other)
    some = sorted({0, M // 3, M // 2, M - 1})
    assert torch.equal(dx[some], (dy[some].double() @ decoded(*w)).float().to(TYPES[ty]))


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
def test_every_bit_of_the_gradient_counts(ty):
    """One weight a column: dx is dy itself, to the last bit, over the type's range."""
    N = K = 128
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    for n in range(N):
        codes[n, n // 2] = 2 << (4 * (n % 2))            # 1.0
    scales = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    bits = torch.randint(-2 ** 31, 2 ** 31 - 1, (300, N), generator=torch.Generator().manual_seed(2))
    if ty == "f32":
        dy = bits.to(torch.int32).view(torch.float32)
    else:
        dy = bits.to(torch.int16).view(TYPES[ty])
    # parts down to the smallest normal bfloat16 (and their float32 sums) are kept
    low = {"f32": 2.0 ** -126 * 2 ** 24, "bf16": 2.0 ** -126, "f16": 0.0}[ty]
    dy = torch.where(torch.isfinite(dy.double()) & (dy.double().abs() >= low), dy, torch.ones_like(dy))
    dx = torch.empty(300, K, dtype=TYPES[ty], device="cuda")
    pq2.pq2_mx4_gemm_grad(dy.cuda(), codes, scales, dx)
    assert torch.equal(dx.cpu(), dy)


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N", [64, 100, 200])
def test_infinities_and_nan_stay_in_their_rows(N, ty):
    M, K = 70, 256
    w = weights(N, K, 3, flat=True)
    w[0][:, 0] = 0x22                                    # the first two columns: ones
    dy = torch.randint(-4, 5, (M, N), device="cuda").to(TYPES[ty])
    want = dy.double() @ decoded(*w)
    dy[5, N - 1], dy[40, 0], dy[69, N // 2] = torch.inf, torch.nan, -torch.inf
    dx = torch.empty(M, K, dtype=TYPES[ty], device="cuda")
    pq2.pq2_mx4_gemm_grad(dy, *w, dx)
    rest = [m for m in range(M) if m not in (5, 40, 69)]
    assert torch.equal(dx[rest], want[rest].float().to(TYPES[ty]))
    assert torch.isnan(dx[40]).all() and not torch.isfinite(dx[[5, 69]]).any()
    assert (dx[5, :2] == torch.inf).all() and (dx[69, :2] == -torch.inf).all()


@pytest.mark.gpu
def test_a_scale_that_is_not_a_number_stays_in_its_columns():
    M, N, K = 33, 100, 512
    w, dy = weights(N, K, 3, flat=True), torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
    w[1][N - 1, 3] = 255
    dx = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    pq2.pq2_mx4_gemm_grad(dy, *w, dx)
    nan = torch.isnan(dx)
    assert nan[:, 96:128].all() and not nan[:, :96].any() and not nan[:, 128:].any()


def gated_reference(dh, gu, act, ty):
    """Exact dgu and its bound."""
    F = dh.shape[1]
    g, u, d = gu[:, :F].double(), gu[:, F:].double(), dh.double()
    a, s = (torch.from_numpy(v).cuda() for v in mx4.act(act, g.cpu().numpy()))
    z = torch.maximum(g.abs(), 1.6 * (g + 0.0447 * g ** 3).abs()) if act == "gelu_tanh" else g.abs()
    rel = torch.minimum((10 + 3 * torch.maximum(z, g * g)) * 2.0 ** -23, torch.ones_like(g))
    dg, du = d * u * s, d * a
    # the slope's second term dies off with the distance from zero faster than its bound grows
    own = torch.cat([(d * u).abs() * 2.5 * torch.minimum(rel, torch.full_like(rel, 60 * 2.0 ** -23)),
                     rel * du.abs()], 1)
    want = torch.cat([dg, du], 1)
    return want, own + 2.0 ** -22 * want.abs()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,F,K", [(1, 1, 128), (1, 8, 256), (3, 33, 384), (17, 100, 640), (65, 200, 1024),
                                   (131, 1411, 896), (1, 5120, 640), (3100, 132, 4096)])
def test_gated_grad(M, F, K, ty, act):
    w = weights(2 * F, K, F + K)
    dh, gu = randn(M, F, ty, M + F), 2 * randn(M, 2 * F, ty, F)
    dx, dgu = (torch.full((M, n), 7.0, dtype=TYPES[ty], device="cuda") for n in (K, 2 * F))
    pq2.pq2_mx4_gated_grad(dh, gu, *w, dx, dgu=dgu, act=act)
    want, bound = gated_reference(dh, gu, act, ty)
    check(dgu, want, bound, ty)
    check(dx, *product(dgu, decoded(*w), ty), ty)
    # without dgu, and with dgu in place of gu: the same
    again = torch.empty_like(dx)
    pq2.pq2_mx4_gated_grad(dh, gu, *w, again, act=act)
    assert torch.equal(again, dx)
    pq2.pq2_mx4_gated_grad(dh, gu, *w, again, dgu=gu, act=act)
    assert torch.equal(again, dx) and torch.equal(gu, dgu)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_gated_grad_far_ends(act):
    """Gates of every size: slopes 0 and 1, never NaN."""
    g = torch.tensor([-3e38, -1e30, -1e10, -300.0, -90.0, -40.0, 0.0, -0.0, 40.0, 90.0, 300.0, 1e6])
    if act == "gelu_tanh":
        g = g.clamp(-1e12, 1e12)                         # its cube is finite
    g = g.repeat(8)
    F = len(g)
    gu = torch.cat([g, torch.ones(F)])[None].cuda()
    w = weights(2 * F, 128, 1)
    dx, dgu = torch.empty(1, 128, device="cuda"), torch.empty(1, 2 * F, device="cuda")
    pq2.pq2_mx4_gated_grad(torch.ones(1, F, device="cuda"), gu, *w, dx, dgu=dgu, act=act)
    a, s = mx4.act(act, g.double().numpy())
    # far out the functions are 0, 1 and g to the last bit
    for got, want in ((dgu[0, :F], s), (dgu[0, F:], a)):
        want = torch.from_numpy(np.nan_to_num(want, nan=0.0))
        assert ((got.cpu().double() - want).abs() <= 2.0 ** -20 * want.abs() + 2.0 ** -30).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """dx of float32 against central differences of the forward formula in
    float64, along random directions: of step t = 2^-10, the error is t^2 / 6
    times a third derivative of order ten, beside the kernel's own of about
    1e-5, on results of order one to a hundred."""
    M, F, K, t = 6, 96, 256, 2.0 ** -10
    w = weights(2 * F, K, 7)
    v = decoded(*w) / 8
    w[1].sub_(3)
    g = torch.Generator(device="cuda").manual_seed(3)
    a, dh = (torch.randn(M, n, device="cuda", generator=g) for n in (K, F))

    def loss(x):
        gu = x @ v.t()
        h = torch.from_numpy(mx4.act(act, gu[:, :F].cpu().numpy())[0]).cuda() * gu[:, F:]
        return (h * dh.double()).sum(1)

    gu = (a.double() @ v.t()).float()
    dx = torch.empty(M, K, device="cuda")
    pq2.pq2_mx4_gated_grad(dh, gu, *w, dx, act=act)
    for _ in range(8):
        e = torch.randn(M, K, device="cuda", generator=g, dtype=torch.float64)
        e /= e.norm(dim=1, keepdim=True)
        slope = (loss(a.double() + t * e) - loss(a.double() - t * e)) / (2 * t)
        got = (dx.double() * e).sum(1)
        scale = dx.double().norm(dim=1)
        assert ((got - slope).abs() <= 1e-4 * scale + 1e-4).all()


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 5120, 2048), (16, 5120, 5120), (300, 1411, 896), (4096, 520, 4096)])
def test_workspaces_of_every_size_and_repeats(M, N, K, ty):
    w, dy = weights(N, K, 2), randn(M, N, ty, 1)
    want, bound = product(dy, decoded(*w), ty)
    most = pq2.mx4_grad_workspace_bytes(M, N, K, TYPES[ty])
    least = 0 if ty == "bf16" and N % 8 == 0 else (PARTS[ty] * M * ((N + 63) // 64 * 64) * 2 + 255) // 256 * 256
    assert most >= least
    for n in sorted({least, least + 16, (least + most) // 2, most - 1, most, 2 * most + 64}):
        if n < least:
            continue
        work = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")[:n]
        dx, again = (torch.empty(M, K, dtype=TYPES[ty], device="cuda") for _ in range(2))
        pq2.pq2_mx4_gemm_grad(dy, *w, dx, workspace=work if n else None)
        check(dx, want, bound, ty)
        pq2.pq2_mx4_gemm_grad(dy, *w, again, workspace=work if n else None)
        assert torch.equal(dx, again)
    if least:
        with pytest.raises(pq2.PQ2Error, match="SCRATCH"):
            pq2.pq2_mx4_gemm_grad(dy, *w, dx, workspace=torch.empty(least - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("M,F,K", [(1, 1024, 2048), (70, 200, 640)])
def test_streams_and_graph_replays(M, F, K, ty):
    w = weights(2 * F, K, 2)
    dhs, gus = [randn(M, F, ty, i) for i in range(2)], [randn(M, 2 * F, ty, 5 + i) for i in range(2)]
    want = []
    for dh, gu in zip(dhs, gus):
        dx, dgu = torch.empty(M, K, dtype=TYPES[ty], device="cuda"), torch.empty_like(gu)
        pq2.pq2_mx4_gated_grad(dh, gu, *w, dx, dgu=dgu)
        want.append((dx, dgu))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(t) for t in want[0]] for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            pq2.pq2_mx4_gated_grad(dhs[i], gus[i], *w, outs[i][0], dgu=outs[i][1], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])
    dh, gu, dx, dgu = dhs[0].clone(), gus[0].clone(), outs[0][0], outs[0][1]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pq2.pq2_mx4_gated_grad(dh, gu, *w, dx, dgu=dgu)
    for i in (1, 0, 1):
        dh.copy_(dhs[i]), gu.copy_(gus[i]), dx.fill_(7), dgu.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, want[i][0]) and torch.equal(dgu, want[i][1])


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 64])
def test_weights_past_4_gib(M):
    N, K = 2 ** 20 + 300, 2 ** 13 + 128
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    at = [0, 5, N // 2, N - 17, N - 1]
    rows = weights(len(at), K, 3, flat=True)
    codes[at] = rows[0]
    dy = torch.randint(-4, 5, (M, N), device="cuda").to(torch.bfloat16)
    dx = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    pq2.pq2_mx4_gemm_grad(dy, codes, scales, dx)
    want = dy[:, at].double() @ decoded(*rows)
    assert torch.equal(dx, want.float().to(torch.bfloat16))


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["bf16", "f32"])
def test_rows_past_4_gib(ty):
    M, N, K = (2 ** 20 + 77, 2 ** 12, 128) if ty == "bf16" else (2 ** 18 + 77, 2 ** 12 + 4, 128)
    w = weights(N, K, 3, flat=True)
    dy = torch.zeros(M, N, dtype=TYPES[ty], device="cuda")
    at = [0, 255, M // 2, M - 2, M - 1]
    dy[at] = torch.randint(-4, 5, (len(at), N), device="cuda").to(TYPES[ty])
    dx = torch.full((M, K), 7.0, dtype=TYPES[ty], device="cuda")
    pq2.pq2_mx4_gemm_grad(dy, *w, dx)
    assert torch.equal(dx[at], (dy[at].double() @ decoded(*w)).float().to(TYPES[ty]))
    assert torch.count_nonzero(dx) <= len(at) * K


@pytest.mark.gpu
def test_outputs_aligned_like_their_elements():
    for ty in ("f32", "bf16"):
        for M in (3, 3100):
            w, dy = weights(64, 4096, 1, flat=True), torch.ones(M, 64, dtype=TYPES[ty], device="cuda")
            buf = torch.full((M * 4096 + 9,), 7.0, dtype=TYPES[ty], device="cuda")
            dx = buf[1:1 + M * 4096].view(M, 4096)
            pq2.pq2_mx4_gemm_grad(dy, *w, dx)
            assert torch.equal(dx, (dy.double() @ decoded(*w)).float().to(TYPES[ty]))
            assert buf[0] == 7 and (buf[1 + M * 4096:] == 7).all()


@pytest.mark.gpu
def test_no_rows():
    w = weights(64, 128, 1)
    e = lambda n: torch.empty(0, n, device="cuda")  # noqa: E731
    pq2.pq2_mx4_gemm_grad(e(64), *w, e(128))
    pq2.pq2_mx4_gated_grad(e(32), e(64), *w, e(128), dgu=e(64))


@pytest.mark.gpu
def test_binding_checks_on_the_gpu():
    w = weights(6, 128, 2)
    dy, dx = torch.empty(2, 6, device="cuda"), torch.empty(2, 128, device="cuda")
    with pytest.raises(TypeError, match="dx must be"):
        pq2.pq2_mx4_gemm_grad(dy, *w, dx.half())
    with pytest.raises(ValueError, match="w must have 5 rows"):
        pq2.pq2_mx4_gemm_grad(dy[:, :5].contiguous(), *w, dx)
    with pytest.raises(ValueError, match="w must have 12 rows"):
        pq2.pq2_mx4_gated_grad(dy, torch.empty(2, 12, device="cuda"), *w, dx)
    with pytest.raises(ValueError, match="gu must have shape"):
        pq2.pq2_mx4_gated_grad(dy[:, :3].contiguous(), dy[:, :5].contiguous(), *w, dx)
    with pytest.raises(ValueError, match="act must be one of"):
        pq2.pq2_mx4_gated_grad(dy[:, :3].contiguous(), dy, *w, dx, act="relu")
