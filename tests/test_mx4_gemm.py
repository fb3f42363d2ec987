"""pq2_mx4_gemm and pq2_mx4_gated: products of two MX4 matrices.

The reference is float64 on the decoded values. Products of two codes and their
scales are exact in float32, and a float32 sum of K of them, in any order and
with additions that round or truncate, is within E = K 2^-23 sum|terms| of the
exact one; with all scales alike every partial sum is a multiple of a quarter
below 2^24 quarters, so there the result is exact.

The gated block's h = a(g) u adds, beside E_g and E_u of the two sums (|a'| is
below 1.2 for the three activations), the activation's own error. With an error
of at most 8 steps of 2^-23 for the exponential or complementary error function,
quotient and products together, and the function's argument known to 5 2^-24
relative, whose effect is multiplied by the condition number of the logistic
function (|z|) or of erfc (g^2 + 1), that is relative
    A = (10 + 3 max(|z|, g^2)) 2^-23.
A stored 16-bit value adds half a step of its type, and an absolute 2^-25 (half
the smallest float16) or 2^-126 covers what underflows.
"""

import numpy as np
import pytest
import torch

from oracle import mx4

pq2 = pytest.importorskip("gemm_pq2_w2a8_amd")

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}
ACTS = ("silu", "gelu", "gelu_tanh")
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_HIP, ERR_ARG, ERR_SCRATCH = range(7)
P = 0x100000
for _t, _v in HALF.items():
    assert _v == torch.finfo(TYPES[_t]).eps / 2


# ------------------------------------------------------------------ refusals (CPU)

def gemm(a=P, s=P, w=P, ws=P, y=P, fmt=0, M=1, N=1, K=128, work=None, size=0):
    return pq2.lib.pq2_mx4_gemm(a, s, w, ws, y, fmt, M, N, K, work, size, None)


def gated(a=P, s=P, w=P, ws=P, act=0, y=P, gu=None, fmt=0, hq=None, hs=None, M=1, N=1, K=128,
          work=None, size=0):
    return pq2.lib.pq2_mx4_gated(a, s, w, ws, act, y, gu, fmt, hq, hs, M, N, K, work, size, None)


@pytest.mark.parametrize("call", [gemm, gated])
@pytest.mark.parametrize("kw,want", [
    (dict(a=None), ERR_NULL), (dict(s=None), ERR_NULL), (dict(w=None), ERR_NULL),
    (dict(ws=None), ERR_NULL), (dict(y=None), ERR_NULL),
    (dict(M=-1), ERR_SHAPE), (dict(N=0), ERR_SHAPE), (dict(N=(1 << 21) + 1), ERR_SHAPE),
    (dict(K=0), ERR_SHAPE), (dict(K=64), ERR_SHAPE), (dict(K=160), ERR_SHAPE),
    (dict(K=(1 << 21) + 128), ERR_SHAPE), (dict(M=(1 << 26) + 1), ERR_SHAPE),
    (dict(M=1 << 26, N=1 << 15), ERR_SHAPE), (dict(M=1 << 26, K=1 << 15), ERR_SHAPE),
    (dict(fmt=3), ERR_ARG), (dict(fmt=-1), ERR_ARG),
    (dict(a=P + 8), ERR_ALIGN), (dict(w=P + 8), ERR_ALIGN), (dict(s=P + 2), ERR_ALIGN),
    (dict(ws=P + 1), ERR_ALIGN), (dict(y=P + 2), ERR_ALIGN), (dict(y=P + 1, fmt=1), ERR_ALIGN),
    (dict(work=P + 8, size=64), ERR_ALIGN), (dict(M=0), OK), (dict(M=0, a=None), OK),
])
def test_refusals(call, kw, want):
    assert call(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(y=None, gu=None), ERR_NULL), (dict(hq=P), ERR_NULL), (dict(hs=P), ERR_NULL),
    (dict(hq=P, hs=P, N=48), ERR_SHAPE), (dict(N=(1 << 20) + 1), ERR_SHAPE),
    (dict(N=1 << 20, K=1 << 15), ERR_SHAPE), (dict(act=3), ERR_ARG), (dict(act=-1), ERR_ARG),
    (dict(gu=P + 2), ERR_ALIGN), (dict(hq=P + 8, hs=P, N=32), ERR_ALIGN),
])
def test_refusals_of_the_gated_block(kw, want):
    assert gated(**kw) == want


def test_workspace_query():
    f = pq2.lib.pq2_mx4_workspace_bytes
    for g in (0, 1):
        assert f(0, 8, 128, g) == 0 and f(1, 0, 128, g) == 0 and f(1, 8, 100, g) == 0
    assert f(1, 1 << 21, 128, 0) >= 0 and f(1, 1 << 21, 128, 1) == 0   # too wide for a gated block


def test_binding_refusals():
    u8 = torch.zeros(2, 64, dtype=torch.uint8)
    with pytest.raises(TypeError, match="y must be float32, bfloat16 or float16"):
        pq2.pq2_mx4_gemm(u8, u8, u8, u8, u8)
    with pytest.raises(ValueError, match="GPU"):
        pq2.pq2_mx4_gemm(u8, u8, u8, u8, torch.zeros(2, 2))
    with pytest.raises(ValueError, match="act must be one of"):
        pq2.pq2_mx4_gated(u8, u8, u8, u8, torch.zeros(2, 2), act="relu")


# ------------------------------------------------------------------ GPU

class Matrix:
    """A random MX4 matrix: packed codes and scales on the GPU, float64 values there."""

    def __init__(self, rows, K, seed, spread=6, flat=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=g)
        self.scales = torch.randint(127 - spread, 128 + spread, (rows, K // 32), dtype=torch.uint8,
                                    device="cuda", generator=g)
        if flat:
            self.scales.fill_(127)
        self.refresh()

    def refresh(self):
        table = torch.tensor(np.concatenate([mx4.VALUES, -mx4.VALUES]), device="cuda")
        c = torch.stack([self.codes & 15, self.codes >> 4], -1).flatten(1).long()
        s = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), self.scales.int() - 127)
        s = torch.where(self.scales == 255, torch.nan, s)
        self.v = table[c] * s.repeat_interleave(32, 1)

    @property
    def args(self):
        return self.codes, self.scales


def product(a, w):
    """Exact sums and their bound."""
    return a.v @ w.v.t(), a.v.shape[1] * 2.0 ** -23 * (a.v.abs() @ w.v.abs().t())


def check(got, want, bound, ty):
    tol = bound + HALF[ty] * (want.abs() + bound) + TINY[ty]
    off = (got.double() - want).abs()
    worst = (off / tol).max().item()
    assert (off <= tol).all(), worst


# every tile and its edges: rows, columns, K of one step, an odd number of steps,
# a multiple of 512 (scales copied 16 bytes at a time) and not
SHAPES = [(1, 1, 128), (1, 16, 256), (2, 63, 384), (15, 64, 512), (16, 65, 640), (17, 100, 1024),
          (33, 256, 896), (63, 31, 128), (64, 512, 1536), (65, 129, 2048), (130, 300, 1152),
          (1, 5119, 640), (5, 2050, 5120), (257, 511, 512), (300, 1411, 896)]
BIG = [(2100, 6200, 640), (4096, 3083, 512), (3100, 4097, 1024)]


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SHAPES + BIG)
def test_gemm(M, N, K, ty):
    a, w = Matrix(M, K, M + K, 2), Matrix(N, K, N + K, 2)
    y = torch.full((M, N), 7.0, dtype=TYPES[ty], device="cuda")
    pq2.pq2_mx4_gemm(*a.args, *w.args, y)
    want, bound = product(a, w)
    check(y, want, bound, ty)
    none = torch.empty_like(y)
    pq2.pq2_mx4_gemm(*a.args, *w.args, none, workspace=None)
    check(none, want, bound, ty)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES + BIG + [(3, 40, 17408), (200, 5120, 17408)])
def test_gemm_exact(M, N, K):
    """All scales alike: no rounding anywhere."""
    a, w = Matrix(M, K, 3 * M + K, flat=True), Matrix(N, K, 3 * N + K, flat=True)
    y = torch.empty(M, N, device="cuda")
    pq2.pq2_mx4_gemm(*a.args, *w.args, y)
    assert torch.equal(y.double(), product(a, w)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,gated", [
    (33, 5120, 17408, False), (100, 1000, 8192, False), (130, 5120, 17408, False), (500, 5120, 17408, False),
    (1000, 5120, 6144, False), (1000, 17408, 1152, False), (4096, 4352, 8192, False), (2000, 8704, 5120, False),
    (40, 2048, 17408, True), (300, 8704, 5120, True), (1030, 2176, 8192, True), (4000, 2200, 5120, True),
    (256, 5120, 17408, True), (300, 2560, 17408, True), (1024, 1024, 17408, True), (2048, 8704, 5120, True),
    (2048, 8704, 1152, True), (1000, 8704, 5120, True)])
def test_plans_agree(M, N, K, gated):
    """Every tile, whole and split along K in any workspace: with all scales alike
    nothing is rounded, so the results are the same bits; some rows against
    float64."""
    a, w = Matrix(M, K, M, flat=True), Matrix(2 * N if gated else N, K, N, flat=True)
    w.scales -= 10                                   # the block's sums of order one
    w.refresh()
    call = pq2.pq2_mx4_gated if gated else pq2.pq2_mx4_gemm
    y, z = (torch.full((M, N), 7.0, device="cuda") for _ in range(2))
    call(*a.args, *w.args, y)
    call(*a.args, *w.args, z, workspace=None)
    assert torch.equal(y, z)
    most = pq2.mx4_workspace_bytes(M, N, K, gated)
    for n in {most // 2, most // 7} - {0}:
        call(*a.args, *w.args, z, workspace=torch.full((n,), 255, dtype=torch.uint8, device="cuda"))
        assert torch.equal(y, z)
    some = torch.tensor(sorted({0, M // 3, M // 2, M - 2, M - 1}), device="cuda")
    want = a.v[some] @ w.v.t()
    if gated:
        g, u = want[:, :N], want[:, N:]
        v = torch.from_numpy(mx4.act("silu", g.cpu().numpy())[0]).cuda() * u
        rel = torch.minimum((10 + 3 * g * g) * 2.0 ** -23, torch.ones_like(g))
        check(y[some], v, rel * v.abs(), "f32")
    else:
        assert torch.equal(y[some].double(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 20, 70, 2500])
def test_extreme_scales_and_nan_stay_where_they_are(M):
    N, K = 4112, 1152
    a, w = Matrix(M, K, 5, flat=True), Matrix(N, K, 6, flat=True)
    a.scales[M - 1], w.scales[3] = 0, 254            # 2^-127 and 2^127: products of order one
    a.scales[M // 2, 2] = 255                        # one block of one row
    w.scales[N - 1, K // 32 - 1] = 255
    w.codes[7] = 0                                   # a row of zeros, its scales the largest
    w.scales[7] = 254
    a.refresh(), w.refresh()
    y = torch.empty(M, N, device="cuda")
    pq2.pq2_mx4_gemm(*a.args, *w.args, y)
    want = a.v @ w.v.t()
    # column 3's sums of order 2^127 pass float32's range on the way; row M - 1's is of order one
    look = torch.ones_like(want, dtype=torch.bool)
    look[:M - 1, 3] = False
    assert torch.equal(torch.isnan(y)[look], torch.isnan(want)[look])
    fits = look & ~torch.isnan(want)
    # exact, but for what lies below float32's normal range
    assert ((y[fits].double() - want[fits]).abs() <= 2.0 ** -126).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("ty", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,F,K", [(1, 1, 128), (1, 32, 256), (3, 33, 384), (16, 64, 512), (17, 100, 640),
                                   (65, 200, 1024), (130, 1411, 896), (1, 5120, 1024), (2100, 3200, 640)])
def test_gated(M, F, K, ty, act):
    a, w = Matrix(M, K, M + K, 1), Matrix(2 * F, K, F + K, 1)
    w.scales -= 6                                    # sums of order one to ten
    w.refresh()
    h, gu = (torch.full((M, n), 7.0, dtype=TYPES[ty], device="cuda") for n in (F, 2 * F))
    pq2.pq2_mx4_gated(*a.args, *w.args, h, act=act, gu=gu)
    want, bound = product(a, w)
    check(gu, want, bound, ty)
    g, u, eg, eu = want[:, :F], want[:, F:], bound[:, :F], bound[:, F:]
    v = torch.from_numpy(mx4.act(act, g.cpu().numpy())[0]).cuda()
    z = torch.maximum(g.abs(), 1.6 * (g + 0.0447 * g ** 3).abs() if act == "gelu_tanh" else g.abs())
    rel = (10 + 3 * torch.maximum(z, g * g)) * 2.0 ** -23
    # the activation's relative error counts only while its value does not vanish
    own = torch.minimum(rel, torch.ones_like(rel)) * (v * u).abs()
    check(h, v * u, 1.2 * eg * (u.abs() + eu) + v.abs() * eu + own, ty)
    only = torch.empty_like(h)
    pq2.pq2_mx4_gated(*a.args, *w.args, only, act=act, workspace=None)
    check(only, v * u, 1.2 * eg * (u.abs() + eu) + v.abs() * eu + own, ty)


@pytest.mark.gpu
@pytest.mark.parametrize("M,F,K", [(1, 32, 128), (5, 160, 384), (16, 5120, 512), (70, 96, 640),
                                   (130, 1408, 896), (2100, 3200, 640)])
def test_gated_quantised(M, F, K):
    """hcodes and hscales are the quantiser's of the float32 h, bit for bit."""
    a, w = Matrix(M, K, M + K, 1), Matrix(2 * F, K, F + K, 1)
    h = torch.empty(M, F, device="cuda")
    codes, scales = (torch.full((M, F // n), 9, dtype=torch.uint8, device="cuda") for n in (2, 32))
    pq2.pq2_mx4_gated(*a.args, *w.args, h, hcodes=codes, hscales=scales)
    want = pq2.mx4_quantize(h)
    assert torch.equal(scales, want[1]) and torch.equal(codes, want[0])
    codes.zero_(), scales.zero_()
    pq2.pq2_mx4_gated(*a.args, *w.args, hcodes=codes, hscales=scales)
    assert torch.equal(scales, want[1]) and torch.equal(codes, want[0])


@pytest.mark.gpu
def test_gated_far_ends():
    """Gates far out: a(g) is 0 and g there, infinite sums give what the formula does."""
    K, F = 128, 64
    for act in ACTS:
        a, w = Matrix(4, K, 1, flat=True), Matrix(2 * F, K, 2, flat=True)
        a.scales += 12
        a.refresh()
        h = torch.empty(4, F, device="cuda")
        pq2.pq2_mx4_gated(*a.args, *w.args, h, act=act)
        g, u = (a.v @ w.v.t()).chunk(2, 1)
        assert g.abs().min() > 200 or (g.abs() < 200).sum() < 8
        far = g.abs() > 200
        want = torch.where(g > 0, g * u, 0.0)
        assert ((h.double() - want).abs() <= 2.0 ** -22 * want.abs())[far].all()


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(3, 64), (70, 127), (2100, 6200)])
def test_outputs_aligned_like_their_elements(M, N, ty):
    """An output that starts one element into its buffer; its surroundings stay."""
    a, w = Matrix(M, 256, 1, flat=True), Matrix(N, 256, 2, flat=True)
    buf = torch.full((M * N + 9,), 7.0, dtype=TYPES[ty], device="cuda")
    y = buf[1:1 + M * N].view(M, N)
    pq2.pq2_mx4_gemm(*a.args, *w.args, y)
    check(y, product(a, w)[0], torch.zeros((), device="cuda"), ty)
    assert buf[0] == 7 and (buf[1 + M * N:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 40, 2100])
def test_scales_on_a_4_byte_address(M):
    """Scales whose base is 4- but not 16-byte aligned, K a multiple of 512."""
    N, K = 4200, 1024
    a, w = Matrix(M, K, 1, flat=True), Matrix(N, K, 2, 2)
    buf = torch.empty(4 + N * (K // 32), dtype=torch.uint8, device="cuda")
    ws = buf[4:].view(N, K // 32)
    ws.copy_(w.scales)
    y, z = (torch.empty(M, N, device="cuda") for _ in range(2))
    pq2.pq2_mx4_gemm(*a.args, *w.args, y)
    pq2.pq2_mx4_gemm(*a.args, w.codes, ws, z)
    assert torch.equal(y, z)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 5120, 6144), (16, 5120, 17408), (100, 700, 2048), (4096, 5120, 2048)])
def test_workspaces_of_every_size_and_repeats(M, N, K):
    a, w = Matrix(M, K, 1, 3), Matrix(N, K, 2, 3)
    want, bound = product(a, w)
    most = pq2.mx4_workspace_bytes(M, N, K)
    for n in sorted({0, 16, most // 5, most // 2, most - 1, most, 2 * most + 64}):
        if n < 0:
            continue
        work = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")[:n]
        y = torch.empty(M, N, device="cuda")
        pq2.pq2_mx4_gemm(*a.args, *w.args, y, workspace=work if n else None)
        check(y, want, bound, "f32")
        again = torch.empty_like(y)
        pq2.pq2_mx4_gemm(*a.args, *w.args, again, workspace=work if n else None)
        assert torch.equal(y, again)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 640, 2048), (16, 5120, 6144), (300, 1411, 896)])
def test_streams_and_graph_replays(M, N, K):
    """Two products on two streams at once, and a captured one replayed with new
    contents between the program's own work."""
    a, w = Matrix(M, K, 1, flat=True), Matrix(N, K, 2, flat=True)
    b = Matrix(M, K, 3, flat=True)
    want, other = product(a, w)[0], product(b, w)[0]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    y, z = (torch.empty(M, N, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    for _ in range(10):
        pq2.pq2_mx4_gemm(*a.args, *w.args, y, stream=s1)
        pq2.pq2_mx4_gemm(*b.args, *w.args, z, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(y.double(), want) and torch.equal(z.double(), other)
    graph = torch.cuda.CUDAGraph()
    codes = a.codes.clone()
    h = torch.empty(M, N // 2, device="cuda")
    with torch.cuda.graph(graph):
        pq2.pq2_mx4_gemm(codes, a.scales, *w.args, y)
        if N % 2 == 0:
            pq2.pq2_mx4_gated(codes, a.scales, *w.args, h)
    for src, want in ((b, other), (a, want), (b, other)):
        codes.copy_(src.codes)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.double(), want)
        if N % 2 == 0:
            eager = torch.empty_like(h)
            pq2.pq2_mx4_gated(codes, a.scales, *w.args, eager)
            assert torch.equal(h, eager)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 64])
def test_weights_past_4_gib(M):
    N, K = 2 ** 20 + 300, 2 ** 13 + 128
    w = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    ws = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    at = [0, 5, N // 2, N - 17, N - 1]
    rows = Matrix(len(at), K, 3, flat=True)
    w[at] = rows.codes
    a = Matrix(M, K, 4, flat=True)
    y = torch.full((M, N), 7.0, device="cuda")
    pq2.pq2_mx4_gemm(*a.args, w, ws, y)
    assert torch.equal(y[:, at].double(), product(a, rows)[0])
    assert torch.count_nonzero(y) <= M * len(at)
    F = N // 2
    at = [0, 5, F // 2, F - 17, F - 1]
    w.zero_()
    w[at], w[[F + i for i in at]] = rows.codes, rows.codes
    h = torch.full((M, F), 7.0, dtype=torch.bfloat16, device="cuda")
    small = torch.empty(M, len(at), dtype=torch.bfloat16, device="cuda")
    pq2.pq2_mx4_gated(*a.args, w, ws, h)
    pq2.pq2_mx4_gated(*a.args, torch.cat([rows.codes, rows.codes]), torch.cat([rows.scales, rows.scales]), small)
    assert torch.equal(h[:, at], small) and torch.count_nonzero(h) <= M * len(at)


@pytest.mark.gpu
def test_tokens_and_outputs_past_4_gib():
    M, N, K = 2 ** 18 + 77, 2 ** 13 + 1, 2 ** 14 + 2 ** 12
    a = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((M, K // 32), 127, dtype=torch.uint8, device="cuda")
    at = [0, 255, M // 2, M - 2, M - 1]
    rows = Matrix(len(at), K, 3, flat=True)
    a[at] = rows.codes
    w = Matrix(N, K, 4, flat=True)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")   # 4.3 GB
    pq2.pq2_mx4_gemm(a, scales, *w.args, y)
    assert torch.equal(y[at], product(rows, w)[0].float().to(torch.bfloat16))
    assert torch.count_nonzero(y[1:255]) == 0 and torch.count_nonzero(y[M // 2 + 1:M - 2]) == 0


@pytest.mark.gpu
def test_no_rows():
    w = Matrix(64, 128, 1)
    empty = torch.empty(0, 64, dtype=torch.uint8, device="cuda"), torch.empty(0, 4, dtype=torch.uint8, device="cuda")
    pq2.pq2_mx4_gemm(*empty, *w.args, torch.empty(0, 64, device="cuda"))
    pq2.pq2_mx4_gated(*empty, *w.args, torch.empty(0, 32, device="cuda"))
    assert pq2.mx4_linear(torch.empty(0, 128, device="cuda"), *w.args).shape == (0, 64)


@pytest.mark.gpu
def test_binding_checks_on_the_gpu():
    a, w = Matrix(2, 128, 1), Matrix(6, 128, 2)
    y = torch.empty(2, 6, device="cuda")
    with pytest.raises(ValueError, match="wscale must have shape"):
        pq2.pq2_mx4_gemm(*a.args, w.codes, w.scales[:5].contiguous(), y)
    with pytest.raises(ValueError, match="w must have shape"):
        pq2.pq2_mx4_gemm(*a.args, w.codes[:, :32].contiguous(), w.scales, y)
    with pytest.raises(ValueError, match="even number of rows"):
        pq2.pq2_mx4_gated(*a.args, w.codes[:5], w.scales[:5], y)
    with pytest.raises(TypeError, match="gu must be"):
        pq2.pq2_mx4_gated(*a.args, *w.args, torch.empty(2, 3, device="cuda"), gu=y.half())
    with pytest.raises(pq2.PQ2Error, match="NULL"):
        pq2.pq2_mx4_gated(*a.args, *w.args)
    w = Matrix(80, 128, 2)                            # F = 40
    with pytest.raises(pq2.PQ2Error, match="SHAPE"):
        pq2.pq2_mx4_gated(*a.args, *w.args, hcodes=torch.empty(2, 20, dtype=torch.uint8, device="cuda"),
                          hscales=torch.empty(2, 1, dtype=torch.uint8, device="cuda"))
