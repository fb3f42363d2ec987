"""Microscaled 4-bit floating point: the quantiser and its inverse.

Both are exact: codes and scale bytes are compared for equality with the plain
definition (oracle/mx4.py), whose own pins come first, and values with theirs
(float16 ones rounded once, to nearest even).
"""

import numpy as np
import pytest
import torch

from oracle import mx4

pq2 = pytest.importorskip("gemm_pq2_w2a8_amd")

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_HIP, ERR_ARG = 0, 1, 2, 3, 4, 5
P = 0x100000


# ------------------------------------------------------------------ pins of the definition (CPU)

def block(*first):
    """A block that starts with these values, zeros behind."""
    x = np.zeros((1, 32), np.float32)
    x[0, :len(first)] = first
    return x


def test_every_value_is_its_own_code():
    v = np.concatenate([mx4.VALUES, -mx4.VALUES[1:]]).astype(np.float32)
    codes, scales = mx4.quantise(block(*v))
    assert scales[0, 0] == 127                      # the largest is 6: 2^(2 - 2)
    assert list(codes[0, :15]) == list(range(8)) + list(range(9, 16))
    assert np.array_equal(mx4.values(codes, scales)[0, :15], v)


def test_ties_go_to_the_even_code():
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    codes, _ = mx4.quantise(block(*mids, 6.0))
    assert list(codes[0, :7]) == [0, 2, 2, 4, 4, 6, 6]
    up, down = np.nextafter(np.float32(mids), np.float32(9)), np.nextafter(np.float32(mids), np.float32(0))
    assert list(mx4.quantise(block(*up, 6.0))[0][0, :7]) == [1, 2, 3, 4, 5, 6, 7]
    assert list(mx4.quantise(block(*down, 6.0))[0][0, :7]) == [0, 1, 2, 3, 4, 5, 6]


def test_scale_is_the_largest_values_exponent():
    for e in (-130, -126, -20, 0, 1, 100, 127):
        for f in (1.0, 1.25, 1.999):
            top = np.float32(np.ldexp(f, e))
            _, scales = mx4.quantise(block(top))
            assert scales[0, 0] == max(0, e - 2 + 127)
    codes, scales = mx4.quantise(block(np.float32(7.99), -7.0))
    assert scales[0, 0] == 127 and list(codes[0, :2]) == [7, 15]     # beyond 6: 6


def test_zeros_and_what_is_not_finite():
    codes, scales = mx4.quantise(block(0.0, -0.0))
    assert scales[0, 0] == 0 and list(codes[0, :3]) == [0, 8, 0]
    for bad in (np.inf, -np.inf, np.nan):
        codes, scales = mx4.quantise(block(1.0, bad))
        assert scales[0, 0] == 255 and not codes.any()
        assert np.isnan(mx4.values(codes, scales)).all()


def test_packing():
    codes = np.arange(32, dtype=np.uint8)[None] % 16
    assert mx4.pack(codes)[0, 0] == 0x10 and np.array_equal(mx4.unpack(mx4.pack(codes)), codes)


def test_activations_of_the_definition():
    """Derivatives against differences, and values at points known in closed form."""
    g = np.linspace(-8, 8, 81)
    for name in ("silu", "gelu", "gelu_tanh"):
        a, d = mx4.act(name, g)
        h = 1e-5
        diff = (mx4.act(name, g + h)[0] - mx4.act(name, g - h)[0]) / (2 * h)
        # second-order difference: h^2 / 6 * |a'''| (< 4) and 2^-53 * 8 / h of rounding
        assert np.abs(d - diff).max() < 1e-9
        assert a[40] == 0 and abs(d[40] - 0.5) < 1e-15
    assert abs(mx4.act("silu", np.array([1.0]))[0][0] - 1 / (1 + np.exp(-1))) < 1e-15
    assert abs(mx4.act("gelu", np.array([1.0]))[0][0] - 0.8413447460685429) < 1e-15


# ------------------------------------------------------------------ refusals (CPU)

def quantize(x=P, fmt=0, codes=P, scales=P, M=1, K=32):
    return pq2.lib.pq2_mx4_quantize(x, fmt, codes, scales, M, K, None)


def dequantize(x=P, fmt=0, codes=P, scales=P, M=1, K=32):
    return pq2.lib.pq2_mx4_dequantize(codes, scales, x, fmt, M, K, None)


@pytest.mark.parametrize("call", [quantize, dequantize])
@pytest.mark.parametrize("kw,want", [
    (dict(x=None), ERR_NULL), (dict(codes=None), ERR_NULL), (dict(scales=None), ERR_NULL),
    (dict(M=-1), ERR_SHAPE), (dict(K=0), ERR_SHAPE), (dict(K=16), ERR_SHAPE), (dict(K=48), ERR_SHAPE),
    (dict(K=-32), ERR_SHAPE), (dict(K=(1 << 24) + 32), ERR_SHAPE), (dict(M=(1 << 30) + 1), ERR_SHAPE),
    (dict(M=1 << 30, K=2048), ERR_SHAPE), (dict(fmt=3), ERR_ARG), (dict(fmt=-1), ERR_ARG),
    (dict(x=P + 8), ERR_ALIGN), (dict(codes=P + 8), ERR_ALIGN),
    (dict(M=0), OK), (dict(M=0, x=None), OK),
])
def test_refusals(call, kw, want):
    assert call(**kw) == want


def test_binding_refusals():
    x = torch.zeros(2, 64)
    u8 = torch.zeros(2, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        pq2.pq2_mx4_quantize(x, u8, u8)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        pq2.pq2_mx4_quantize(x.double(), u8, u8)
    with pytest.raises(ValueError, match="2-D"):
        pq2.pq2_mx4_dequantize(u8, u8, x[0])


# ------------------------------------------------------------------ GPU

def special(M, K, ty, seed):
    """Rows with everything a block can hold: wide ranges of exponents, ties,
    zeros of both signs, subnormals, the largest values, infinities and NaN."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((M, K)).astype(np.float32)
    for m in range(M):
        for b in range(K // 32):
            v = x[m, 32 * b:32 * b + 32]
            kind = g.integers(0, 10)
            e = int(g.integers(-20, 15)) if ty == "f16" else int(g.integers(-150, 126))
            if kind < 3:
                v *= np.float32(np.ldexp(1.0, max(e, -126)))
                v *= np.float32(np.ldexp(1.0, e - max(e, -126)))
            elif kind == 3:      # ties at every border, and beyond 6
                mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 7.75, 4.0, 0, 6], np.float32)
                scale = np.float32(np.ldexp(1.0, max(-100, min(e, 100))) if ty != "f16" else 1.0)
                v[:] = g.choice(mids, 32) * g.choice(np.float32([-1, 1]), 32) * scale
                v[5] = 4 * scale
            elif kind == 4:
                v[:] = 0.0
                v[::3] = -0.0
            elif kind == 5:      # subnormals alone
                v[:] = v * np.float32(2.0 ** -24 if ty == "f16" else 2.0 ** -130)
            elif kind == 6:
                v[g.integers(0, 32)] = g.choice(np.float32([np.inf, -np.inf, np.nan]))
            elif kind == 7:      # one value far above the others
                v[g.integers(0, 32)] = np.float32(60000.0 if ty == "f16" else 3.0e38)
            elif kind == 8:
                v[:] = g.choice(np.float32([-1, 1]), 32)
    return torch.from_numpy(x).to(TYPES[ty])


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", [(1, 32), (1, 128), (3, 160), (17, 96), (2, 5120), (129, 416)])
def test_quantize(M, K, ty):
    x = special(M, K, ty, 31 * M + K)
    codes, scales = pq2.mx4_quantize(x.cuda())
    oc, os_ = mx4.quantise(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), os_)
    assert np.array_equal(codes.cpu().numpy(), mx4.pack(oc))


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["f32", "bf16", "f16"])
def test_dequantize_everything(ty):
    """All 16 codes under all 256 scale bytes."""
    codes = np.tile(np.arange(32, dtype=np.uint8) % 16, (256, 3))
    codes[:, 40:] = codes[:, 40:][:, ::-1]
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 3, 1)
    scales[:, 1] = scales[::-1, 1]
    x = torch.empty(256, 96, dtype=TYPES[ty], device="cuda")
    pq2.pq2_mx4_dequantize(torch.from_numpy(mx4.pack(codes)).cuda(), torch.from_numpy(scales).cuda(), x)
    want = torch.from_numpy(mx4.values(codes, scales)).to(TYPES[ty])   # exact, or rounded once
    assert torch.equal(torch.isnan(x.cpu()), torch.isnan(want))
    same = (x.cpu() == want) | torch.isnan(want)
    assert same.all()
    assert torch.equal(torch.signbit(x.cpu())[~torch.isnan(want)], torch.signbit(want)[~torch.isnan(want)])


@pytest.mark.gpu
@pytest.mark.parametrize("ty", ["f32", "bf16", "f16"])
def test_quantizing_values_of_the_format_gives_them_back(ty):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(67, 1024, generator=g).to(TYPES[ty]).cuda()
    codes, scales = pq2.mx4_quantize(x)
    v = torch.empty_like(x)
    pq2.pq2_mx4_dequantize(codes, scales, v)
    again = pq2.mx4_quantize(v)
    assert torch.equal(again[0], codes) and torch.equal(again[1], scales)


@pytest.mark.gpu
def test_empty():
    x = torch.empty(0, 64, device="cuda")
    codes, scales = pq2.mx4_quantize(x)
    pq2.pq2_mx4_dequantize(codes, scales, x)
    assert codes.shape == (0, 32) and scales.shape == (0, 2)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """More than 2^32 bytes of input and 2^32 values: the last rows are theirs."""
    M, K = 2 ** 16 + 5, 2 ** 16 + 32
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, M // 2, M - 2, M - 1]
    rows = torch.randn(len(at), K, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[at] = rows.cuda()
    codes, scales = pq2.mx4_quantize(x)
    want = pq2.mx4_quantize(rows.cuda())
    assert torch.equal(codes[at], want[0]) and torch.equal(scales[at], want[1])
    x.fill_(7.0)
    pq2.pq2_mx4_dequantize(codes, scales, x)
    v = torch.empty(len(at), K, dtype=torch.bfloat16, device="cuda")
    pq2.pq2_mx4_dequantize(*want, v)
    assert torch.equal(x[at], v) and not x[2:M // 2].any()


@pytest.mark.gpu
def test_streams_and_graph_replays():
    x = torch.randn(33, 640, device="cuda")
    side = torch.cuda.Stream()
    codes, scales, v = (torch.empty(33, 320, dtype=torch.uint8, device="cuda"),
                        torch.empty(33, 20, dtype=torch.uint8, device="cuda"), torch.empty_like(x))
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pq2.pq2_mx4_quantize(x, codes, scales)
        pq2.pq2_mx4_dequantize(codes, scales, v)
    for seed in range(3):
        x.copy_(torch.randn(33, 640, generator=torch.Generator().manual_seed(seed)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = pq2.mx4_quantize(x, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
        assert torch.equal(v.cpu().double(), torch.from_numpy(mx4.values(
            mx4.unpack(codes.cpu().numpy()), scales.cpu().numpy())))


@pytest.mark.gpu
def test_binding_checks_on_the_gpu():
    x = torch.zeros(2, 64, device="cuda")
    codes = torch.zeros(2, 32, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(2, 2, dtype=torch.uint8, device="cuda")
    pq2.pq2_mx4_quantize(x, codes, scales)
    with pytest.raises(ValueError, match="codes must have shape"):
        pq2.pq2_mx4_quantize(x, codes[:1], scales)
    with pytest.raises(ValueError, match="contiguous"):
        pq2.pq2_mx4_quantize(torch.zeros(64, 2, device="cuda").t(), codes, scales)
    with pytest.raises(TypeError, match="scales must be"):
        pq2.pq2_mx4_quantize(x, codes, scales.to(torch.int8))
    with pytest.raises(pq2.PQ2Error):
        pq2.pq2_mx4_quantize(torch.zeros(2, 48, device="cuda"), codes[:, :24].contiguous(), scales[:, :1].contiguous())
