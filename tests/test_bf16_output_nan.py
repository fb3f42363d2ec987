"""bfloat16 outputs of NaN sums: a weight scale or a row scale that is not a number
(whatever its payload: 0x7fff and 0xffff bits carry out of a rounding done as an
integer addition) gives NaN in bfloat16 y exactly where float32 y is NaN, and every
other output is the float32 one rounded to nearest even, bit for bit."""

import numpy as np
import pytest
import torch

import pq2_synth as synth

pq2 = pytest.importorskip("gemm_pq2_w2a8_amd")

pytestmark = pytest.mark.gpu

NAN16 = (0x7FFF, 0xFFFF, 0x7E00, 0xFE00, 0x7C01)              # binary16 NaN patterns
NAN32 = (0x7FFFFFFF, 0xFFFFFFFF, 0x7FC00000, 0xFFFF8000, 0x7FFFE000)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def compare(y32, y16, expect):
    """expect: the outputs that are NaN."""
    torch.cuda.synchronize()
    y32, y16, expect = y32.cpu(), y16.cpu(), torch.from_numpy(expect)
    assert torch.equal(torch.isnan(y32), expect)
    assert torch.equal(torch.isnan(y16), expect)
    got, want = y16.view(torch.int16), y32.to(torch.bfloat16).view(torch.int16)
    assert torch.equal(got[~expect], want[~expect])


# the GEMV (plain and persistent), panel with and without split K, token tiles, tiled, ring
# and wide kernels
@pytest.mark.parametrize("M,N,K", [(1, 300, 2048), (2, 5120, 6144), (4, 520, 2048), (5, 70, 2304),
                                   (16, 300, 17408), (40, 200, 2048), (130, 260, 1024),
                                   (256, 8192, 1024), (300, 129, 640), (1100, 17408, 1024)])
def test_gemm(M, N, K):
    print(f"bf16 NaN gemm M={M} N={N} K={K} path={pq2.gemm_kernel_path(M, N, K)}", flush=True)
    x = synth.activations(M, K, M + N, outlier_frac=0.01)
    w = synth.weights(N, K, synth.matrix_seed(N))
    bits = np.array(w.wscale_bits.view(np.uint16))
    at = np.arange(3, N, 11)
    bits[at, at % (K // 128)] = np.array(NAN16, np.uint16)[at % len(NAN16)]
    q, s, t = pq2.quantize_act(dev(x))
    cd, wd = dev(w.codes), dev(bits.view(np.int16))
    y32 = torch.empty((M, N), dtype=torch.float32, device="cuda")
    y16 = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    pq2.pq2_gemm(q, s, t, cd, wd, y32)
    pq2.pq2_gemm(q, s, t, cd, wd, y16)
    expect = np.zeros((M, N), bool)
    expect[:, at] = True
    compare(y32, y16, expect)


# the stream kernel, ring, wide and staged tiles
@pytest.mark.parametrize("counts,N,K", [([3, 0, 1], 50, 384), ([9, 7], 70, 1024),
                                        ([200, 90], 300, 1024), ([60, 3, 9], 70, 896)])
@pytest.mark.parametrize("where", ["row_scale", "wscale"])
def test_grouped(where, counts, N, K):
    print(f"bf16 NaN grouped {counts} N={N} K={K} {where}", flush=True)
    E, T = len(counts), sum(counts)
    x = synth.activations(T, K, T, outlier_frac=0.0)
    w = synth.weights(E * N, K, synth.matrix_seed(N))
    bits = np.array(w.wscale_bits.view(np.uint16)).reshape(E, N, K // 128)
    scale = np.linspace(0.5, 1.5, T).astype(np.float32)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    expect = np.zeros((T, N), bool)
    if where == "row_scale":
        at = np.arange(0, T, 2)
        scale.view(np.uint32)[at] = np.array(NAN32, np.uint32)[at % len(NAN32)]
        expect[at] = True
    else:
        for e in range(E):
            at = np.arange(e, N, 5)
            bits[e, at, at % (K // 128)] = np.array(NAN16, np.uint16)[at % len(NAN16)]
            expect[off[e]:off[e + 1], at] = True
    q, s, t = pq2.quantize_act(dev(x))
    args = (q, s, t, dev(w.codes.reshape(E, N, K // 4)), dev(bits.view(np.int16)), dev(off))
    y32 = torch.empty((T, N), dtype=torch.float32, device="cuda")
    y16 = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    for y in (y32, y16):
        pq2.pq2_gemm_grouped(*args, y, row_scale=dev(scale))
    compare(y32, y16, expect)
