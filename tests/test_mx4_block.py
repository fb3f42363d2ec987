"""The MX4 operators together, as a feed-forward block uses them between two of
the library's norms: norm (whose rows go out unquantised), quantise, the gated
block with its own quantised output, the down product, an adapter beside it, the
next norm with the residual; then the way back for the adapter and the layers
below. Every operator is held to its own bounds on the inputs it was given, and
the captured step replays to the bits of the eager one."""

import pytest
import torch

pq2 = pytest.importorskip("gemm_pq2_w2a8_amd")

import test_mx4_gemm as forward  # noqa: E402
import test_mx4_grad as backward  # noqa: E402
from oracle import mx4  # noqa: E402

pytestmark = pytest.mark.gpu

K, F, RANK, L = 1024, 1408, 16, 3
BF = torch.bfloat16


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    w = {name: (1 + 0.1 * torch.randn(K, generator=g)).cuda() for name in ("w_in", "w_next")}
    w["a"] = (torch.randn(L, RANK, F, generator=g) / 32).to(BF).cuda()
    w["b"] = (torch.randn(L, K, RANK, generator=g) / 4).to(BF).cuda()
    w["gate_up"] = pq2.mx4_quantize((torch.randn(2 * F, K, generator=g) / K ** 0.5).cuda())
    w["down"] = pq2.mx4_quantize((torch.randn(K, F, generator=g) / F ** 0.5).cuda())
    return w


def step(w, x, residual, adapter, dy):
    M = x.shape[0]
    bf = lambda n: torch.empty(M, n, dtype=BF, device="cuda")  # noqa: E731
    o = {"n": bf(K), "h": bf(F), "gu": bf(2 * F), "y": bf(K), "r": bf(K), "r2": bf(K), "dh": bf(F),
         "dgu": bf(2 * F), "dn": bf(K)}
    pq2.pq2_norm_quantize(x, residual=residual, w_pre=w["w_in"], h=o["r"], n=o["n"])
    o["a"] = pq2.mx4_quantize(o["n"])
    hq = (torch.empty(M, F // 2, dtype=torch.uint8, device="cuda"),
          torch.empty(M, F // 32, dtype=torch.uint8, device="cuda"))
    pq2.pq2_mx4_gated(*o["a"], *w["gate_up"], o["h"], gu=o["gu"], hcodes=hq[0], hscales=hq[1])
    o["hq"] = hq
    pq2.pq2_mx4_gemm(*hq, *w["down"], o["y"])
    o["down"] = o["y"].clone()
    pq2.pq2_lora_add(o["h"], w["a"], w["b"], adapter, o["y"])
    o["q"], o["s"], o["t"] = (torch.empty(M, K, dtype=torch.int8, device="cuda"),
                              torch.empty(M, K // 128, device="cuda"),
                              torch.empty(M, K // 128, dtype=torch.int32, device="cuda"))
    pq2.pq2_norm_quantize(o["y"], o["q"], o["s"], o["t"], residual=o["r"], w_pre=w["w_next"], h=o["r2"])
    # the way back, from the gradient of the down product
    pq2.pq2_mx4_gemm_grad(dy, *w["down"], o["dh"])
    pq2.pq2_mx4_gated_grad(o["dh"], o["gu"], *w["gate_up"], o["dn"], dgu=o["dgu"])
    return o


def draw(M, seed):
    g = torch.Generator().manual_seed(seed)
    x, residual, dy = (torch.randn(M, K, generator=g).to(BF).cuda() for _ in range(3))
    return x, residual, torch.randint(-1, L, (M,), generator=g).to(torch.int32).cuda(), dy


class Given(forward.Matrix):
    """An MX4 matrix that a call made."""

    def __init__(self, codes, scales):
        self.codes, self.scales = codes, scales
        self.refresh()


@pytest.mark.parametrize("M", [1, 7, 64, 200])
def test_step(M):
    w, (x, residual, adapter, dy) = weights(5), draw(M, M)
    o = step(w, x, residual, adapter, dy)
    # the quantiser, on some rows in full
    some = [0, M // 2, M - 1]
    codes, scales = mx4.quantise(o["n"][some].float().cpu().numpy())
    assert torch.equal(o["a"][0][some].cpu(), torch.from_numpy(mx4.pack(codes)))
    assert torch.equal(o["a"][1][some].cpu(), torch.from_numpy(scales))
    # both projections and the gate
    a, gate_up, hq, down = (Given(*t) for t in (o["a"], w["gate_up"], o["hq"], w["down"]))
    gu, bound = forward.product(a, gate_up)
    forward.check(o["gu"], gu, bound, "bf16")
    g, u = gu.chunk(2, 1)
    v = torch.from_numpy(mx4.act("silu", g.cpu().numpy())[0]).cuda()
    eg, eu = bound.chunk(2, 1)
    err = 1.2 * eg * (u.abs() + eu) + v.abs() * eu + 80 * 2.0 ** -23 * (v * u).abs()
    forward.check(o["h"], v * u, err, "bf16")
    # the quantised rows: within half a step of the format (a quarter of a value
    # in [1, 2), a sixth above 6: what lies beyond is up to a quarter off) of h
    off = (hq.v - v * u).abs()
    step_ = 2.0 ** (o["hq"][1].double() - 127).repeat_interleave(32, 1)
    assert (off <= torch.maximum(0.25 * (v * u).abs(), 0.25 * step_) * (1 + 1e-5) + err).all()
    y, bound = forward.product(hq, down)
    forward.check(o["down"], y, bound, "bf16")
    # and back
    backward.check(o["dh"], *backward.product(dy, down.v, "bf16"), "bf16")
    want, bound = backward.gated_reference(o["dh"], o["gu"], "silu", "bf16")
    backward.check(o["dgu"], want, bound, "bf16")
    backward.check(o["dn"], *backward.product(o["dgu"], gate_up.v, "bf16"), "bf16")


def test_step_in_a_graph():
    """Captured once, replayed with other inputs between eager steps: the same bits."""
    w, (x, residual, adapter, dy) = weights(6), draw(9, 0)
    step(w, x, residual, adapter, dy)                             # warm
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step(w, x, residual, adapter, dy)
    for seed in (1, 2, 3):
        new = draw(9, seed)
        for dst, src in zip((x, residual, adapter, dy), new):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        want = step(w, *new)
        torch.cuda.synchronize()
        for key in ("h", "gu", "y", "q", "s", "t", "r2", "dh", "dgu", "dn"):
            assert torch.equal(o[key], want[key]), (seed, key)
