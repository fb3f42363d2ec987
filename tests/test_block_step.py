"""The operators around the product together, as a decode step uses them: norm
and quantise, a projection with its requests' adapters, the next norm with the
residual, a router's choice, the experts' two products, and the norm behind
them. Every operator is held to its own bounds on the inputs it was given, and
the captured step replays to the bits of the eager one."""

import numpy as np
import pytest
import torch

pq2 = pytest.importorskip("gemm_pq2_w2a8_amd")

import pq2_synth as synth  # noqa: E402
import test_gemm_grouped as grouped  # noqa: E402
import test_lora_add as lora  # noqa: E402
import test_norm_quantize as norm  # noqa: E402

pytestmark = pytest.mark.gpu

K, E, TOP, INNER, RANK, L = 1024, 12, 3, 256, 16, 4
BF = torch.bfloat16


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    w = {"w_in": 1 + 0.1 * torch.randn(K, generator=g), "w_mid": 1 + 0.1 * torch.randn(K, generator=g),
         "w_post": 1 + 0.1 * torch.randn(K, generator=g), "w_next": 1 + 0.1 * torch.randn(K, generator=g),
         "a": (torch.randn(L, RANK, K, generator=g) / 32).to(BF),
         "b": (torch.randn(L, K, RANK, generator=g) / 4).to(BF),
         "router": torch.randn(K, E, generator=g) / 32}
    rng = np.random.default_rng(seed)
    for name, n, k in (("proj", K, K), ("up", E * 2 * INNER, K), ("down", E * K, INNER)):
        w[name] = torch.from_numpy(synth.draw_codes(n, k, rng))
        w[name + "_s"] = torch.from_numpy(synth.draw_wscale(n, k, rng) * np.float16(0.25))
    w["up"], w["up_s"] = w["up"].view(E, 2 * INNER, -1), w["up_s"].view(E, 2 * INNER, -1)
    w["down"], w["down_s"] = w["down"].view(E, K, -1), w["down_s"].view(E, K, -1)
    return {k: v.cuda() for k, v in w.items()}


def step(w, x, residual, adapter):
    """One block; returns every operator's inputs and outputs."""
    M = x.shape[0]
    o = {}
    n = torch.empty_like(x)
    q, s, t = (torch.empty(M, K, dtype=torch.int8, device="cuda"),
               torch.empty(M, K // 128, device="cuda"),
               torch.empty(M, K // 128, dtype=torch.int32, device="cuda"))
    h = torch.empty_like(x)
    pq2.pq2_norm_quantize(x, q, s, t, residual=residual, w_pre=w["w_in"], h=h, n=n)
    y = torch.empty(M, K, dtype=BF, device="cuda")
    pq2.pq2_gemm(q, s, t, w["proj"], w["proj_s"], y)
    o["proj"] = y.clone()
    pq2.pq2_lora_add(n, w["a"], w["b"], adapter, y)              # in place, beside the projection
    o.update(n=n, adapted=y, h=h)
    n2 = torch.empty_like(x)
    h2, q2, s2, t2 = (torch.empty_like(x), torch.empty_like(q), torch.empty_like(s), torch.empty_like(t))
    pq2.pq2_norm_quantize(y, q2, s2, t2, residual=h, w_pre=w["w_mid"], h=h2, n=n2)
    o.update(h2=h2, n2=n2, q2=q2, s2=s2, t2=t2)
    # the router: the TOP largest of E, slots in expert order
    p = torch.softmax(n2.float() @ w["router"], -1)
    pick_w, pick = torch.topk(p, TOP)
    expert, order = torch.sort(pick.flatten(), stable=True)
    offsets = torch.searchsorted(expert, torch.arange(E + 1, device="cuda")).to(torch.int32)
    rows = (order // TOP).to(torch.int32)
    share = pick_w.flatten()[order].contiguous()
    up = torch.empty(M * TOP, 2 * INNER, device="cuda")
    pq2.pq2_gemm_grouped(q2, s2, t2, w["up"], w["up_s"], offsets, up, rows=rows)
    act = (torch.nn.functional.silu(up[:, :INNER]) * up[:, INNER:]).contiguous()
    q3, s3, t3 = pq2.quantize_act(act)
    down = torch.empty(M * TOP, K, device="cuda")
    pq2.pq2_gemm_grouped(q3, s3, t3, w["down"], w["down_s"], offsets, down, row_scale=share)
    o.update(offsets=offsets, rows=rows, share=share, up=up, q3=q3, s3=s3, t3=t3, down=down)
    back = torch.empty_like(order)
    back[order] = torch.arange(M * TOP, device="cuda")
    block = down[back].view(M, TOP, K).sum(1).to(BF)
    q4, s4, t4, n4 = torch.empty_like(q), torch.empty_like(s), torch.empty_like(t), torch.empty_like(x)
    pq2.pq2_norm_quantize(block, q4, s4, t4, residual=h2, w_post=w["w_post"], alpha=0.5,
                          w_pre=w["w_next"], h=h2, n=n4)         # the residual stream in place
    o.update(block=block, h4=h2, n4=n4, q4=q4, s4=s4, t4=t4)
    return o


def natural(q):
    m = q.shape[0]
    return q.cpu().numpy().reshape(m, -1, 4, 32).transpose(0, 1, 3, 2).reshape(m, -1)


def check_grouped(o, w, name, q, s, t, out, rows, share):
    p = grouped.Problem.__new__(grouped.Problem)
    p.codes, p.ws = w[name].cpu().numpy(), w[name + "_s"].cpu().numpy()
    p.E, p.N, p.K = p.codes.shape[0], p.codes.shape[1], 4 * p.codes.shape[2]
    p.G = p.K // 128
    p.q, p.s, p.t = natural(q), s.cpu().numpy(), t.cpu().numpy()
    p.off, p.T = o["offsets"].cpu().numpy(), out.shape[0]
    p.rows = None if rows is None else rows.cpu().numpy()
    p.row_scale = None if share is None else share.cpu().numpy()
    p.check(out.cpu().double().numpy())


@pytest.mark.parametrize("M", [1, 7, 64])
def test_step(M):
    print(f"block step M={M}", flush=True)
    w = weights(5)
    g = torch.Generator().manual_seed(M)
    x, residual = (torch.randn(M, K, generator=g).to(BF).cuda() for _ in range(2))
    adapter = torch.randint(-1, L, (M,), generator=g).to(torch.int32).cuda()
    keep = residual.clone()
    o = step(w, x, residual, adapter)
    assert torch.equal(residual, keep)
    # the norms
    f = {"x": x.cpu(), "residual": residual.cpu(), "w_post": None, "w_pre": w["w_in"].cpu(), "gate": None}
    h, eh, n, en = norm.reference(f, 1.0)
    for got, ref, err in ((o["h"], h, eh), (o["n"], n, en)):
        got = got.cpu().double().numpy()
        assert (np.abs(got - ref) <= err + norm.half_step(BF, np.abs(ref) + err)).all()
    f = {"x": o["adapted"].cpu(), "residual": o["h"].cpu(), "w_post": None, "w_pre": w["w_mid"].cpu(),
         "gate": None}
    mid = norm.run(f, 1.0)
    norm.check(mid, f, 1.0, BF)
    norm.same({"n": o["n2"], "q": o["q2"], "s": o["s2"], "t": o["t2"]}, {k: mid[k] for k in "nqst"})
    f = {"x": o["block"].cpu(), "residual": mid["h"].cpu(), "w_post": w["w_post"].cpu(),
         "w_pre": w["w_next"].cpu(), "gate": None}
    norm.check({"h": o["h4"], "n": o["n4"], "q": o["q4"], "s": o["s4"], "t": o["t4"]}, f, 0.5, BF)
    # the adapters beside the projection
    p = lora.Problem.__new__(lora.Problem)
    p.M, p.N, p.K, p.R, p.L = M, K, K, RANK, L
    p.x, p.a, p.b, p.ids = o["n"].cpu(), w["a"].cpu(), w["b"].cpu(), adapter.cpu()
    p.ranks = p.scale = None
    p.base = p.y0 = o["proj"].cpu()
    p.check(o["adapted"].cpu())
    # the experts
    check_grouped(o, w, "up", o["q2"], o["s2"], o["t2"], o["up"], o["rows"], None)
    check_grouped(o, w, "down", o["q3"], o["s3"], o["t3"], o["down"], None, o["share"])


def test_step_in_a_graph():
    """Captured once, replayed with other activations and adapters between eager
    steps: the same bits."""
    M = 9
    w = weights(6)
    draw = lambda seed: (torch.randn(M, K, generator=torch.Generator().manual_seed(seed)).to(BF).cuda(),  # noqa: E731
                         torch.randn(M, K, generator=torch.Generator().manual_seed(seed + 50)).to(BF).cuda(),
                         (torch.arange(M) * (seed + 1) % (L + 1) - 1).to(torch.int32).cuda())
    x, residual, adapter = draw(0)
    step(w, x, residual, adapter)                                 # warm
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step(w, x, residual, adapter)
    for seed in (1, 2, 3):
        new = draw(seed)
        for dst, src in zip((x, residual, adapter), new):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        want = step(w, *new)
        torch.cuda.synchronize()
        for key in ("adapted", "n2", "q2", "up", "down", "h4", "q4", "s4", "t4"):
            assert torch.equal(o[key], want[key]), (seed, key)
