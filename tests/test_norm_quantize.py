"""pq2_norm_quantize: the norms after and before a block with its gate and
residual scale, ending in the quantiser.

The reference is float64 (numpy). Bounds, with u = 2^-24 and every operation
rounded once:

* a sum of squares adds at most 16 * 4 terms per thread, 6 exchange steps and
  16 waves, all positive: relative error at most 86 u for every K tested, so
  the norm's scale (a square root, a division, a product) is within 51 u;
* the block's part b = alpha * gate * rms(x) * w_post is then within 56 u of
  its magnitude and h within E_h = 56 u |b| + 2 u |h|;
* n = h * scale * w_pre: |scale * w_pre| E_h, the scale's own 51 u and what h's
  errors do to its mean square (at most norm(E_h) / norm(h)), two products.

A stored 16-bit value adds half a step of its type. The integers are checked
through the exact quotient: q is a nearest integer of n / s up to the quotient's
own error. Bit for bit: float32 rows quantise as pq2_quantize_act's rule does on
the n that is returned, 16-bit rows as the widened rows do in float32.
"""

import ctypes

import numpy as np
import pytest
import torch

import oracle

pq2 = pytest.importorskip("gemm_pq2_w2a8_amd")

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_HIP, ERR_ARG = 0, 1, 2, 3, 4, 5
P = 0x100000


# ------------------------------------------------------------------ refusals (CPU)

def call(x=P, fmt=0, residual=None, w_post=None, gate=None, gate_rows=0, alpha=1.0, w_pre=P,
         eps=EPS, h=None, n=None, q=P, s=P, t=P, M=0, K=128):
    """The C entry with fake addresses; M = 0 is refused after every check that
    comes before the shape's, so nothing here can launch."""
    return pq2.lib.pq2_norm_quantize(x, fmt, residual, w_post, gate, gate_rows, alpha, w_pre, eps,
                                     h, n, q, s, t, M, K, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), ERR_NULL), (dict(s=None), ERR_NULL), (dict(t=None), ERR_NULL),
    (dict(q=None), ERR_NULL), (dict(q=None, s=None, t=None), ERR_NULL),
    (dict(M=0), ERR_SHAPE), (dict(M=-1), ERR_SHAPE), (dict(M=1, K=64), ERR_SHAPE),
    (dict(M=1, K=0), ERR_SHAPE), (dict(M=1, K=(1 << 24) + 128), ERR_SHAPE),
    (dict(M=(1 << 30) + 1), ERR_SHAPE), (dict(M=1 << 20, K=1 << 21), ERR_SHAPE),
    (dict(M=4, gate=P, gate_rows=0), ERR_SHAPE), (dict(M=4, gate=P, gate_rows=3), ERR_SHAPE),
    (dict(M=4, gate=P, gate_rows=-1), ERR_SHAPE), (dict(M=4, gate_rows=1), ERR_SHAPE),
    (dict(M=1, x=P + 8), ERR_ALIGN), (dict(M=1, residual=P + 8), ERR_ALIGN),
    (dict(M=1, w_post=P + 4), ERR_ALIGN), (dict(M=1, w_pre=P + 8), ERR_ALIGN),
    (dict(M=1, gate=P + 8, gate_rows=1), ERR_ALIGN), (dict(M=1, h=P + 2), ERR_ALIGN),
    (dict(M=1, n=P + 2), ERR_ALIGN), (dict(M=1, q=P + 8), ERR_ALIGN),
    (dict(M=1, s=P + 2), ERR_ALIGN), (dict(M=1, t=P + 1), ERR_ALIGN),
    (dict(M=1, fmt=3), ERR_ARG), (dict(M=1, fmt=-1), ERR_ARG),
    (dict(M=1, eps=0.0), ERR_ARG), (dict(M=1, eps=-1.0), ERR_ARG),
    (dict(M=1, eps=float("nan")), ERR_ARG), (dict(M=1, eps=float("inf")), ERR_ARG),
    (dict(M=1, alpha=float("nan")), ERR_ARG), (dict(M=1, alpha=float("-inf")), ERR_ARG),
])
def test_refusals(kw, want):
    assert call(**kw) == want


def test_binding_refusals():
    x = torch.zeros(2, 128)
    with pytest.raises(ValueError):
        pq2.norm_quantize(x)                                  # not on a GPU
    with pytest.raises(TypeError):
        pq2.norm_quantize(x.double())
    with pytest.raises(TypeError):
        pq2.norm_quantize("x")
    with pytest.raises(ValueError):
        pq2.pq2_norm_quantize(torch.zeros(2, 2, 128))


class Elsewhere(torch.Tensor):
    """A tensor that says it is on another GPU (no such GPU is needed to ask)."""
    get_device = lambda self: 1                      # noqa: E731
    is_cuda, device = True, torch.device("cuda:1")


def test_binding_refuses_another_device():
    """Tensors of one call share a GPU, and the launch is made on theirs."""
    other = torch.zeros(2, 128).as_subclass(Elsewhere)
    assert pq2._ptr(other, "x", torch.float32, (2, 128), 1) == other.data_ptr()
    with pytest.raises(ValueError, match="residual must be on cuda:0, got cuda:1"):
        pq2._ptr(other, "residual", torch.float32, (2, 128), 0)
    with pytest.raises(ValueError, match="GPU"):
        pq2._gpu(torch.zeros(2, 128), "x")


def test_launch_is_on_the_tensors_device(monkeypatch):
    seen = []

    class On:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            seen.append(("enter", self.index))

        def __exit__(self, *_):
            seen.append("exit")

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", On)
    call = lambda *a: seen.append(a) or 0            # noqa: E731
    pq2._launch(0, None, call, 1, 2)
    pq2._launch(1, None, call, 3)
    pq2._launch(1, 55, call, 4)
    assert seen == [(1, 2, 100), ("enter", 1), (3, 101), "exit", ("enter", 1), (4, 55), "exit"]
    with pytest.raises(pq2.PQ2Error):
        pq2._launch(0, None, lambda *a: ERR_ARG)


# ------------------------------------------------------------------ reference

def inputs(M, K, ty, seed, post, pre, gate, residual):
    g = torch.Generator().manual_seed(seed)
    f = {}
    x = torch.randn(M, K, generator=g)
    x[torch.rand(M, K, generator=g) < 0.01] *= 10
    f["x"] = x.to(ty)
    f["residual"] = (2 * torch.randn(M, K, generator=g)).to(ty) if residual else None
    f["w_post"] = 1 + 0.2 * torch.randn(K, generator=g) if post else None
    f["w_pre"] = 1 + 0.2 * torch.randn(K, generator=g) if pre else None
    f["gate"] = torch.randn(gate, K, generator=g).to(ty) if gate else None
    return f


def reference(f, alpha):
    """float64 h and n and the bounds of their float32 evaluation."""
    a = {k: None if v is None else v.double().numpy() for k, v in f.items()}
    alpha = float(np.float32(alpha))
    x = a["x"]
    M = x.shape[0]
    b = x
    if a["w_post"] is not None:
        b = x / np.sqrt((x ** 2).mean(1, keepdims=True) + EPS) * a["w_post"]
    if a["gate"] is not None:
        b = b * np.repeat(a["gate"], M // a["gate"].shape[0], 0)
    b = alpha * b
    h = b if a["residual"] is None else a["residual"] + b
    eh = 56 * U * np.abs(b) + 2 * U * np.abs(h)
    n, en = h, eh
    if a["w_pre"] is not None:
        sc = 1 / np.sqrt((h ** 2).mean(1, keepdims=True) + EPS)
        n = h * sc * a["w_pre"]
        norm = np.maximum(np.linalg.norm(h, axis=1, keepdims=True), 1e-300)
        en = np.abs(sc * a["w_pre"]) * eh + np.abs(n) * (
            55 * U + np.linalg.norm(eh, axis=1, keepdims=True) / norm)
    return h, eh, n, en


def half_step(ty, v):
    """Half a step of a 16-bit type at v (of its smallest value for tiny v)."""
    if ty == torch.float32:
        return np.zeros_like(v)
    fi = torch.finfo(ty)
    return np.maximum(np.abs(v) * fi.eps / 2 * (1 + 64 * U), fi.tiny * fi.eps / 2)


def check(out, f, alpha, ty):
    h64, eh, n64, en = reference(f, alpha)
    M, K = h64.shape
    for key, ref, err in (("h", h64, eh), ("n", n64, en)):
        got = out[key].cpu().double().numpy()
        bad = np.abs(got - ref) > err + half_step(ty, np.abs(ref) + err) + 1e-37
        assert not bad.any(), (key, np.abs(got - ref).max())
    q = out["q"].cpu().numpy().reshape(M, -1, 4, 32).transpose(0, 1, 3, 2).reshape(M, -1, 128)
    s, t = out["s"].cpu().double().numpy(), out["t"].cpu().numpy()
    np.testing.assert_array_equal(q.astype(np.int64).sum(-1), t)
    parts, errs = n64.reshape(M, -1, 128), en.reshape(M, -1, 128)
    s64 = np.abs(parts).max(-1) / 127
    es = errs.max(-1) / 127 + U * s64 + 1e-45
    assert (np.abs(s - s64) <= es).all()
    live = s > 1e-30
    v = parts / np.where(live, s, 1.0)[..., None]
    slack = 0.5 + errs / np.where(live, s, 1.0)[..., None] + 128 * U
    assert (np.abs(q - v) <= slack)[live].all()
    assert np.abs(q.astype(int)).max() <= 127
    assert (q[s == 0] == 0).all()


def run(f, alpha, dev="cuda", **kw):
    d = {k: None if v is None else v.to(dev) for k, v in f.items()}
    M, K = f["x"].shape
    out = {"h": torch.empty_like(d["x"]), "n": torch.empty_like(d["x"]),
           "q": torch.empty(M, K, dtype=torch.int8, device=dev),
           "s": torch.empty(M, K // 128, device=dev),
           "t": torch.empty(M, K // 128, dtype=torch.int32, device=dev)}
    x = d.pop("x")
    pq2.pq2_norm_quantize(x, out["q"], out["s"], out["t"], alpha=alpha, eps=EPS, h=out["h"],
                          n=out["n"], **d, **kw)
    return out


def same(a, b):
    for k in a:
        assert torch.equal(a[k], b[k]), k


# M, K, post, pre, gate rows, residual, alpha
SHAPES = [
    (1, 128, True, True, 1, True, 1.0),
    (1, 5120, False, True, 0, True, 1.0),
    (7, 5120, True, True, 7, True, 0.25),
    (6, 640, True, True, 2, True, -1.5),
    (16, 6144, True, False, 1, True, 0.5),
    (3, 1408, False, False, 0, True, 1.0),
    (5, 384, False, True, 5, False, 2.0),
    (4, 256, True, True, 0, False, 0.1),
    (3, 16384, True, True, 3, True, 1.0),      # 1024 threads, one group per slot
    (3, 16512, True, True, 1, True, 1.0),      # two groups per slot
    (2, 17408, False, True, 2, True, 1.0),
    (2, 32768, True, True, 2, True, 0.7),
    (3, 32896, True, True, 3, True, 0.7),      # rows read again per sweep
    (2, 65536, False, True, 0, True, 1.0),
    (2, 33024, True, False, 1, False, 1.0),
    (300, 768, True, True, 100, True, 1.0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:2])))
def test_against_float64(shape, ty):
    M, K, post, pre, gate, residual, alpha = shape
    print(f"norm_quantize {shape} {ty}", flush=True)
    f = inputs(M, K, TYPES[ty], 17 + K, post, pre, gate, residual)
    out = run(f, alpha)
    check(out, f, alpha, TYPES[ty])
    if ty == "f32":       # the quantiser's rule on the n returned, bit for bit
        qo, so, to = oracle.quantize(out["n"].cpu().numpy())
        np.testing.assert_array_equal(out["q"].cpu().numpy(), oracle.plane_order(qo))
        np.testing.assert_array_equal(out["s"].cpu().numpy().view(np.uint32), so.view(np.uint32))
        np.testing.assert_array_equal(out["t"].cpu().numpy(), to)
    else:                 # the widened rows' results, rounded once
        wide = {k: None if v is None else v.float() for k, v in f.items()}
        ref = run(wide, alpha)
        ref["h"], ref["n"] = ref["h"].to(TYPES[ty]), ref["n"].to(TYPES[ty])
        same(out, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("ty", list(TYPES))
def test_outputs_are_optional_and_in_place(ty):
    """Each output alone is what it is among the others; h over residual or x."""
    M, K = 5, 1280
    f = inputs(M, K, TYPES[ty], 3, True, True, 5, True)
    full = run(f, 0.5)
    d = {k: v.cuda() for k, v in f.items()}
    x = d.pop("x")
    h = torch.empty_like(x)
    pq2.pq2_norm_quantize(x, alpha=0.5, eps=EPS, h=h, **d)
    assert torch.equal(h, full["h"])
    n = torch.empty_like(x)
    pq2.pq2_norm_quantize(x, alpha=0.5, eps=EPS, n=n, **d)
    assert torch.equal(n, full["n"])
    q, s, t = (torch.empty_like(full[k]) for k in "qst")
    pq2.pq2_norm_quantize(x, q, s, t, alpha=0.5, eps=EPS, **d)
    same({"q": q, "s": s, "t": t}, {k: full[k] for k in "qst"})
    for target in ("residual", "x"):
        e = {k: v.cuda() for k, v in f.items()}
        q.zero_()
        pq2.pq2_norm_quantize(e["x"], q, s, t, residual=e["residual"], w_post=e["w_post"],
                              w_pre=e["w_pre"], gate=e["gate"], alpha=0.5, eps=EPS, h=e[target])
        same({"h": e[target], "q": q, "s": s, "t": t}, {k: full[k] for k in "hqst"})
    hh, qq, ss, tt = pq2.norm_quantize(x, alpha=0.5, eps=EPS, **d)
    same({"h": hh, "q": qq, "s": ss, "t": tt}, {k: full[k] for k in "hqst"})


@pytest.mark.gpu
@pytest.mark.parametrize("K", [640, 17408, 32896])
def test_in_place_long_rows(K):
    f = inputs(3, K, torch.bfloat16, 5, True, True, 1, True)
    full = run(f, 1.0)
    for target in ("residual", "x"):
        d = {k: v.cuda() for k, v in f.items()}
        q = torch.empty_like(full["q"])
        s, t = torch.empty_like(full["s"]), torch.empty_like(full["t"])
        pq2.pq2_norm_quantize(d["x"], q, s, t, residual=d["residual"], w_post=d["w_post"],
                              w_pre=d["w_pre"], gate=d["gate"], alpha=1.0, eps=EPS, h=d[target])
        same({"h": d[target], "q": q, "s": s, "t": t}, {k: full[k] for k in "hqst"})


@pytest.mark.gpu
@pytest.mark.parametrize("K", [512, 5120, 20480, 33024])
def test_rows_do_not_depend_on_each_other(K):
    """A row's bits are the same alone and in a batch, and a row of NaN or of
    zeros leaves its neighbours as they were."""
    f = inputs(6, K, torch.float32, 9, True, True, 6, True)
    whole = run(f, 0.5)
    for m in (0, 4):
        one = {k: v[m:m + 1] if v is not None and v.dim() == 2 else v for k, v in f.items()}
        got = run(one, 0.5)
        same({k: got[k][0] for k in got}, {k: whole[k][m] for k in whole})
    g = {k: v.clone() for k, v in f.items()}
    g["x"][2] = float("nan")
    g["x"][3] = 0
    g["residual"][3] = 0
    got = run(g, 0.5)
    for m in (0, 1, 4, 5):
        same({k: got[k][m] for k in got}, {k: whole[k][m] for k in whole})
    for k in ("h", "n", "q", "s", "t"):          # eps keeps a row of zeros at zero
        assert not got[k][3].any()
    assert torch.isnan(got["h"][2]).all()


@pytest.mark.gpu
def test_extremes_of_the_types():
    """Rows at the ends of the types' ranges: tiny rows (eps decides), the
    largest float16 values, a group that underflows to scale zero."""
    K = 512
    f = {"x": torch.full((4, K), 1e-7), "residual": None, "w_post": None, "gate": None,
         "w_pre": torch.ones(K)}
    f["x"][1, :128] = 65504.0
    f["x"][2] = torch.linspace(-60000, 60000, K)
    f["x"][3, 128:] = 0
    for ty in (torch.float16, torch.float32):
        g = {k: v.to(ty) if k == "x" else v for k, v in f.items()}
        check(run(g, 1.0), g, 1.0, ty)
    f["w_pre"][:128] = 1e-44          # n / 127 underflows in the first group
    out = run(f, 1.0)
    assert (out["s"][:, 0] == 0).all() and not out["q"][:, :128].any()
    assert (out["s"][2, 1:] > 0).all() and (out["s"][3] == 0).all()


@pytest.mark.gpu
def test_streams_and_graph_replays():
    """Another stream by argument; captured once and replayed with new inputs."""
    f = inputs(4, 2560, torch.bfloat16, 21, True, True, 4, True)
    want = run(f, 0.5)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = run(f, 0.5, stream=st)
    torch.cuda.synchronize()
    same(got, want)
    d = {k: v.cuda() for k, v in f.items()}
    out = {k: torch.zeros_like(v) for k, v in want.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pq2.pq2_norm_quantize(d["x"], out["q"], out["s"], out["t"], residual=d["residual"],
                              w_post=d["w_post"], gate=d["gate"], alpha=0.5, w_pre=d["w_pre"],
                              eps=EPS, h=out["h"], n=out["n"])
    for seed in (1, 2, 3):
        new = inputs(4, 2560, torch.bfloat16, seed, True, True, 4, True)
        for k in d:
            d[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        same(out, run(new, 0.5))


@pytest.mark.gpu
def test_binding_checks_on_the_gpu():
    x = torch.zeros(4, 256, device="cuda")
    q = torch.empty(4, 256, dtype=torch.int8, device="cuda")
    s = torch.empty(4, 2, device="cuda")
    t = torch.empty(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        pq2.pq2_norm_quantize(x, q, s, t, residual=x.half())
    with pytest.raises(TypeError):
        pq2.pq2_norm_quantize(x, q, s, t, w_pre=torch.ones(256, device="cuda").half())
    with pytest.raises(ValueError):
        pq2.pq2_norm_quantize(x, q, s, t, w_pre=torch.ones(128, device="cuda"))
    with pytest.raises(ValueError):
        pq2.pq2_norm_quantize(x, q, s, t, residual=x.cpu())
    with pytest.raises(ValueError):
        pq2.pq2_norm_quantize(x.t().contiguous().t(), q, s, t)
    with pytest.raises(pq2.PQ2Error):
        pq2.pq2_norm_quantize(x, q, s, t, gate=torch.ones(3, 256, device="cuda"))
    with pytest.raises(pq2.PQ2Error):
        pq2.pq2_norm_quantize(x, q, s, None)
    with pytest.raises(pq2.PQ2Error):
        pq2.pq2_norm_quantize(x)
    with pytest.raises(pq2.PQ2Error):
        pq2.pq2_norm_quantize(x, q, s, t, eps=0.0)
    g1 = torch.rand(256, device="cuda")
    a, b = pq2.norm_quantize(x + 1, gate=g1), pq2.norm_quantize(x + 1, gate=g1[None])
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [((1 << 22) + 3, 128), (430000, 5120)])
def test_many_rows_and_offsets_past_32_bits(M, K):
    """More rows than blocks, and element offsets beyond 2^31: the rows at the
    ends are those of a small call."""
    print(f"norm_quantize large M={M} K={K}", flush=True)
    x = torch.randn(1000, K, device="cuda").bfloat16().repeat(M // 1000 + 1, 1)[:M].contiguous()
    x[-1] *= 2
    w = 1 + 0.1 * torch.randn(K, device="cuda")
    out = {"h": torch.empty_like(x), "q": torch.empty(M, K, dtype=torch.int8, device="cuda"),
           "s": torch.empty(M, K // 128, device="cuda"),
           "t": torch.empty(M, K // 128, dtype=torch.int32, device="cuda")}
    pq2.pq2_norm_quantize(x, out["q"], out["s"], out["t"], w_pre=w, h=out["h"], alpha=0.5)
    for sl in (slice(0, 3), slice(M // 2, M // 2 + 3), slice(M - 3, M)):
        h, q, s, t = pq2.norm_quantize(x[sl].contiguous(), w_pre=w, alpha=0.5)
        same({k: out[k][sl] for k in out}, {"h": h, "q": q, "s": s, "t": t})


@pytest.mark.gpu
@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("K", [640, 17408, 32896])
def test_signed_zeros_without_a_residual(K, ty):
    """alpha * gate * p of powers of two is exact, its signed zeros among it: what
    a call leaves out adds nothing, not even +0 to a -0."""
    g = torch.Generator().manual_seed(K)
    x = torch.randint(-3, 4, (3, K), generator=g).float()
    x[:, 1::5] = -0.0
    x[:, 2::5] = 0.0
    gate = torch.where(torch.rand(K, generator=g) < 0.5, -2.0, 0.5)
    bits = torch.int32 if ty == "f32" else torch.int16
    print(f"signed zeros K={K} {ty}", flush=True)
    for alpha, gt in ((1.0, None), (-0.5, None), (2.0, gate), (0.0, None)):
        want = (alpha * x if gt is None else alpha * (x * gt)).to(TYPES[ty])
        xd = x.to(TYPES[ty]).cuda()
        h, n = torch.empty_like(xd), torch.empty_like(xd)
        pq2.pq2_norm_quantize(xd, h=h, n=n, alpha=alpha,
                              gate=None if gt is None else gt.to(TYPES[ty]).cuda())
        assert torch.equal(h.cpu().view(bits), want.view(bits))
        assert torch.equal(n.cpu().view(bits), want.view(bits))
