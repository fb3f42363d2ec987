"""pq2_lora_add: low-rank adapters of many requests beside a shared projection.

The reference is float64 (numpy). With u = 2^-24, and 2 u for every addition
inside the matrix cores (whose rounding is taken as a truncation):

* a sum of A x passes at most 32 additions in a matrix step, K / 128 steps of a
  wave, 4 waves and 16 chunks: E_v = 2 (52 + K / 128) u sum |A| |x|, with the
  split of a float32 or binary16 operand into bfloat16 parts dropping at most
  2^-22 of each product (8 u more);
* B v passes at most 32 additions in a step and 8 steps of at most 5 part
  products: E_d = |scale| (sum |B| E_v + 2 (72 + 8) u sum |B| |v|);
* y = base + d is rounded once: u |y| for float32, half a step (2^-8 |y|) for
  bfloat16.

Small integers pass through every step exactly, so with them y has to be exact.
"""

import numpy as np
import pytest
import torch

pq2 = pytest.importorskip("gemm_pq2_w2a8_amd")

U = 2.0 ** -24
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_HIP, ERR_ARG, ERR_SCRATCH = 0, 1, 2, 3, 4, 5, 6
P = 0x100000
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


# ------------------------------------------------------------------ refusals (CPU)

def call(x=P, xf=1, a=P, b=P, wf=1, adapter=P, ranks=None, scale=None, base=None, y=P, yf=0, M=2,
         N=8, K=128, R=8, L=3, work=None, work_bytes=0):
    """The C entry with fake addresses; without a workspace nothing can launch."""
    return pq2.lib.pq2_lora_add(x, xf, a, b, wf, adapter, ranks, scale, base, y, yf, M, N, K, R, L,
                                work, work_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), ERR_NULL), (dict(a=None), ERR_NULL), (dict(b=None), ERR_NULL),
    (dict(adapter=None), ERR_NULL), (dict(y=None), ERR_NULL),
    (dict(M=0), ERR_SHAPE), (dict(M=(1 << 24) + 1), ERR_SHAPE), (dict(N=0), ERR_SHAPE),
    (dict(N=(1 << 20) + 1), ERR_SHAPE), (dict(K=64), ERR_SHAPE), (dict(K=130), ERR_SHAPE),
    (dict(K=(1 << 24) + 128), ERR_SHAPE), (dict(L=0), ERR_SHAPE), (dict(L=(1 << 20) + 1), ERR_SHAPE),
    (dict(R=0), ERR_SHAPE), (dict(R=12), ERR_SHAPE), (dict(R=264), ERR_SHAPE), (dict(R=-8), ERR_SHAPE),
    (dict(L=1 << 20, R=256, K=1 << 13), ERR_SHAPE),          # A above PQ2_MAX_ELEMS
    (dict(L=1 << 20, R=256, N=1 << 13), ERR_SHAPE),          # B above PQ2_MAX_ELEMS
    (dict(M=1 << 24, N=1 << 17), ERR_SHAPE),
    (dict(xf=3), ERR_ARG), (dict(xf=-1), ERR_ARG), (dict(wf=0), ERR_ARG), (dict(wf=3), ERR_ARG),
    (dict(yf=2), ERR_ARG), (dict(yf=-1), ERR_ARG),
    (dict(x=P + 8), ERR_ALIGN), (dict(a=P + 8), ERR_ALIGN), (dict(b=P + 8), ERR_ALIGN),
    (dict(adapter=P + 2), ERR_ALIGN), (dict(ranks=P + 2), ERR_ALIGN), (dict(scale=P + 2), ERR_ALIGN),
    (dict(base=P + 2), ERR_ALIGN), (dict(y=P + 2), ERR_ALIGN), (dict(y=P + 1, yf=1), ERR_ALIGN),
    (dict(base=P + 1, yf=1), ERR_ALIGN), (dict(work=P + 8, work_bytes=1 << 20), ERR_ALIGN),
    (dict(), ERR_SCRATCH), (dict(work=P, work_bytes=2 * 8 * 4 - 1), ERR_SCRATCH),
    (dict(work=None, work_bytes=1 << 20), ERR_SCRATCH),
])
def test_refusals(kw, want):
    assert call(**kw) == want


def test_workspace_query():
    f = pq2.lora_workspace_bytes
    assert f(0, 128, 8) == 0 and f(1, 100, 8) == 0 and f(1, 128, 12) == 0 and f(1, 128, 512) == 0
    for M, K, R in ((1, 128, 8), (1, 5120, 16), (16, 17408, 64), (555, 17408, 32), (4096, 5120, 64),
                    (1 << 24, 128, 256)):
        n = f(M, K, R)
        assert n >= M * R * 4 and n % (M * R * 4) == 0
        assert n <= 16 * M * R * 4


def test_binding_refusals():
    x, a, b = torch.zeros(2, 128), torch.zeros(3, 8, 128).bfloat16(), torch.zeros(3, 4, 8).bfloat16()
    ids, y = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4)
    with pytest.raises(ValueError):
        pq2.pq2_lora_add(x, a, b, ids, y)                     # not on a GPU
    with pytest.raises(TypeError):
        pq2.pq2_lora_add(x.double(), a, b, ids, y)
    with pytest.raises(TypeError):
        pq2.pq2_lora_add(x, a.float(), b, ids, y)
    with pytest.raises(TypeError):
        pq2.pq2_lora_add(x, a, b, ids, y.half())
    with pytest.raises(ValueError):
        pq2.pq2_lora_add(x, a[0], b, ids, y)


# ------------------------------------------------------------------ problems

class Problem:
    def __init__(self, M, K, N, R, L, xt=BF16, wt=BF16, yt=F32, ids="rows", ranks=None, scale=True,
                 base=True, seed=0, integers=False):
        g = torch.Generator().manual_seed(seed)
        rnd = (lambda *s: torch.randint(-2, 3, s, generator=g).float()) if integers else \
            (lambda *s: torch.randn(s, generator=g))  # noqa: E731
        self.M, self.K, self.N, self.R, self.L = M, K, N, R, L
        self.x = rnd(M, K).to(xt)
        self.a = (rnd(L, R, K) / (1 if integers else K ** 0.5)).to(wt)
        self.b = (rnd(L, N, R) / (1 if integers else R ** 0.5)).to(wt)
        if ids == "rows":
            self.ids = torch.randint(-1, L, (M,), generator=g).to(torch.int32)
        elif ids == "runs":
            self.ids = (torch.arange(M) * L // M).to(torch.int32)
        else:
            self.ids = torch.tensor(ids, dtype=torch.int32)
        self.ranks = None if ranks is None else torch.tensor(ranks, dtype=torch.int32)
        self.scale = (torch.randint(1, 3, (L,), generator=g).float() if integers else
                      torch.rand(L, generator=g) * 2 - 1) if scale else None
        self.base = rnd(M, N).to(yt) if base else None
        self.y0 = rnd(M, N).to(yt)

    def device(self):
        d = lambda v: None if v is None else v.cuda()  # noqa: E731
        return dict(x=d(self.x), a=d(self.a), b=d(self.b), adapter=d(self.ids), y=d(self.y0),
                    base=d(self.base), ranks=d(self.ranks), scale=d(self.scale))

    def run(self, **kw):
        d = self.device()
        pq2.pq2_lora_add(**d, **kw)
        return d["y"].cpu()

    def reference(self):
        base = (self.y0 if self.base is None else self.base)
        y, err = base.double().numpy().copy(), np.zeros((self.M, self.N))
        gv = 2 * (52 + self.K / 128) * U + 8 * U
        for m in range(self.M):
            l = int(self.ids[m])
            if not 0 <= l < self.L:
                continue
            r = self.R if self.ranks is None else min(max(int(self.ranks[l]), 0), self.R)
            a, b = self.a[l, :r].double().numpy(), self.b[l, :, :r].double().numpy()
            x = self.x[m].double().numpy()
            f = 1.0 if self.scale is None else float(self.scale[l])
            v = a @ x
            ev = gv * (np.abs(a) @ np.abs(x))
            y[m] += f * (b @ v)
            err[m] = abs(f) * (np.abs(b) @ ev + 160 * U * (np.abs(b) @ np.abs(v)))
        return base, y, err

    def check(self, got, exact=False):
        base, ref, err = self.reference()
        some = ((self.ids >= 0) & (self.ids < self.L)).numpy()
        bits = torch.int32 if base.dtype == F32 else torch.int16
        assert torch.equal(got[~some].view(bits), base[~some].view(bits))      # bit for bit
        g = got.double().numpy()
        if exact:
            assert (g[some] == ref[some]).all()
            return
        step = U if base.dtype == F32 else 2.0 ** -8
        bound = err + (np.abs(ref) + err) * step
        assert (np.abs(g - ref)[some] <= bound[some]).all(), (np.abs(g - ref) - bound).max()


# M, K, N, R, L, ids, ranks
SHAPES = {
    "one_row": (1, 5120, 300, 16, 4, [2], None),
    "one_row_rank8": (1, 128, 1, 8, 1, [0], None),
    "one_without": (1, 256, 40, 8, 3, [-1], None),
    "two": (2, 640, 65, 24, 3, [2, 0], [1, 9, 24]),
    "decode_each_own": (16, 2048, 100, 64, 20, list(range(16)), [1 + 3 * i for i in range(20)]),
    "odd_rows": (17, 1280, 63, 40, 5, "rows", [40, 0, 7, 33, 16]),
    "bad_ids": (20, 384, 48, 16, 3, [0, 3, -1, 2 ** 31 - 1, -2 ** 31] * 4, [99, -5, 16]),
    "mixed": (100, 896, 257, 32, 6, "rows", None),
    "runs": (150, 512, 130, 64, 3, "runs", None),
    "wide_rank": (9, 1024, 70, 256, 4, "rows", [256, 130, 65, 64]),
    "rank_72": (33, 256, 50, 72, 2, "rows", None),
    "long_k": (5, 17408, 30, 16, 2, "rows", None),
    "many_rows": (1100, 128, 20, 8, 4, "rows", None),
    "many_adapters": (300, 256, 70, 8, 250, "rows", None),
    "window_edge": (129, 512, 300, 48, 130, list(range(129)), [48 - i % 48 for i in range(130)]),
    "pipelined_odd": (1500, 256, 131, 40, 5, "rows", [40, 3, 17, 0, 33]),
    "pipelined_runs": (1300, 256, 262, 64, 3, "runs", [64, 64, 10]),
    "deep_many": (1100, 256, 70, 136, 3, "runs", None),
    "prompt": (700, 640, 515, 64, 2, "runs", [64, 17]),
}
TYPES = [(BF16, BF16, F32), (BF16, BF16, BF16), (F16, F16, F32), (F16, F16, BF16), (F32, BF16, F32),
         (F32, F16, F32), (BF16, F16, BF16), (F16, BF16, F32)]


@pytest.mark.gpu
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(v)[6:] for v in t))
@pytest.mark.parametrize("name", list(SHAPES))
def test_against_float64(name, types):
    M, K, N, R, L, ids, ranks = SHAPES[name]
    print(f"lora_add {name} {types}", flush=True)
    p = Problem(M, K, N, R, L, *types, ids=ids, ranks=ranks, seed=len(name))
    p.check(p.run())
    p = Problem(M, K, N, R, L, *types, ids=ids, ranks=ranks, seed=3, base=False, scale=False)
    p.check(p.run())                                          # in place


@pytest.mark.gpu
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(v)[6:] for v in t))
@pytest.mark.parametrize("name", list(SHAPES))
def test_exact_with_small_integers(name, types):
    M, K, N, R, L, ids, ranks = SHAPES[name]
    print(f"lora_add integers {name} {types}", flush=True)
    xt, wt, _ = types
    p = Problem(M, K, N, R, L, xt, wt, F32, ids=ids, ranks=ranks, seed=5, integers=True)
    p.check(p.run(), exact=True)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(10))
def test_random_shapes(seed):
    rng = np.random.default_rng(77 + seed)
    M, K = int(np.exp(rng.uniform(0, 6))), 128 * int(rng.integers(1, 30))
    N, R, L = int(rng.integers(1, 600)), 8 * int(rng.integers(1, 17)), int(rng.integers(1, 12))
    ranks = rng.integers(0, R + 1, L).tolist() if seed % 2 else None
    types = TYPES[seed % len(TYPES)]
    print(f"lora_add random M={M} K={K} N={N} R={R} L={L} {types}", flush=True)
    p = Problem(M, K, N, R, L, *types, ids="rows" if seed % 3 else "runs", ranks=ranks, seed=seed)
    p.check(p.run())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [6, 200])
@pytest.mark.parametrize("wt", [BF16, F16])
def test_what_is_masked_has_no_influence(wt, M):
    """NaN and infinities behind the ranks, in adapters no row uses and in the
    rows of other requests stay where they are."""
    R, L = 40, 4
    ids = [[0, 1, 3, -1, 1, 0][i % 6] for i in range(M)]
    p = Problem(M, 512, 90, R, L, wt, wt, F32, ids=ids, ranks=[17, 40, 40, 1], seed=2)
    clean = p.run()
    p.check(clean)
    q = Problem(M, 512, 90, R, L, wt, wt, F32, ids=ids, ranks=[17, 40, 40, 1], seed=2)
    q.a[0, 17:], q.b[0, :, 17:] = float("nan"), float("inf")
    q.a[3, 1:], q.b[3, :, 1:] = float("inf"), float("nan")
    q.a[2], q.b[2] = float("nan"), float("nan")               # nobody's
    assert torch.equal(q.run(), clean)
    q.a[1] = float("nan")                                     # rows 1, 4 of every 6 alone
    q.b[1] = float("inf")
    q.x[2] = float("nan")                                     # and row 2
    got = q.run()
    hit = torch.tensor([i % 6 in (1, 4) or i == 2 for i in range(M)])
    assert torch.equal(got[~hit], clean[~hit]) and torch.isnan(got[hit]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("wt", [BF16, F16])
def test_extremes_of_the_types(wt):
    """Subnormal and large 16-bit values keep their products."""
    K, N, R = 256, 40, 8
    p = Problem(4, K, N, R, 2, wt, wt, F32, ids=[0, 1, 0, 1], scale=False, seed=4)
    big, small = (60000.0, 6e-8) if wt == F16 else (1e15, 1e-15)
    p.x[0], p.x[1] = small, big
    p.a[0, :, ::2], p.a[1, :, ::2] = big, small
    p.b[0, ::3] = small * 3
    p.base.zero_()
    p.check(p.run())
    q = Problem(4, K, N, R, 2, F32, wt, F32, ids=[0, 1, 0, 1], scale=False, seed=4)
    q.x[0] = 1e-30
    q.x[1] *= 1e20
    q.base.zero_()
    q.check(q.run())


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,R", [(1, 5120, 16), (30, 5120, 72), (555, 1280, 32)])
def test_workspace_sizes(M, K, R):
    """The least workspace, one in between and the query's, each right and each
    the same on a repeat; the workspace's contents before a call do not matter."""
    p = Problem(M, K, 120, R, 3, seed=6)
    full = pq2.lora_workspace_bytes(M, K, R)
    for n in (M * R * 4, min(full, 3 * M * R * 4), full):
        work = torch.full((n // 4,), float("nan"), device="cuda")
        y = p.run(workspace=work)
        p.check(y)
        work.fill_(1e30)
        assert torch.equal(y, p.run(workspace=work))
    with pytest.raises(pq2.PQ2Error):
        p.run(workspace=torch.empty(M * R * 4 - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pq2.PQ2Error):
        p.run(workspace=None)
    with pytest.raises(ValueError):
        p.run(workspace=torch.empty(full, dtype=torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [5, 1200])
@pytest.mark.parametrize("N", [64, 66, 67])
@pytest.mark.parametrize("yt", [F32, BF16])
def test_outputs_aligned_like_their_elements(yt, N, M):
    """base and y that begin one element after a 16-byte boundary, with guards."""
    p = Problem(M, 256, N, 24, 3, seed=11, yt=yt, ranks=[24, 5, 16])
    want = p.run()
    d = p.device()
    flat = [torch.full((M * N + 32,), 7.0, dtype=yt, device="cuda") for _ in range(2)]
    base, y = (f[1:1 + M * N].view(M, N) for f in flat)
    base.copy_(d["base"])
    pq2.pq2_lora_add(**{**d, "base": base, "y": y})
    assert torch.equal(y.cpu(), want)
    assert (flat[1][:1] == 7).all() and (flat[1][1 + M * N:] == 7).all()
    assert torch.equal(base, d["base"])


@pytest.mark.gpu
def test_in_place_is_the_same():
    p = Problem(37, 640, 100, 24, 4, seed=7, yt=BF16)
    want = p.run()
    d = p.device()
    y = d["base"].clone()
    pq2.pq2_lora_add(d["x"], d["a"], d["b"], d["adapter"], y, scale=d["scale"])
    assert torch.equal(y.cpu(), want)
    y = d["base"].clone()
    pq2.pq2_lora_add(d["x"], d["a"], d["b"], d["adapter"], y, base=y, scale=d["scale"])
    assert torch.equal(y.cpu(), want)


@pytest.mark.gpu
def test_streams_and_graph_replays():
    """Two streams with a workspace each; a captured call replayed with other
    adapters and inputs, between eager calls."""
    p = Problem(20, 1024, 200, 32, 5, seed=8)
    want = p.run()
    outs = []
    for _ in range(2):
        st = torch.cuda.Stream()
        d = p.device()
        st.wait_stream(torch.cuda.current_stream())
        pq2.pq2_lora_add(**d, stream=st)
        outs.append(d["y"])
    torch.cuda.synchronize()
    assert all(torch.equal(o.cpu(), want) for o in outs)
    d = p.device()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pq2.pq2_lora_add(**d)
    for seed in (1, 2, 3):
        n = Problem(20, 1024, 200, 32, 5, seed=seed)
        for k, v in n.device().items():
            if v is not None:
                d[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d["y"].cpu(), n.run())


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Adapters beyond 4 GiB, and outputs beyond 2^31 elements."""
    L, R, K, N = 70, 256, 1 << 17, 64                          # A: 4.7 GB
    print("lora_add 4.7 GB of adapters", flush=True)
    a = (torch.randn(1, R, K, device="cuda") / K ** 0.5).bfloat16().repeat(L, 1, 1)
    b = (torch.randn(1, N, R, device="cuda") / 16).bfloat16().repeat(L, 1, 1)
    x = torch.randn(2, K, device="cuda").bfloat16()
    y = [torch.zeros(2, N, device="cuda") for _ in range(2)]
    for at, ids in ((0, [0, 0]), (1, [L - 1, 0])):
        pq2.pq2_lora_add(x, a, b, torch.tensor(ids, dtype=torch.int32, device="cuda"), y[at])
    assert torch.equal(*y)
    del a, b
    M, N, K, R = 60000, 40000, 128, 8                          # 2.4e9 outputs
    print("lora_add 2.4e9 outputs", flush=True)
    p = Problem(64, K, N, R, 3, seed=9, yt=BF16)
    d = p.device()
    reps = M // 64 + 1
    x, ids = d["x"].repeat(reps, 1)[:M].contiguous(), d["adapter"].repeat(reps)[:M].contiguous()
    y = torch.zeros(M, N, dtype=BF16, device="cuda")
    pq2.pq2_lora_add(x, d["a"], d["b"], ids, y, scale=d["scale"])
    want = torch.zeros(64, N, dtype=BF16, device="cuda")
    sl = slice(M // 64 * 64 - 64, M // 64 * 64)
    pq2.pq2_lora_add(x[sl].contiguous(), d["a"], d["b"], ids[sl].contiguous(), want,
                     scale=d["scale"])
    err = (y[sl].float() - want.float()).abs()
    assert (err <= want.float().abs() * 2.0 ** -7 + 1e-6).all()


@pytest.mark.gpu
def test_binding_checks_on_the_gpu():
    p = Problem(4, 256, 30, 16, 3, seed=1)
    d = p.device()
    for key, bad in (("adapter", d["adapter"].long()), ("b", d["b"].half()), ("base", d["base"].half()),
                     ("scale", d["scale"].half())):
        with pytest.raises(TypeError):
            pq2.pq2_lora_add(**{**d, key: bad})
    for key, bad in (("adapter", d["adapter"][:3]), ("b", d["b"][:2]), ("base", d["base"].cpu()),
                     ("x", d["x"].t().contiguous().t()), ("ranks", d["adapter"])):
        with pytest.raises(ValueError):
            pq2.pq2_lora_add(**{**d, key: bad})
    with pytest.raises(pq2.PQ2Error):
        pq2.pq2_lora_add(d["x"], d["a"][:, :12].contiguous(), d["b"][:, :, :12].contiguous(),
                         d["adapter"], d["y"])


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 1100])
@pytest.mark.parametrize("N", [1, 2, 3, 5, 63, 254, 257, 511])
def test_columns_at_the_end_of_the_last_adapter(N, M):
    """Columns that are no multiple of four, B followed by NaN: nothing behind an
    adapter's last column counts, and no column is lost."""
    p = Problem(M, 256, N, 24, 3, seed=N, ids=[2, 0, 2] + [i % 3 for i in range(M - 3)],
                ranks=[24, 7, 17])
    want = p.run()
    p.check(want)
    d = p.device()
    flat = torch.full((p.b.numel() + 4096,), float("nan"), dtype=BF16, device="cuda")
    flat[:p.b.numel()] = d["b"].view(-1)
    pq2.pq2_lora_add(**{**d, "b": flat[:p.b.numel()].view(p.b.shape)})
    assert torch.equal(d["y"].cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("K,N", [((1 << 17) + 128, 64), (128, (1 << 17) + 3)])
def test_the_last_of_adapters_past_4_gib(K, N):
    """A, then B, of 4.7 GB whose last adapter alone has contents of its own and a
    stride that does not divide 2^32: an offset cut to 32 bits, or another
    adapter's, gives another result. Equal to a call on that adapter by itself."""
    L, R = 70, 256
    assert L * R * max(K, N) * 2 > 1 << 32 and (1 << 32) % (R * max(K, N) * 2) != 0
    print(f"lora_add last of {L} adapters K={K} N={N}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(12)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    a, b = (rnd(1, R, K) / K ** 0.5).repeat(L, 1, 1), (rnd(1, N, R) / 16).repeat(L, 1, 1)
    a[L - 1], b[L - 1] = rnd(R, K) / K ** 0.5, rnd(N, R) / 16
    x = rnd(2, K)
    ids = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    y, alone, first = (torch.zeros(2, N, device="cuda") for _ in range(3))
    pq2.pq2_lora_add(x, a, b, ids(L - 1, 5), y)
    pq2.pq2_lora_add(x, a[L - 1:], b[L - 1:], ids(0, 0), alone)
    pq2.pq2_lora_add(x, a[:1], b[:1], ids(0, 0), first)
    assert torch.equal(y[0], alone[0]) and torch.equal(y[1], first[1])
    assert not torch.equal(alone[0], first[0])
    v = a[L - 1].double() @ x[0].double()
    ref = b[L - 1].double() @ v
    size = b[L - 1].double().abs() @ (a[L - 1].double().abs() @ x[0].double().abs())
    # the file's bounds: E_v = 2 (52 + K / 128) u, 160 u for B v, y's own rounding
    bound = (2 * (52 + K / 128) + 8 + 160 + 1) * U * size
    assert ((y[0].double() - ref).abs() <= bound).all()
