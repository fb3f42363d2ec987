"""pq2_gemm_grouped: PQ2_0 products grouped by expert with ragged sizes.

The reference is float64 (numpy) from the unpacked codes. The float32 epilogue
adds G terms in some fixed order, each with a rounded scale product, and the row
scale is one more product: |y - y64| <= (G + 4) 2^-24 sum_g |term_g|, whatever
the order. With unit scales every partial sum is an integer below 2^24 and y has
to be exact. A bfloat16 y adds half a step (2^-8 of its magnitude).
"""

import numpy as np
import pytest
import torch

pq2 = pytest.importorskip("gemm_pq2_w2a8_amd")

import pq2_synth as synth  # noqa: E402

U = 2.0 ** -24
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_HIP, ERR_ARG = 0, 1, 2, 3, 4, 5
P = 0x100000


# ------------------------------------------------------------------ refusals (CPU)

def call(q=P, s=P, t=P, R=4, codes=P, ws=P, offsets=P, E=2, rows=P, row_scale=None, y=P, fmt=0,
         T=4, N=8, K=64):
    """The C entry with fake addresses; the default K is refused after every
    check that comes before the shape's, so nothing here can launch."""
    return pq2.lib.pq2_gemm_grouped(q, s, t, R, codes, ws, offsets, E, rows, row_scale, y, fmt, T,
                                    N, K, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), ERR_NULL), (dict(s=None), ERR_NULL), (dict(t=None), ERR_NULL),
    (dict(codes=None), ERR_NULL), (dict(ws=None), ERR_NULL), (dict(offsets=None), ERR_NULL),
    (dict(y=None), ERR_NULL),
    (dict(), ERR_SHAPE), (dict(K=0), ERR_SHAPE), (dict(K=(1 << 24) + 128), ERR_SHAPE),
    (dict(E=0, K=128), ERR_SHAPE), (dict(E=-1, K=128), ERR_SHAPE), (dict(E=4097, K=128), ERR_SHAPE),
    (dict(T=-1, K=128), ERR_SHAPE), (dict(T=(1 << 24) + 1, K=128), ERR_SHAPE),
    (dict(N=0, K=128), ERR_SHAPE), (dict(N=(1 << 20) + 1, K=128), ERR_SHAPE),
    (dict(R=0, K=128), ERR_SHAPE), (dict(R=3, rows=None, K=128), ERR_SHAPE),
    (dict(E=4096, N=1 << 20, K=128), ERR_SHAPE),            # E*N above PQ2_MAX_DIM
    (dict(E=1024, N=1 << 20, K=1 << 13), ERR_SHAPE),        # E*N*K/4 above PQ2_MAX_ELEMS
    (dict(T=1 << 24, N=1 << 17, K=128), ERR_SHAPE),         # T*N above PQ2_MAX_ELEMS
    (dict(fmt=2, K=128), ERR_ARG), (dict(fmt=-1, K=128), ERR_ARG),
    (dict(q=P + 8, K=128), ERR_ALIGN), (dict(codes=P + 8, K=128), ERR_ALIGN),
    (dict(s=P + 2, K=128), ERR_ALIGN), (dict(t=P + 2, K=128), ERR_ALIGN),
    (dict(ws=P + 1, K=128), ERR_ALIGN), (dict(offsets=P + 2, K=128), ERR_ALIGN),
    (dict(rows=P + 2, K=128), ERR_ALIGN), (dict(row_scale=P + 2, K=128), ERR_ALIGN),
    (dict(y=P + 2, K=128), ERR_ALIGN), (dict(y=P + 1, fmt=1, K=128), ERR_ALIGN),
])
def test_refusals(kw, want):
    assert call(**kw) == want


def test_no_slots_is_no_work():
    assert call(T=0, K=128) == OK
    assert call(T=0, y=None, rows=None, K=128) == OK


def test_binding_refusals():
    q = torch.zeros(2, 128, dtype=torch.int8)
    s, t = torch.zeros(2, 1), torch.zeros(2, 1, dtype=torch.int32)
    codes = torch.zeros(3, 8, 32, dtype=torch.uint8)
    ws = torch.zeros(3, 8, 1, dtype=torch.float16)
    off = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        pq2.pq2_gemm_grouped(q, s, t, codes, ws, off, torch.zeros(2, 8))      # not on a GPU
    with pytest.raises(ValueError):
        pq2.pq2_gemm_grouped(q, s, t, codes[0], ws, off, torch.zeros(2, 8))
    with pytest.raises(TypeError):
        pq2.pq2_gemm_grouped(q, s, t, codes, ws, off, torch.zeros(2, 8).half())


# ------------------------------------------------------------------ problems

class Problem:
    def __init__(self, counts, N, K, R=None, seed=0, unit=False, spare=0, weighted=False,
                 invalid=False, lead=0):
        """counts: slots per expert; R: gathered rows (None: row i); spare / lead:
        slots behind / before all experts; invalid: some rows out of range."""
        rng = np.random.default_rng(seed)
        self.counts, self.N, self.K, self.E = list(counts), N, K, len(counts)
        self.G = K // 128
        self.off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32) + np.int32(lead)
        self.T = int(self.off[-1]) + spare
        n_rows = R if R is not None else max(self.T, 1)
        self.q = rng.integers(-127, 128, size=(n_rows, K)).astype(np.int8)
        self.t = self.q.reshape(n_rows, self.G, 128).astype(np.int32).sum(-1).astype(np.int32)
        self.s = (np.ones((n_rows, self.G)) if unit else
                  rng.uniform(0.005, 0.05, (n_rows, self.G))).astype(np.float32)
        self.codes = synth.draw_codes(self.E * N, K, rng).reshape(self.E, N, K // 4)
        self.ws = (np.ones((self.E, N, self.G), np.float16) if unit else
                   synth.draw_wscale(self.E * N, K, rng).reshape(self.E, N, self.G))
        self.rows = None
        if R is not None:
            self.rows = rng.integers(0, R, self.T).astype(np.int32)
            if invalid:
                bad = rng.random(self.T) < 0.3
                self.rows[bad] = rng.choice([-1, R, 2 ** 31 - 1, -2 ** 31], bad.sum())
        self.row_scale = rng.uniform(-1, 1, self.T).astype(np.float32) if weighted else None

    def plane(self):
        n = self.q.shape[0]
        return np.ascontiguousarray(
            self.q.reshape(n, -1, 32, 4).transpose(0, 1, 3, 2).reshape(n, self.K))

    def reference(self):
        """float64 y and sum of |terms| of every slot that an expert owns (others NaN)."""
        y = np.full((self.T, self.N), np.nan)
        tabs = np.zeros((self.T, self.N))
        for e in range(self.E):
            lo, hi = self.off[e], self.off[e + 1]
            if lo == hi:
                continue
            c = self.codes[e][:, :, None] >> np.array([0, 2, 4, 6], np.uint8) & 3
            w = (c.astype(np.float64) - 1).reshape(self.N, self.G, 128)
            rows = np.arange(lo, hi) if self.rows is None else self.rows[lo:hi]
            good = (rows >= 0) & (rows < self.q.shape[0])
            rows = np.where(good, rows, 0)
            x = self.q[rows].reshape(-1, self.G, 128).astype(np.float64)
            d = np.matmul(x.transpose(1, 0, 2), w.transpose(1, 2, 0))         # [G][slots][N]
            scale = self.s[rows].astype(np.float64).T[:, :, None] * \
                self.ws[e].astype(np.float64).T[:, None, :]
            f = np.ones(hi - lo) if self.row_scale is None else self.row_scale[lo:hi].astype(np.float64)
            f = np.where(good, f, 0.0)[:, None]
            y[lo:hi] = (d * scale).sum(0) * f
            tabs[lo:hi] = np.abs(d * scale).sum(0) * np.abs(f)
        return y, tabs

    def device(self):
        d = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return dict(q=d(self.plane()), s=d(self.s), t=d(self.t), codes=d(self.codes),
                    wscale=d(self.ws), offsets=d(self.off), rows=d(self.rows),
                    row_scale=d(self.row_scale))

    def run(self, ty=torch.float32, **kw):
        y = torch.full((self.T, self.N), 7.0, dtype=ty, device="cuda")
        pq2.pq2_gemm_grouped(y=y, **self.device(), **kw)
        return y.cpu().float().double().numpy()

    def check(self, got, ty=torch.float32, exact=False):
        ref, tabs = self.reference()
        owned = ~np.isnan(ref[:, 0]) if self.N else np.zeros(self.T, bool)
        assert (got[~owned] == 7.0).all()                    # left as they were
        err = np.abs(got - ref)[owned]
        bound = np.zeros_like(err) if exact else (self.G + 4) * U * tabs[owned]
        if ty == torch.bfloat16:
            bound = bound + (np.abs(ref[owned]) + bound) * 2.0 ** -8
        assert (err <= bound).all(), (err - bound).max()


SHAPES = {
    "one_slot": ([0, 1, 0], 16, 128),
    "one_expert_row": ([1], 1, 128),
    "token_of_8_experts": ([0, 1, 1, 0, 1, 0, 1, 1, 0, 0, 1, 1, 1, 0, 0, 0], 96, 1280),
    "two_to_five": ([2, 3, 0, 4, 5, 1], 40, 640),
    "eights": ([8, 7, 6, 9, 0], 33, 1152),
    "around_16": ([15, 16, 17, 0, 1, 32, 33], 65, 512),
    "around_64": ([63, 64, 65, 1, 0, 128, 129], 130, 384),
    "skewed": ([0, 300, 1, 0, 0, 5, 40], 257, 256),
    "last_only": ([0, 0, 0, 77], 100, 1024),
    "long_k": ([3, 20, 1], 24, 17408),
    "odd_groups": ([4, 30, 70], 129, 128 * 41),
    "wide": ([5, 0, 17], 2050, 256),
    "large_tiles": ([600, 0, 513, 255], 515, 640),
    "tiles_of_64": ([40, 70, 33, 0, 64, 129], 300, 2048),
    "tiles_of_128": ([600, 0, 513, 255, 1], 515, 1024),
    "one_long": ([391], 257, 5120),
    "few_blocks_of_16": ([9, 5, 0, 14, 7], 70, 1024),
    "many_blocks_of_16": ([8, 3, 11] * 20, 1100, 1024),
    "many_streams": ([1, 0, 2] * 20 + [6, 1], 1000, 1152),
    "staged_32": ([8, 17, 33, 3], 100, 1152),
    "many_experts": ([i % 4 for i in range(200)], 17, 256),
    "most_experts": ([i % 2 for i in range(4096)], 9, 128),
    "over_4_per_lane": ([(i * 7) % 3 for i in range(700)], 16, 128),
}


@pytest.mark.gpu
@pytest.mark.parametrize("ty", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_against_float64(name, ty):
    counts, N, K = SHAPES[name]
    print(f"gemm_grouped {name} {ty}", flush=True)
    for kw in (dict(R=11, weighted=True, spare=3), dict()):
        p = Problem(counts, N, K, seed=len(name), **kw)
        p.check(p.run(ty), ty)


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(SHAPES))
def test_exact_with_unit_scales(name):
    """Unit scales: y is the integer dot, so every code, activation and group
    has to be where it belongs."""
    counts, N, K = SHAPES[name]
    print(f"gemm_grouped exact {name}", flush=True)
    p = Problem(counts, N, K, R=9, seed=3, unit=True)
    p.check(p.run(), exact=True)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(seed):
    rng = np.random.default_rng(1000 + seed)
    E = int(rng.integers(1, 40))
    mean = float(np.exp(rng.uniform(np.log(0.3), np.log(120))))
    counts = rng.poisson(rng.exponential(mean, E))
    N, K = int(rng.integers(1, 400)), 128 * int(rng.integers(1, 24))
    R = None if seed % 3 == 0 else int(rng.integers(1, 50))
    print(f"gemm_grouped random E={E} T={counts.sum()} N={N} K={K} R={R}", flush=True)
    if counts.sum() == 0:
        counts[0] = 1
    p = Problem(counts, N, K, R=R, seed=seed, weighted=seed % 2 == 0, spare=seed % 4)
    ty = torch.bfloat16 if seed % 4 == 1 else torch.float32
    p.check(p.run(ty), ty)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K", [([3, 9, 0, 1], 50, 384), ([40, 9, 130], 70, 1024),
                                        ([500, 1], 300, 1024), ([20, 5, 9], 40, 1024),
                                        ([9, 5, 0, 14, 7], 70, 1024), ([170, 3], 9000, 1024)])
def test_rows_out_of_range_give_zeros(counts, N, K):
    """Also where such a slot's row scale is no number."""
    p = Problem(counts, N, K, R=6, seed=4, weighted=True, invalid=True)
    want = p.run()
    p.check(want)
    bad = (p.rows < 0) | (p.rows >= 6)
    assert bad.any() and not want[bad].any()
    p.row_scale[bad] = np.where(np.arange(bad.sum()) % 2 == 0, np.nan, np.inf)
    got = p.run()
    assert (got == want).all()


@pytest.mark.gpu
def test_slots_before_and_behind_are_left_alone():
    for counts, K in (([2, 0, 3], 256), ([70, 20, 90], 256), ([70, 20, 90], 1024)):
        p = Problem(counts, 33, K, R=4, seed=5, lead=5, spare=21)
        p.check(p.run())
    p = Problem([0, 0], 8, 128, R=4, seed=5, spare=9)          # no expert has a slot
    assert (p.run() == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("off", [[-5, 3, 999], [6, 2, 4], [0, 2 ** 31 - 1, -2 ** 31],
                                 [2 ** 31 - 1] * 3, [-2 ** 31] * 3])
@pytest.mark.parametrize("T,K", [(10, 256), (200, 1024)])
def test_bad_offsets_stay_inside(off, T, K):
    """Contents that are no offsets: whatever y then is, its guard rows keep
    their values."""
    N = 20
    p = Problem([T // 2, T // 2], N, K, R=3, seed=6)
    d = p.device()
    d["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
    big = torch.full((T + 64, N), 7.0, device="cuda")
    pq2.pq2_gemm_grouped(y=big[32:32 + T], **d)
    torch.cuda.synchronize()
    assert (big[:32] == 7).all() and (big[32 + T:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 4, 16, 70, 300])
def test_one_expert_is_pq2_gemm(M):
    """A single expert's product against pq2_gemm's of the same operands."""
    N, K = 200, 2048
    p = Problem([M], N, K, seed=8)
    d = p.device()
    y = torch.empty(M, N, device="cuda")
    pq2.pq2_gemm(d["q"], d["s"], d["t"], d["codes"][0], d["wscale"][0], y)
    ref, tabs = p.reference()
    got = p.run()
    assert (np.abs(got - y.cpu().double().numpy()) <= 2 * (p.G + 4) * U * tabs).all()


# counts, N, K whose tiles fill the GPU, by kernel
LARGE = {
    "256x32": ([40, 13, 0, 70, 33, 1, 64, 32, 31, 5, 16, 90, 48, 47, 49, 100], 2500, 1024),
    "256x128": ([500, 385, 130, 33, 64, 0, 65, 400], 8500, 1024),
    "64x64": ([130, 64, 3, 200], 3000, 640),
    "stream": ([1, 2, 4, 0, 3, 5, 1, 1] * 4, 4100, 4096),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(LARGE))
def test_large_shapes(name):
    """Every expert's slots against pq2_gemm on the gathered rows: equal with
    unit scales, and within both bounds (on sampled columns) with real ones."""
    counts, N, K = LARGE[name]
    print(f"gemm_grouped large {name}", flush=True)
    for unit in (True, False):
        p = Problem(counts, N, K, R=77, seed=21, unit=unit)
        d = p.device()
        y = torch.full((p.T, N), 7.0, device="cuda")
        pq2.pq2_gemm_grouped(y=y, **d)
        for e in range(p.E):
            lo, hi = int(p.off[e]), int(p.off[e + 1])
            if lo == hi:
                continue
            at = d["rows"][lo:hi].long()
            want = torch.empty(hi - lo, N, device="cuda")
            pq2.pq2_gemm(d["q"][at], d["s"][at], d["t"][at], d["codes"][e], d["wscale"][e], want)
            if unit:
                assert torch.equal(y[lo:hi], want), (name, e)
        if not unit:
            keep = np.random.default_rng(1).permutation(N)[:60]
            keep[:3] = 0, N - 1, N // 2
            p.codes, p.ws, p.N = p.codes[:, keep], p.ws[:, keep], len(keep)
            p.check(y.cpu().double().numpy()[:, keep])


@pytest.mark.gpu
def test_gathered_rows_past_31_bits():
    """Activations beyond 2^31 bytes: the rows at the end and beyond it against
    the same rows in a small array."""
    K, N = 16384, 50
    R = (1 << 31) // K + 40
    print(f"gemm_grouped {R} x {K} activations", flush=True)
    p = Problem([3, 0, 5, 30], N, K, R=60, seed=12, weighted=True, invalid=True)
    d = p.device()
    q = torch.zeros(R, K, dtype=torch.int8, device="cuda")
    s, t = torch.zeros(R, K // 128, device="cuda"), torch.zeros(R, K // 128, dtype=torch.int32, device="cuda")
    q[R - 60:], s[R - 60:], t[R - 60:] = d["q"], d["s"], d["t"]
    rows = d["rows"]
    good = (rows >= 0) & (rows < 60)
    d.update(q=q, s=s, t=t, rows=torch.where(good, rows + (R - 60), torch.full_like(rows, -1)))
    y = torch.full((p.T, N), 7.0, device="cuda")
    pq2.pq2_gemm_grouped(y=y, **d)
    p.check(y.cpu().double().numpy())


@pytest.mark.gpu
def test_repeats_and_streams_and_graph_replays():
    """Identical y on repeats; a captured call replayed with other sizes."""
    repeats_and_streams_and_graph_replays(640, 1)
    repeats_and_streams_and_graph_replays(1024, 10)


def repeats_and_streams_and_graph_replays(K, times):
    p = Problem([5 * times, 0, 40 * times, 3 * times], 100, K, R=12, seed=10, weighted=True)
    a = p.run()
    assert (a == p.run()).all()
    st = torch.cuda.Stream()
    y = torch.full((p.T, p.N), 7.0, device="cuda")
    d = p.device()
    st.wait_stream(torch.cuda.current_stream())
    pq2.pq2_gemm_grouped(y=y, stream=st, **d)
    torch.cuda.synchronize()
    assert (y.cpu().double().numpy() == a).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pq2.pq2_gemm_grouped(y=y, **d)
    for counts in ([48, 0, 0, 0], [1, 2, 3, 4], [0, 0, 0, 48], [16, 16, 0, 16]):
        counts = [c * times for c in counts]
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        d["offsets"].copy_(torch.from_numpy(off))
        y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        p.counts, p.off = counts, off
        p.check(y.cpu().double().numpy())


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Weights beyond 4 GiB and outputs beyond 2^31 elements: the last expert's
    slots and columns against a small call on the same operands."""
    E, N, K = 40, 1 << 17, 3840                  # 5 GB of codes
    print("gemm_grouped 5 GB of codes", flush=True)
    b = torch.randint(0, 81, (N, K // 4), device="cuda", dtype=torch.int32)
    codes1 = torch.zeros_like(b, dtype=torch.uint8)
    for k in range(4):
        codes1 |= ((b // 3 ** k % 3) << (2 * k)).to(torch.uint8)
    codes = codes1.repeat(E, 1, 1)
    codes[E - 1] = codes1.flip(0)
    ws = torch.full((E, N, K // 128), 0.05, dtype=torch.float16, device="cuda")
    q, s, t = pq2.quantize_act(torch.randn(3, K, device="cuda"))
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E - 1], off[E] = 1, 3
    off[1:E - 1] = 1
    y = torch.empty(3, N, device="cuda")
    pq2.pq2_gemm_grouped(q, s, t, codes, ws, off, y)
    want = torch.empty(3, N, device="cuda")
    pq2.pq2_gemm_grouped(q, s, t, codes1[None].contiguous(), ws[:1], off[[0, E]].contiguous(), want)
    assert torch.equal(y[0], want[0])
    assert torch.equal(y[1:], want[1:].flip(1))
    del codes, ws, codes1, b
    T, N, K = 70000, 40000, 128                  # 2.8e9 outputs
    print("gemm_grouped 2.8e9 outputs", flush=True)
    p = Problem([1, 1], N, K, seed=2)
    d = p.device()
    q, s, t = pq2.quantize_act(torch.randn(64, K, device="cuda"))
    rows = (torch.arange(T, device="cuda") % 64).to(torch.int32)
    off = torch.tensor([0, 100, T], dtype=torch.int32, device="cuda")
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    pq2.pq2_gemm_grouped(q, s, t, d["codes"], d["wscale"], off, y, rows=rows)
    tail = torch.empty(64, N, dtype=torch.bfloat16, device="cuda")
    pq2.pq2_gemm_grouped(q, s, t, d["codes"], d["wscale"],
                         torch.tensor([0, 0, 64], dtype=torch.int32, device="cuda"), tail,
                         rows=rows[T - 64:].contiguous())
    err = (y[T - 64:].float() - tail.float()).abs()
    assert (err <= tail.float().abs() * 2.0 ** -7 + 1e-6).all()


@pytest.mark.gpu
def test_binding_checks_on_the_gpu():
    p = Problem([2, 1], 8, 256, R=4, seed=1)
    d = p.device()
    y = torch.empty(3, 8, device="cuda")
    for key, bad in (("rows", d["rows"].long()), ("offsets", d["offsets"].long())):
        with pytest.raises(TypeError):
            pq2.pq2_gemm_grouped(y=y, **{**d, key: bad})
    for key, bad in (("rows", d["rows"][:2]), ("offsets", d["offsets"][:2]),
                     ("offsets", d["offsets"].cpu()), ("row_scale", torch.ones(4, device="cuda")),
                     ("codes", d["codes"].transpose(0, 1))):
        with pytest.raises(ValueError):
            pq2.pq2_gemm_grouped(y=y, **{**d, key: bad})
    with pytest.raises(pq2.PQ2Error):       # without rows every slot needs its row
        pq2.pq2_gemm_grouped(y=torch.empty(9, 8, device="cuda"), **{**d, "rows": None})
    empty = torch.empty(0, 8, device="cuda")
    pq2.pq2_gemm_grouped(y=empty, **{**d, "rows": None})


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[1, 0, 2, 3], [1] * 40])
@pytest.mark.parametrize("N", [1, 16, 31, 33])
@pytest.mark.parametrize("G", [1, 2, 3, 5, 6, 7, 9, 41])
def test_groups_at_the_end_of_the_last_expert(G, N, counts):
    """Few slots an expert, groups that are no multiple of four: exact with unit
    scales whatever stands behind the codes and scales of the last expert."""
    p = Problem(counts, N, 128 * G, seed=G + N, unit=True)
    d = p.device()
    codes = torch.full((p.codes.size + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    codes[:p.codes.size] = d["codes"].view(-1)
    ws = torch.full((p.ws.size + 4096,), float("nan"), dtype=torch.float16, device="cuda")
    ws[:p.ws.size] = d["wscale"].view(-1)
    y = torch.full((p.T, N), 7.0, device="cuda")
    pq2.pq2_gemm_grouped(**{**d, "codes": codes[:p.codes.size].view(p.codes.shape),
                            "wscale": ws[:p.ws.size].view(p.ws.shape)}, y=y)
    p.check(y.cpu().double().numpy(), exact=True)
