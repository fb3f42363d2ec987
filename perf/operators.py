"""Measured cases of the operators around the PQ2_0 product.

Three operators: ``norm_quantize`` (norms after and before a block with its gate
and residual scale, ending in the int8 quantiser), ``gemm_grouped`` (products
grouped by expert with ragged sizes) and ``lora_add`` (low-rank adapters of many
requests beside a shared projection). ``listed()`` names the cases, ``draw()``
gives more of the same ranges, ``prepare()`` makes a case's inputs from a seed,
``run()`` is one pass: in elementary torch operations, or through the
framework's kernels where ``own`` is set. ``exact()`` evaluates the operator's
definition in float64.
"""

import random

import torch

own = False

GROUP = 128
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6

# ------------------------------------------------------------------ cases


def listed():
    return [
        # one token between two blocks of the 5120-wide model: add the block's
        # output to the residual stream, normalise, quantise for the next projection
        _norm("norm one token", M=1, K=5120, dtype="bf16"),
        # a decode batch with a sandwich norm, a gate per token and a scaled
        # residual; the normalised rows also go out unquantised, as adapters read them
        _norm("norm decode batch gated", M=16, K=6144, dtype="f16", post=True, gate=16, alpha=0.25,
              n_out=True),
        # an odd number of MLP-wide float32 rows, one gate for all of them
        _norm("norm wide float32", M=333, K=17408, dtype="f32", gate=1, residual=False),
        # a long prompt through a sandwich norm
        _norm("norm prompt", M=4096, K=5120, dtype="bf16", post=True, alpha=0.5),
        # one token through the 8 experts its router chose of 64 (gate / up product)
        _grouped("experts one token", T=8, R=1, E=64, N=2048, K=5120, skew=0.0, y="bf16"),
        # 16 tokens x 8 experts through the narrow down product, weighted by the router
        _grouped("experts decode batch", T=128, R=128, E=64, N=5120, K=1024, skew=0.7, y="f32",
                 weighted=True),
        # odd sizes, few experts, uneven shares
        _grouped("experts odd sizes", T=1003, R=511, E=7, N=1411, K=896, skew=1.0, y="f32"),
        # a prompt of 2048 tokens x 8 experts of 64, uneven shares
        _grouped("experts prompt", T=16384, R=2048, E=64, N=2048, K=5120, skew=0.4, y="bf16"),
        # one token of a request with an adapter beside the 5120 -> 6144 projection
        _lora("adapter one token", M=1, K=5120, N=6144, R=16, L=32, used=1, dtype="bf16", y="f32"),
        # 16 requests, each with its own adapter of its own rank, beside the MLP's first product
        _lora("adapters decode batch", M=16, K=5120, N=17408, R=64, L=48, used=16, dtype="f16",
              y="bf16", ragged=True),
        # prompts and single tokens in one batch, some rows without an adapter, odd widths
        _lora("adapters mixed batch", M=555, K=17408, N=5119, R=32, L=16, used=11, dtype="bf16",
              y="f32", bare=True, ragged=True),
        # four prompts of 1024 tokens, each with its adapter
        _lora("adapters prompt", M=4096, K=5120, N=17408, R=64, L=8, used=4, order="requests",
              dtype="bf16", y="bf16"),
    ]


def _norm(name, M, K, dtype, post=False, pre=True, gate=0, alpha=1.0, residual=True, n_out=False):
    """gate: rows of the gate (0: none; they divide M)."""
    c = {"op": "norm_quantize", "M": M, "K": K, "dtype": dtype, "post": post, "pre": pre,
         "gate": gate, "alpha": alpha, "residual": residual, "n_out": n_out}
    return {"name": name, **c} if name else c


def _grouped(name, T, R, E, N, K, skew, y, weighted=False):
    """T slots of E experts gathered from R token rows; the experts' shares fall
    off as rank ** -skew."""
    c = {"op": "gemm_grouped", "T": T, "R": R, "E": E, "N": N, "K": K, "skew": skew, "y": y,
         "weighted": weighted}
    return {"name": name, **c} if name else c


def _lora(name, M, K, N, R, L, used, dtype, y, order="rows", bare=False, ragged=False):
    """used: adapters in use of L; order: rows of one request together
    ("requests") or interleaved ("rows"); bare: every fifth row has no adapter."""
    c = {"op": "lora_add", "M": M, "K": K, "N": N, "R": R, "L": L, "used": used, "dtype": dtype,
         "y": y, "order": order, "bare": bare, "ragged": ragged}
    return {"name": name, **c} if name else c


def _log(rng, lo, hi):
    return min(hi, int(lo * (hi / lo) ** rng.random() + 0.5))


def draw(rng: random.Random):
    op = rng.choice(("norm_quantize", "gemm_grouped", "lora_add"))
    if op == "norm_quantize":
        K = GROUP * _log(rng, 1, 136)
        M = _log(rng, 1, min(4096, max(1, 4096 * 5120 // K)))
        gates = [0, 1, M] + [d for d in (2, 3, 4, 5, 8) if M % d == 0]
        return _norm(None, M, K, rng.choice(("bf16", "f16", "f32")), post=rng.random() < 0.5,
                     pre=rng.random() < 0.8, gate=rng.choice(gates),
                     alpha=round(rng.uniform(0.1, 2.0), 3), residual=rng.random() < 0.8,
                     n_out=rng.random() < 0.5)
    if op == "gemm_grouped":
        E = _log(rng, 2, 128)
        K = GROUP * _log(rng, 1, 40)
        N = _log(rng, 16, min(4096, 64 * 2048 * 5120 // (E * K)))
        T = _log(rng, 1, 16384)
        return _grouped(None, T, rng.randint(1, min(T, 4096)), E, N, K,
                        round(rng.uniform(0.0, 1.0), 2), rng.choice(("bf16", "f32")),
                        weighted=rng.random() < 0.5)
    L = _log(rng, 1, 64)
    K = GROUP * _log(rng, 1, 136)
    N = _log(rng, 8, 17408)
    M = _log(rng, 1, min(4096, 4096 * 22528 // (K + N)))
    return _lora(None, M, K, N, 8 * rng.randint(1, 8), L, rng.randint(1, min(L, M)),
                 rng.choice(("bf16", "f16")), rng.choice(("bf16", "f32")),
                 order=rng.choice(("rows", "requests")), bare=rng.random() < 0.3,
                 ragged=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs


def _shares(case):
    """Slots per expert rank: the T slots dealt by rank ** -skew, largest remainders first."""
    T, E = case["T"], case["E"]
    w = [(e + 1.0) ** -case["skew"] for e in range(E)]
    exact_share = [T * v / sum(w) for v in w]
    n = [int(v) for v in exact_share]
    order = sorted(range(E), key=lambda e: (n[e] - exact_share[e], e))
    for e in order[: T - sum(n)]:
        n[e] += 1
    return n


def _rank(case, l):
    """Rank of adapter l: R, or one of 1 .. R in turn."""
    return case["R"] if not case["ragged"] else case["R"] - (5 * l) % case["R"]


def _rows_of(case):
    """Index among the used adapters of every row (-1: none)."""
    M, used = case["M"], case["used"]
    if case["order"] == "requests":
        at = [i * used // M for i in range(M)]
    else:
        at = [i % used for i in range(M)]
    return [-1 if case["bare"] and i % 5 == 3 else a for i, a in enumerate(at)]


def _codes(g, *shape):
    """Packed ternary codes, each of 0, 1, 2 with the same probability."""
    b = torch.zeros(shape, dtype=torch.uint8, device=DEV)
    for k in range(4):
        b |= torch.randint(0, 3, shape, dtype=torch.uint8, device=DEV, generator=g) << (2 * k)
    return b


def _plane_order(v):
    """Natural to plane order inside each group: element 4 b + s to 32 s + b."""
    return v.reshape(v.shape[0], -1, 32, 4).transpose(2, 3).reshape(v.shape)


def _quantised(x):
    """int8 activations in plane order, scales and group sums of float32 rows."""
    v = x.reshape(x.shape[0], -1, GROUP)
    s = v.abs().amax(-1) / 127.0
    q = torch.where(s[..., None] > 0, (v / s[..., None]).round().clamp(-127, 127), 0.0)
    t = q.sum(-1).to(torch.int32)
    return _plane_order(q.to(torch.int8).reshape(x.shape)).contiguous(), s.contiguous(), t.contiguous()


def _randn(g, *shape, outliers=0.0):
    x = torch.randn(shape, device=DEV, generator=g)
    if outliers:
        x *= torch.where(torch.rand(shape, device=DEV, generator=g) < outliers, 10.0, 1.0)
    return x


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "norm_quantize":
        M, K, ty = case["M"], case["K"], TYPES[case["dtype"]]
        st["x"] = _randn(g, M, K, outliers=0.01).to(ty)
        st["residual"] = (2 * _randn(g, M, K)).to(ty) if case["residual"] else None
        st["w_post"] = 1 + 0.2 * _randn(g, K) if case["post"] else None
        st["w_pre"] = 1 + 0.2 * _randn(g, K) if case["pre"] else None
        st["gate"] = torch.sigmoid(_randn(g, case["gate"], K)).to(ty) if case["gate"] else None
        # output buffers, as a serving loop keeps them
        st["h"] = torch.empty(M, K, dtype=ty, device=DEV)
        st["n"] = torch.empty(M, K, dtype=ty, device=DEV) if case["n_out"] else None
        st["q"] = torch.empty(M, K, dtype=torch.int8, device=DEV)
        st["s"] = torch.empty(M, K // GROUP, dtype=torch.float32, device=DEV)
        st["t"] = torch.empty(M, K // GROUP, dtype=torch.int32, device=DEV)
        st["values"] = torch.empty(M, K // GROUP, 32, 4, dtype=torch.bfloat16, device=DEV)
        st["sums"] = torch.empty(M, K // GROUP, dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "gemm_grouped":
        T, R, E, N, K = (case[k] for k in "TRENK")
        st["q"], st["s"], st["t"] = _quantised(_randn(g, R, K, outliers=0.01))
        st["codes"] = _codes(g, E, N, K // 4)
        ws = 0.01 + 0.09 * torch.rand(E, N, K // GROUP, device=DEV, generator=g)
        st["wscale"] = ws.to(torch.float16)
        counts = torch.tensor(_shares(case), device=DEV)
        counts = counts[torch.randperm(E, device=DEV, generator=g)]
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        st["rows"] = torch.randint(0, R, (T,), device=DEV, generator=g, dtype=torch.int32)
        st["row_scale"] = torch.rand(T, device=DEV, generator=g) if case["weighted"] else None
        st["most"] = max(_shares(case))   # rows of the busiest expert, a plan's bound
        st["y"] = torch.empty(T, N, dtype=TYPES[case["y"]], device=DEV)
    else:
        M, K, N, R, L = (case[k] for k in "MKNRL")
        ty = TYPES[case["dtype"]]
        st["x"] = _randn(g, M, K, outliers=0.01).to(ty)
        st["a"] = (_randn(g, L, R, K) / K ** 0.5).to(ty)
        st["b"] = (_randn(g, L, N, R) / R ** 0.5).to(ty)
        st["ranks"] = torch.tensor([_rank(case, l) for l in range(L)], dtype=torch.int32, device=DEV)
        st["scale"] = 0.5 + torch.rand(L, device=DEV, generator=g)
        pick = torch.cat([torch.randperm(L, device=DEV, generator=g)[: case["used"]],
                          torch.full((1,), -1, device=DEV)])
        st["adapter"] = pick[torch.tensor(_rows_of(case), device=DEV)].to(torch.int32)
        st["base"] = (2 * _randn(g, M, N)).to(TYPES[case["y"]])
        st["y"] = torch.empty(M, N, dtype=TYPES[case["y"]], device=DEV)
    return st


# ------------------------------------------------------------------ one pass


def run(state):
    return _RUN[state["case"]["op"]](state)


def _rms(v, w):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * w


def _run_norm(st):
    case = st["case"]
    M, K = case["M"], case["K"]
    if own:
        import gemm_pq2_w2a8_amd as pq2
        pq2.pq2_norm_quantize(st["x"], st["q"], st["s"], st["t"], residual=st["residual"],
                              w_post=st["w_post"], gate=st["gate"], alpha=case["alpha"],
                              w_pre=st["w_pre"], eps=EPS, h=st["h"], n=st["n"])
        # the int8 rows as the values they stand for
        q = st["q"].view(M, -1, 4, 32).transpose(2, 3)
        torch.mul(q, st["s"].view(M, -1, 1, 1), out=st["values"])
        torch.mul(st["t"], st["s"], out=st["sums"])
        out = {"h": st["h"], "values": st["values"].view(M, K), "s": st["s"], "sums": st["sums"]}
        return {**out, "n": st["n"]} if case["n_out"] else out
    ty = st["x"].dtype
    p = st["x"].float()
    if case["post"]:
        p = _rms(p, st["w_post"])
    if case["gate"]:
        p = (p.view(case["gate"], -1, K) * st["gate"].float()[:, None, :]).view(M, K)
    h = case["alpha"] * p
    if case["residual"]:
        h = h + st["residual"].float()
    n = _rms(h, st["w_pre"]) if case["pre"] else h
    v = n.view(M, -1, GROUP)
    s = v.abs().amax(-1) / 127.0
    q = torch.where(s[..., None] > 0, (v / s[..., None]).round().clamp(-127, 127), 0.0)
    out = {"h": h.to(ty), "values": (q * s[..., None]).view(M, K).to(torch.bfloat16), "s": s,
           "sums": (q.sum(-1) * s).to(torch.bfloat16)}
    return {**out, "n": n.to(ty)} if case["n_out"] else out


def _activations(st):
    """float32 activations the int8 rows stand for, in natural order."""
    q = st["q"]
    v = q.view(q.shape[0], -1, 4, 32).transpose(2, 3).reshape(q.shape[0], -1, GROUP).float()
    return (v * st["s"][..., None]).reshape(q.shape)


def _weights(codes, wscale):
    """float32 weights [..., N, K] of packed codes and scales."""
    shift = torch.arange(0, 8, 2, dtype=torch.uint8, device=codes.device)
    c = ((codes[..., None] >> shift) & 3).reshape(*codes.shape[:-1], -1, GROUP).float() - 1.0
    return (c * wscale.float()[..., None]).flatten(-2)


def _run_grouped(st):
    case = st["case"]
    if own:
        import gemm_pq2_w2a8_amd as pq2
        pq2.pq2_gemm_grouped(st["q"], st["s"], st["t"], st["codes"], st["wscale"], st["offsets"],
                             st["y"], rows=st["rows"], row_scale=st["row_scale"])
        return st["y"]
    T, E = case["T"], case["E"]
    x = _activations(st)[st["rows"].long()]
    slot = torch.arange(T, device=x.device)
    expert = torch.searchsorted(st["offsets"][1:].long(), slot, right=True)
    if T <= E:      # few rows: each with its expert's weights
        w = _weights(st["codes"][expert], st["wscale"][expert])
        y = torch.matmul(w, x[:, :, None])[:, :, 0]
    else:           # every expert's rows padded to the busiest one's
        place = slot - st["offsets"][expert].long()
        xp = x.new_zeros(E, st["most"], case["K"])
        xp[expert, place] = x
        w = _weights(st["codes"], st["wscale"]).transpose(1, 2).contiguous()
        y = torch.bmm(xp, w)[expert, place]
    if case["weighted"]:
        y = y * st["row_scale"][:, None]
    return y.to(TYPES[case["y"]])


def _run_lora(st):
    case = st["case"]
    if own:
        import gemm_pq2_w2a8_amd as pq2
        pq2.pq2_lora_add(st["x"], st["a"], st["b"], st["adapter"], st["y"], base=st["base"],
                         ranks=st["ranks"], scale=st["scale"])
        return st["y"]
    M, K, N, R, L = (case[k] for k in "MKNRL")
    x, id_ = st["x"].float(), st["adapter"].long()
    live = torch.arange(R, device=x.device) < st["ranks"][:, None]         # [L, R]
    some, at = id_ >= 0, id_.clamp(min=0)
    f = torch.where(some, st["scale"][at], 0.0)[:, None]
    if M <= L:      # few rows: each with its adapter's matrices
        v = torch.matmul(st["a"][at].float(), x[:, :, None])[:, :, 0]
        v = torch.where(live[at], v, 0.0) * f
        d = torch.matmul(st["b"][at].float(), v[:, :, None])[:, :, 0]
    else:           # all adapters side by side, each row keeping its own columns
        mine = (at[:, None] == torch.arange(L, device=x.device)) & some[:, None]
        v = torch.matmul(x, st["a"].view(L * R, K).float().t()).view(M, L, R)
        v = torch.where(mine[:, :, None] & live, v * f[:, :, None], 0.0)
        b = st["b"].float().transpose(1, 2).reshape(L * R, N)
        d = torch.matmul(v.view(M, L * R), b)
    return (st["base"].float() + d).to(TYPES[case["y"]])


_RUN = {"norm_quantize": _run_norm, "gemm_grouped": _run_grouped, "lora_add": _run_lora}

# ------------------------------------------------------------------ bounds and reference


def work(case):
    """Bytes (each input read once, each output written once) and operations of one pass."""
    if case["op"] == "norm_quantize":
        M, K = case["M"], case["K"]
        e = TYPES[case["dtype"]].itemsize
        rows = 2 + case["residual"] + case["n_out"]           # x, h, residual, n
        b = M * K * (e * rows + 1) + M * (K // GROUP) * 8 + case["gate"] * K * e
        b += 4 * K * (case["post"] + case["pre"])
        return {"bytes": b, "flops": 10 * M * K}
    if case["op"] == "gemm_grouped":
        T, R, E, N, K = (case[k] for k in "TRENK")
        live = sum(1 for n in _shares(case) if n)
        b = live * N * (K // 4 + 2 * (K // GROUP)) + min(R, T) * (K + 8 * (K // GROUP))
        b += T * N * TYPES[case["y"]].itemsize + 4 * (E + 1) + 4 * T * (1 + case["weighted"])
        return {"bytes": b, "flops": 2 * T * N * K}
    M, K, N, L = (case[k] for k in "MKNL")
    e, ye = TYPES[case["dtype"]].itemsize, TYPES[case["y"]].itemsize
    rows = _rows_of(case)
    ranks = sum(_rank(case, l) for l in range(L)) / L
    ids = len({a for a in rows if a >= 0})
    b = M * K * e + ids * ranks * (K + N) * e + 2 * M * N * ye + 4 * M + 8 * L
    return {"bytes": b, "flops": 2 * sum(a >= 0 for a in rows) * ranks * (K + N)}


def exact(case, seed):
    """The definition in float64, on the same inputs."""
    st = prepare(case, seed)
    if case["op"] == "norm_quantize":
        M, K = case["M"], case["K"]
        h = torch.zeros(M, K, dtype=torch.float64, device=DEV)
        block = st["x"].double()
        if st["w_post"] is not None:
            size = (block ** 2).sum(1) / K + EPS
            block = block / size.sqrt()[:, None] * st["w_post"].double()
        if st["gate"] is not None:
            per = M // case["gate"]
            for j in range(case["gate"]):
                block[j * per:(j + 1) * per] *= st["gate"][j].double()
        h += case["alpha"] * block
        if st["residual"] is not None:
            h += st["residual"].double()
        n = h
        if st["w_pre"] is not None:
            n = h / ((h ** 2).sum(1) / K + EPS).sqrt()[:, None] * st["w_pre"].double()
        parts = n.unflatten(1, (K // GROUP, GROUP))
        s = parts.abs().max(2).values / 127
        step = s.where(s > 0, torch.ones_like(s))[:, :, None]
        q = (parts / step).round()
        out = {"h": h, "values": (q * s[:, :, None]).flatten(1), "s": s, "sums": q.sum(2) * s}
        return {**out, "n": n} if case["n_out"] else out
    if case["op"] == "gemm_grouped":
        K, N = case["K"], case["N"]
        y = torch.zeros(case["T"], N, dtype=torch.float64, device=DEV)
        natural = torch.empty(K, dtype=torch.long, device=DEV)   # where element k is stored
        k = torch.arange(K, device=DEV)
        natural[k] = k // GROUP * GROUP + 32 * (k % 4) + k % GROUP // 4
        x = st["q"][:, natural].double() * st["s"].double().repeat_interleave(GROUP, 1)
        ends = st["offsets"].tolist()
        for e in range(case["E"]):
            if ends[e] == ends[e + 1]:
                continue
            w = torch.empty(N, K, dtype=torch.float64, device=DEV)
            for j in range(4):
                w[:, j::4] = (st["codes"][e].to(torch.int32) // 4 ** j % 4 - 1).double()
            w *= st["wscale"][e].double().repeat_interleave(GROUP, 1)
            pick = st["rows"][ends[e]:ends[e + 1]].long()
            y[ends[e]:ends[e + 1]] = x[pick] @ w.t()
        if st["row_scale"] is not None:
            y *= st["row_scale"].double()[:, None]
        return y
    y = st["base"].double()
    for l in set(st["adapter"].tolist()) - {-1}:
        r = int(st["ranks"][l])
        at = (st["adapter"] == l).nonzero()[:, 0]
        v = st["x"][at].double() @ st["a"][l, :r].double().t()
        y[at] += float(st["scale"][l]) * (v @ st["b"][l, :, :r].double().t())
    return y
