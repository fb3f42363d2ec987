"""Measured cases of the operators in microscaled 4-bit floating point (MX4).

Five operators: ``quantize`` (blocks of 32 values to 4-bit floats under one
power-of-two scale, and back), ``gemm`` (the product of two quantised
matrices), ``gemm_grad`` (the gradient of the product's input), ``gated`` (a
gated feed-forward block: both projections, the activation and the product of
the two) and ``gated_grad`` (its backward pass). ``listed()`` names the cases,
``draw()`` gives more of the same ranges, ``prepare()`` makes a case's inputs
from a seed, ``run()`` is one pass: in elementary torch operations, or through
the framework's kernels where ``own`` is set. ``exact()`` evaluates the
operator's definition in float64.
"""

import math
import random

import torch

own = False

BLOCK = 32
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("silu", "gelu", "gelu_tanh")

# ------------------------------------------------------------------ cases


def listed():
    return [
        # one token before a projection of the 5120-wide model
        _quantize("quantize one token", M=1, K=5120, dtype="bf16"),
        # a long prompt's hidden rows before the down projection
        _quantize("quantize prompt", M=4096, K=17408, dtype="bf16"),
        # one token through the 6144 -> 5120 projection
        _gemm("product one token", M=1, N=5120, K=6144, dtype="bf16"),
        # a decode batch through the down projection
        _gemm("product decode batch", M=16, N=5120, K=17408, dtype="bf16"),
        # a long prompt through the down projection
        _gemm("product prompt", M=4096, N=5120, K=17408, dtype="bf16"),
        # odd numbers of rows and columns, float32 gradients
        _gemm_grad("product gradient odd sizes", M=509, N=1411, K=896, dtype="f32"),
        # the down projection's input gradient for 4096 training tokens
        _gemm_grad("product gradient batch", M=4096, N=5120, K=17408, dtype="bf16"),
        # one token through the 5120-wide model's feed-forward block
        _gated("gated one token", M=1, F=17408, K=5120, act="silu", dtype="bf16"),
        # odd sizes, float32 out
        _gated("gated odd sizes", M=131, F=1411, K=896, act="gelu", dtype="f32"),
        # 2048 training tokens, both projections kept for the backward pass
        _gated("gated batch", M=2048, F=17408, K=5120, act="silu", dtype="bf16", keep=True),
        # odd sizes backward, float32
        _gated_grad("gated gradient odd sizes", M=131, F=1411, K=896, act="gelu_tanh", dtype="f32"),
        # the same 2048 training tokens backward
        _gated_grad("gated gradient batch", M=2048, F=17408, K=5120, act="silu", dtype="bf16"),
    ]


def _case(name, **c):
    return {"name": name, **c} if name else c


def _quantize(name, M, K, dtype):
    return _case(name, op="quantize", M=M, K=K, dtype=dtype)


def _gemm(name, M, N, K, dtype):
    """dtype: of the output."""
    return _case(name, op="gemm", M=M, N=N, K=K, dtype=dtype)


def _gemm_grad(name, M, N, K, dtype):
    """dtype: of both gradients."""
    return _case(name, op="gemm_grad", M=M, N=N, K=K, dtype=dtype)


def _gated(name, M, F, K, act, dtype, keep=False):
    """keep: both projections are returned too, as a backward pass needs them."""
    return _case(name, op="gated", M=M, F=F, K=K, act=act, dtype=dtype, keep=keep)


def _gated_grad(name, M, F, K, act, dtype):
    return _case(name, op="gated_grad", M=M, F=F, K=K, act=act, dtype=dtype)


def _log(rng, lo, hi):
    return min(hi, int(lo * (hi / lo) ** rng.random() + 0.5))


def draw(rng: random.Random):
    op = rng.choice(("quantize", "gemm", "gemm_grad", "gated", "gated_grad"))
    dtype = rng.choice(("bf16", "f16", "f32"))
    K = 128 * _log(rng, 1, 136)
    if op == "quantize":
        return _quantize(None, _log(rng, 1, min(4096, 4096 * 17408 // (2 * K))), K, dtype)
    N = _log(rng, 1, 17408)                   # outputs, or the block's width
    gated = op.startswith("gated")
    most = 2048 * 34816 * 5120 // (K * N * (2 if gated else 1))
    M = _log(rng, 1, min(4096, max(1, most)))
    if dtype == "f32":                        # three bfloat16 parts a value backward
        M = min(M, 1024)
    if op == "gemm":
        return _gemm(None, M, N, K, dtype)
    if op == "gemm_grad":
        return _gemm_grad(None, M, N, K, dtype)
    act = rng.choice(ACTS)
    if op == "gated":
        return _gated(None, M, N, K, act, dtype, keep=rng.random() < 0.5)
    return _gated_grad(None, M, N, K, act, dtype)


# ------------------------------------------------------------------ inputs


def _randn(g, *shape, outliers=0.0):
    x = torch.randn(shape, device=DEV, generator=g)
    if outliers:
        x *= torch.where(torch.rand(shape, device=DEV, generator=g) < outliers, 10.0, 1.0)
    return x


def _nearest(v):
    """|v| rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even one."""
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    return ((v / step).round() * step).clamp(max=6.0)


def _exponents(x):
    """Power of two of every block's scale: that of the largest value, less two."""
    amax = x.view(x.shape[0], -1, BLOCK).abs().amax(-1)
    e = torch.frexp(amax).exponent - 3
    return torch.where(amax > 0, e, -127).clamp(min=-127)


def _quantised(x):
    """Packed codes, scale bytes of float32 rows."""
    e = _exponents(x)
    v = torch.ldexp(x.view(x.shape[0], -1, BLOCK), -e[..., None])
    m = _nearest(v.abs())
    # 0, 0.5 .. 2 are codes 0 .. 4, then 3, 4, 6
    code = torch.where(m <= 2, 2 * m, torch.where(m == 3, 5.0, torch.where(m == 4, 6.0, 7.0)))
    code = (code + 8 * torch.signbit(v)).to(torch.uint8).view(x.shape[0], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def _weights(g, N, K):
    """Quantised rows of normal weights, made in pieces of rows."""
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(N, K // BLOCK, dtype=torch.uint8, device=DEV)
    for i in range(0, N, 8192):
        j = min(N, i + 8192)
        codes[i:j], scales[i:j] = _quantised(_randn(g, j - i, K) / K ** 0.5)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, M, K, ty = case["op"], case["M"], case["K"], TYPES[case["dtype"]]
    st = {"case": case}
    if op == "quantize":
        st["x"] = _randn(g, M, K, outliers=0.01).to(ty)
        # output buffers, as a serving loop keeps them
        st["codes"] = torch.empty(M, K // 2, dtype=torch.uint8, device=DEV)
        st["scales"] = torch.empty(M, K // BLOCK, dtype=torch.uint8, device=DEV)
        st["values"] = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
        return st
    N = case["N"] if "N" in case else case["F"]
    rows = 2 * N if op.startswith("gated") else N
    st["w"], st["ws"] = _weights(g, rows, K)
    if op in ("gemm", "gated"):
        st["a"], st["as"] = _quantised(_randn(g, M, K, outliers=0.01))
        st["y"] = torch.empty(M, N, dtype=ty, device=DEV)
        st["gu"] = torch.empty(M, rows, dtype=ty, device=DEV) if case.get("keep") else None
    else:
        st["dy"] = _randn(g, M, N).to(ty)
        st["dx"] = torch.empty(M, K, dtype=ty, device=DEV)
        if op == "gated_grad":
            st["gu"] = (1.5 * _randn(g, M, rows)).to(ty)
            st["dgu"] = torch.empty(M, rows, dtype=ty, device=DEV)
    return st


# ------------------------------------------------------------------ one pass


def run(state):
    return _RUN[state["case"]["op"]](state)


def _run_quantize(st):
    if own:
        import gemm_pq2_w2a8_amd as pq2
        pq2.pq2_mx4_quantize(st["x"], st["codes"], st["scales"])
        # the 4-bit rows as the values they stand for
        pq2.pq2_mx4_dequantize(st["codes"], st["scales"], st["values"])
        return {"values": st["values"], "exponents": st["scales"]}
    x = st["x"].float()
    e = _exponents(x)
    v = torch.ldexp(x.view(x.shape[0], -1, BLOCK), -e[..., None])
    q = torch.ldexp(torch.copysign(_nearest(v.abs()), v), e[..., None])
    return {"values": q.view(x.shape).to(torch.bfloat16), "exponents": (e + 127).to(torch.uint8)}


def _values(codes, scales):
    """float32 values of packed codes and scale bytes."""
    table = torch.tensor((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0), device=codes.device)
    table = torch.cat([table, -table])
    code = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1, BLOCK)
    v = torch.ldexp(table[code.int()], scales.int()[..., None] - 127)
    return v.view(codes.shape[0], -1)


def _run_gemm(st):
    if own:
        import gemm_pq2_w2a8_amd as pq2
        pq2.pq2_mx4_gemm(st["a"], st["as"], st["w"], st["ws"], st["y"])
        return st["y"]
    y = torch.matmul(_values(st["a"], st["as"]), _values(st["w"], st["ws"]).t())
    return y.to(st["y"].dtype)


def _run_gemm_grad(st):
    if own:
        import gemm_pq2_w2a8_amd as pq2
        pq2.pq2_mx4_gemm_grad(st["dy"], st["w"], st["ws"], st["dx"])
        return st["dx"]
    return torch.matmul(st["dy"].float(), _values(st["w"], st["ws"])).to(st["dx"].dtype)


def _act(name, g):
    if name == "silu":
        return g * torch.sigmoid(g)
    if name == "gelu":
        return 0.5 * g * torch.special.erfc(-g * math.sqrt(0.5))
    return g * torch.sigmoid(math.sqrt(8 / math.pi) * (g + 0.044715 * g * g * g))


def _act_slope(name, g):
    if name == "silu":
        s = torch.sigmoid(g)
        return s * (1 + g * (1 - s))
    if name == "gelu":
        bell = torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
        return 0.5 * torch.special.erfc(-g * math.sqrt(0.5)) + g * bell
    c = math.sqrt(8 / math.pi)
    s = torch.sigmoid(c * (g + 0.044715 * g * g * g))
    return s + g * s * (1 - s) * c * (1 + 3 * 0.044715 * g * g)


def _run_gated(st):
    case = st["case"]
    if own:
        import gemm_pq2_w2a8_amd as pq2
        pq2.pq2_mx4_gated(st["a"], st["as"], st["w"], st["ws"], st["y"], act=case["act"],
                          gu=st["gu"])
        return {"h": st["y"], "gu": st["gu"]} if case["keep"] else st["y"]
    gu = torch.matmul(_values(st["a"], st["as"]), _values(st["w"], st["ws"]).t())
    g, u = gu.chunk(2, 1)
    h = (_act(case["act"], g) * u).to(st["y"].dtype)
    return {"h": h, "gu": gu.to(h.dtype)} if case["keep"] else h


def _run_gated_grad(st):
    case = st["case"]
    if own:
        import gemm_pq2_w2a8_amd as pq2
        pq2.pq2_mx4_gated_grad(st["dy"], st["gu"], st["w"], st["ws"], st["dx"], dgu=st["dgu"],
                               act=case["act"])
        return {"dx": st["dx"], "dgu": st["dgu"]}
    g, u = st["gu"].float().chunk(2, 1)
    dh = st["dy"].float()
    dgu = torch.cat([dh * u * _act_slope(case["act"], g), dh * _act(case["act"], g)], 1)
    dx = torch.matmul(dgu, _values(st["w"], st["ws"]))
    return {"dx": dx.to(st["dx"].dtype), "dgu": dgu.to(st["dx"].dtype)}


_RUN = {"quantize": _run_quantize, "gemm": _run_gemm, "gemm_grad": _run_gemm_grad,
        "gated": _run_gated, "gated_grad": _run_gated_grad}

# ------------------------------------------------------------------ bounds and reference


def work(case):
    """Bytes (each input read once, each output written once) and operations of one pass."""
    op, M, K = case["op"], case["M"], case["K"]
    e = TYPES[case["dtype"]].itemsize
    if op == "quantize":       # x in, the quantised rows and their values out
        return {"bytes": M * K * (e + 2) + M * (K // 2 + K // BLOCK), "flops": 4 * M * K}
    N = case["N"] if "N" in case else case["F"]
    rows = 2 * N if op.startswith("gated") else N
    b = rows * (K // 2 + K // BLOCK)
    if op in ("gemm", "gated"):
        b += M * (K // 2 + K // BLOCK) + M * e * (N + (rows if case.get("keep") else 0))
    else:
        b += M * e * (N + K) + (2 * M * e * rows if op == "gated_grad" else 0)
    return {"bytes": b, "flops": 2 * M * rows * K}


def _float64(codes, scales):
    """Values by the format's fields: sign, two exponent bits, one mantissa bit."""
    out = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        c = (codes // 16 if half else codes % 16).long()
        sign, power, frac = c // 8, c // 2 % 4, (c % 2).double()
        size = torch.where(power == 0, frac / 2, (1 + frac / 2) * 2.0 ** (power - 1).double())
        out[:, half::2] = torch.where(sign == 1, -size, size)
    out *= (2.0 ** (scales.double() - 127)).repeat_interleave(BLOCK, 1)
    return out


def _product64(x, codes, scales):
    """x [M][K] times the weights' transpose, some weight rows at a time."""
    y = torch.empty(x.shape[0], codes.shape[0], dtype=torch.float64, device=x.device)
    for i in range(0, codes.shape[0], 4096):
        w = _float64(codes[i:i + 4096], scales[i:i + 4096])
        y[:, i:i + 4096] = x @ w.t()
    return y


def _gradient64(dy, codes, scales):
    """dy [M][N] times the weights, some weight rows at a time."""
    dx = torch.zeros(dy.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=dy.device)
    for i in range(0, codes.shape[0], 4096):
        dx += dy[:, i:i + 4096] @ _float64(codes[i:i + 4096], scales[i:i + 4096])
    return dx


def _act64(name, g):
    """The activation and its derivative."""
    if name == "silu":
        s = 1 / (1 + (-g).exp())
        return g * s, s + g * s * (1 - s)
    if name == "gelu":
        cdf = torch.special.ndtr(g)
        return g * cdf, cdf + g * (-g ** 2 / 2).exp() / (2 * math.pi) ** 0.5
    inner = (2 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3)
    t = inner.tanh()
    slope = (2 / math.pi) ** 0.5 * (1 + 0.134145 * g ** 2)
    return g * (1 + t) / 2, (1 + t) / 2 + g / 2 * (1 - t ** 2) * slope


def exact(case, seed):
    """The definition in float64, on the same inputs."""
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = st["x"].double().unflatten(1, (-1, BLOCK))
        top = x.abs().max(2, keepdim=True).values
        scale = 2.0 ** (top.log2().floor() - 2).clamp(min=-127)
        grid = torch.tensor((0, 0.5, 1, 1.5, 2, 3, 4, 6), dtype=torch.float64, device=DEV)
        between = (grid[1:] + grid[:-1]) / 2
        v = (x / scale).abs()
        low, high = torch.bucketize(v, between), torch.bucketize(v, between, right=True)
        at = torch.where(low % 2 == 0, low, high)     # on a border: the even code
        return {"values": (grid[at] * x.sign() * scale).flatten(1), "exponents": None}
    if op in ("gemm", "gated"):
        y = _product64(_float64(st["a"], st["as"]), st["w"], st["ws"])
        if op == "gemm":
            return y
        F = case["F"]
        h = _act64(case["act"], y[:, :F])[0] * y[:, F:]
        return {"h": h, "gu": y} if case["keep"] else h
    dy = st["dy"].double()
    if op == "gemm_grad":
        return _gradient64(dy, st["w"], st["ws"])
    F = case["F"]
    g, u = st["gu"][:, :F].double(), st["gu"][:, F:].double()
    a, slope = _act64(case["act"], g)
    dgu = torch.cat((dy * u * slope, dy * a), 1)
    return {"dx": _gradient64(dgu, st["w"], st["ws"]), "dgu": dgu}
