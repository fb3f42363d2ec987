"""Memory that the binding allocates for a call on a stream of its own.

A block of torch's allocator is free to use at once on the stream whose pool it
comes from, even while that stream's earlier work on it is pending, and on no
other. So what a call on `stream` needs (an "auto" workspace) has to come from
that stream's pool: a block of the current stream's pool may still be read or
written by work that nothing orders before the call.
"""

import pytest
import torch

pq2 = pytest.importorskip("gemm_pq2_w2a8_amd")


# ------------------------------------------------------------------ where it comes from (CPU)

class Memory(torch.Tensor):
    """A tensor that passes for a GPU's and notes record_stream calls."""
    is_cuda = True

    def record_stream(self, stream):
        LOG.append(("record", stream))


LOG = []


class On:
    """torch.cuda.stream's stand-in: the streams entered are on the stack."""
    stack = []

    def __init__(self, stream):
        self.stream = stream

    def __enter__(self):
        On.stack.append(self.stream)

    def __exit__(self, *_):
        On.stack.pop()


class Stream:
    """torch.cuda.Stream's stand-in."""


@pytest.fixture
def allocations(monkeypatch):
    """The stream (None: the current one) that every torch.empty was made on."""
    made, empty = [], torch.empty

    def note(*shape, dtype=None, device=None):
        made.append(On.stack[-1] if On.stack else None)
        return empty(*shape, dtype=dtype).as_subclass(Memory)

    LOG.clear()
    monkeypatch.setattr(torch, "empty", note)
    monkeypatch.setattr(torch, "empty_like", lambda x: note(x.shape, dtype=x.dtype))
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda handle, device=None: ("external", handle, device))
    return made


def test_workspace_comes_from_the_launch_streams_pool(allocations):
    st = Stream()
    for stream, want in ((None, None), (st, st), (12345, ("external", 12345, "cuda:0"))):
        allocations.clear()
        ptr, n, keep = pq2._workspace("auto", 2, 128, 8, "cuda:0", stream, lambda *_: 640)
        assert (ptr, n) == (keep.data_ptr(), 640)
        assert allocations == [want]
    assert pq2._workspace("auto", 2, 128, 8, "cuda:0", st, lambda *_: 0) == (0, 0, None)
    assert pq2._workspace(None, 2, 128, 8, "cuda:0", st) == (0, 0, None)


def test_a_stream_of_another_gpu_is_refused(monkeypatch):
    """Before anything is launched; the stream's handle goes on as it is."""
    st, seen = Stream(), []
    st.device_index, st.cuda_stream = 1, 77
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    call = lambda *a: seen.append(a) or 0               # noqa: E731
    with pytest.raises(ValueError, match="stream must be on cuda:0, got cuda:1"):
        pq2._launch(0, st, call, 5)
    assert seen == []
    pq2._launch(1, st, call, 5)
    assert seen == [(5, 77)]
    x = torch.zeros(1).as_subclass(Memory)
    monkeypatch.setattr(Memory, "get_device", lambda self: 0, raising=False)
    with pytest.raises(ValueError, match="stream must be on cuda:0, got cuda:1"):
        pq2._stream(x, st)
    assert pq2._stream(x, 99) == 99


# ------------------------------------------------------------------ beside pending work (GPU)

def block_with_pending_copy(nbytes, busy):
    """A copy of 7s that waits on the current stream behind other work, from a
    block of `nbytes` that has gone back to the current stream's pool."""
    src = torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda")
    dst = torch.zeros_like(src)
    torch.cuda.synchronize()
    for _ in range(20):
        torch.mm(busy, busy)
    dst.copy_(src)
    return dst


def unordered(call, nbytes, want):
    """call(stream) on a stream that nothing orders behind the current one's
    pending copy: the copy and the call's results are both right."""
    busy = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    for _ in range(2):                                  # the first call fills the stream's pool
        torch.cuda.synchronize()
        copies = [block_with_pending_copy(n, busy) for n in nbytes]
        got = call(st)
        st.synchronize()
        torch.cuda.synchronize()
        assert all(bool((c == 7).all()) for c in copies)
        for g, w in zip(got, want):
            assert torch.equal(g, w)


def lora(M=40, K=5120, N=300, R=64, L=3):
    g = torch.Generator().manual_seed(5)
    d = lambda v: v.cuda()                              # noqa: E731
    x = d(torch.randn(M, K, generator=g).bfloat16())
    a, b = d(torch.randn(L, R, K, generator=g).bfloat16()), d(torch.randn(L, N, R, generator=g).bfloat16())
    ids = d(torch.randint(0, L, (M,), generator=g).to(torch.int32))
    return x, a, b, ids, d(torch.randn(M, N, generator=g))


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
def test_lora_add_workspace_beside_pending_work(raw):
    x, a, b, ids, base = lora()
    want, y = torch.empty_like(base), torch.empty_like(base)
    pq2.pq2_lora_add(x, a, b, ids, want, base=base)

    def call(st):
        pq2.pq2_lora_add(x, a, b, ids, y, base=base, stream=st.cuda_stream if raw else st)
        return [y]

    print(f"lora_add beside pending work raw={raw}", flush=True)
    unordered(call, [pq2.lora_workspace_bytes(40, 5120, 64)] * 2, [want])


@pytest.mark.gpu
def test_lora_add_workspace_in_a_capture_on_its_stream():
    """The capturing stream given by name: the replays, among eager calls on other
    streams, leave the eager result."""
    x, a, b, ids, base = lora()
    want, y = torch.empty_like(base), torch.zeros_like(base)
    pq2.pq2_lora_add(x, a, b, ids, want, base=base)
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        pq2.pq2_lora_add(x, a, b, ids, y, base=base, stream=st)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        pq2.pq2_lora_add(x, a, b, ids, y, base=base, stream=st)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,linear", [(16, 300, 17408, False), (600, 17300, 5120, False),
                                          (8, 300, 17408, True)])
def test_split_k_workspace_beside_pending_work(M, N, K, linear):
    import pq2_synth as synth
    x = torch.from_numpy(synth.activations(M, K, 3, outlier_frac=0.0)).cuda()
    w = synth.weights(N, K, synth.matrix_seed(3))
    cd = torch.from_numpy(w.codes).cuda()
    wd = torch.from_numpy(w.wscale_bits.view("int16")).cuda()
    y, want = (torch.empty(M, N, device="cuda") for _ in range(2))
    if linear:
        n = pq2.linear_workspace_bytes(M, N, K)
        run = lambda o, st: pq2.pq2_linear(x, cd, wd, o, stream=st)              # noqa: E731
    else:
        q, s, t = pq2.quantize_act(x)
        n = pq2.gemm_workspace_bytes(M, N, K)
        run = lambda o, st: pq2.pq2_gemm(q, s, t, cd, wd, o, stream=st)          # noqa: E731
    print(f"split K beside pending work M={M} N={N} K={K} linear={linear} bytes={n}", flush=True)
    assert n > 0
    run(want, None)

    def call(st):
        run(y, st)
        return [y]

    unordered(call, [n] * 2, [want])


# ------------------------------------------------------------------ tensors that helpers return

def test_returned_tensors_come_from_the_launch_streams_pool(allocations, monkeypatch):
    """q/s/t, h and y are written on the launch stream, so they come from its pool;
    the caller's stream reads them, so they are recorded there."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: ("current", str(device)))
    for name in ("pq2_quantize_act", "pq2_norm_quantize", "pq2_gemm", "pq2_linear"):
        monkeypatch.setattr(pq2, name, lambda *a, **k: None)
    codes, ws = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.int16)
    x = torch.zeros(3, 256)
    st = Stream()
    calls = [(lambda s: pq2.quantize_act(x, stream=s), 3, 3),
             (lambda s: pq2.norm_quantize(x, w_pre=x[0], stream=s), 4, 4),
             (lambda s: pq2.linear(x[:1], codes, ws, stream=s), 1, 1),
             (lambda s: pq2.linear(x, codes, ws, stream=s), 4, 1),      # q/s/t stay inside
             (lambda s: pq2.linear(x, codes, ws, out=torch.zeros(3, 4), stream=s), 3, 0)]
    for call, count, returned in calls:
        for stream, want in ((None, None), (st, st), (7, ("external", 7, x.device))):
            allocations.clear(), LOG.clear()
            call(stream)
            assert allocations == [want] * count
            assert LOG == [("record", ("current", "cpu"))] * (returned if stream is not None else 0)


@pytest.mark.gpu
def test_helpers_beside_pending_work():
    M, K, N = 64, 5120, 1024
    g = torch.Generator().manual_seed(6)
    x = torch.randn(M, K, generator=g).cuda()
    w = torch.randn(K, generator=g).cuda()
    cd = torch.randint(0, 256, (N, K // 4), generator=g, dtype=torch.uint8).cuda()
    wd = (torch.rand(N, K // 128, generator=g) + 0.5).half().cuda()
    sizes = [M * K * 4, M * K, M * (K // 128) * 4, M * N * 4]
    for name, run in (("quantize_act", lambda s: pq2.quantize_act(x, stream=s)),
                      ("norm_quantize", lambda s: pq2.norm_quantize(x, w_pre=w, stream=s)),
                      ("linear", lambda s: [pq2.linear(x, cd, wd, stream=s)]),
                      ("linear one row", lambda s: [pq2.linear(x[:1], cd, wd, stream=s)])):
        print(f"{name} beside pending work", flush=True)
        want = [v.clone() for v in run(None)]
        unordered(run, sizes, want)


@pytest.mark.gpu
def test_returned_tensors_outlive_the_callers_pending_reads():
    """q of a call on another stream, read on the current one behind long work and
    dropped: the next call on that stream leaves what is still to be read alone."""
    g = torch.Generator().manual_seed(7)
    x = [torch.randn(64, 5120, generator=g).cuda() for _ in range(2)]
    want = pq2.quantize_act(x[0])[0].clone()
    busy = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
    st, copy = torch.cuda.Stream(), torch.zeros_like(want)
    print("returned tensors and pending reads", flush=True)
    for _ in range(2):
        torch.cuda.synchronize()
        q = pq2.quantize_act(x[0], stream=st)[0]
        torch.cuda.current_stream().wait_stream(st)
        for _ in range(20):
            torch.mm(busy, busy)
        copy.copy_(q)
        del q
        pq2.quantize_act(x[1], stream=st)
        torch.cuda.synchronize()
        assert torch.equal(copy, want)
