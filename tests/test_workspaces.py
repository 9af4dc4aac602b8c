"""The binding's own workspaces: which calls share one."""
import threading

import pytest
import torch


def in_threads(n, f):
    """[f(0), .., f(n - 1)], each in a thread of its own, all alive at once."""
    out, errors = [None] * n, []
    gate = threading.Barrier(n)

    def run(i):
        try:
            gate.wait(60)
            out[i] = f(i)
            gate.wait(60)
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(e)
            gate.abort()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    return out


# ------------------------------------------------------------------- CPU --
@pytest.fixture
def tgs_cpu(monkeypatch):
    """The binding with every tensor's stream taken to be one and the same, and not captured."""
    import top_gradient_sparsification_amd as tgs
    monkeypatch.setattr(tgs, "_stream_handle", lambda device: 7)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return tgs


def test_threads_on_one_stream_have_workspaces_of_their_own(tgs_cpu):
    cpu = torch.device("cpu")
    for get in (lambda i: tgs_cpu.workspace("threads", 1000, cpu),
                lambda i: tgs_cpu._scratch("threads", 1000, cpu, 7)):
        a, b = in_threads(2, get)
        assert a.numel() >= 1000 and b.numel() >= 1000 and a.data_ptr() != b.data_ptr()
    here = tgs_cpu.workspace("threads", 1000, cpu)
    assert tgs_cpu._scratch("threads", 900, cpu, 7) is here and tgs_cpu.workspace("threads", 1000, cpu) is here
    assert tgs_cpu.workspace("threads", 2000, cpu) is not here  # it grows
    assert not here.any()


def test_a_call_under_capture_leaves_the_kept_workspace_alone(tgs_cpu, monkeypatch):
    """A graph writes to its workspace at every replay: one that a larger call
    later replaces, and frees, must not be it."""
    cpu = torch.device("cpu")
    kept = tgs_cpu.workspace("capture", 40_000, cpu)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    for get in (lambda: tgs_cpu.workspace("capture", 40_000, cpu), lambda: tgs_cpu._scratch("capture", 40_000, cpu, 7)):
        buf = get()
        assert buf.data_ptr() != kept.data_ptr() and buf.numel() >= 40_000 and not buf[:32768].any()
        assert get() is not buf
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    assert tgs_cpu.workspace("capture", 40_000, cpu) is kept


def test_a_workspace_on_another_device_is_refused(tgs_cpu):
    with pytest.raises(ValueError, match="ws is on cpu, expected cuda:0"):
        tgs_cpu._require_ws(torch.zeros(32768, dtype=torch.uint8), torch.device("cuda", 0))
    with pytest.raises(TypeError, match="ws"):
        tgs_cpu._require_ws(b"0" * 32768, torch.device("cuda", 0))
    with pytest.raises(ValueError, match="contiguous"):
        tgs_cpu._require_ws(torch.zeros(9, 9)[:, 0], torch.device("cpu"))


# ------------------------------------------------------------------- GPU --
@pytest.mark.gpu
def test_two_threads_on_one_stream_get_what_one_gets(tgs_gpu):
    """Sequences of launches, enqueued by two threads at once on the stream they share."""
    T, V, D, rounds = 20_000, 3_000, 64, 25

    def inputs(i):
        gen = torch.Generator(device="cuda").manual_seed(i)
        return (torch.randint(-1, V, (T,), device="cuda", generator=gen), torch.randn(T, D, device="cuda", generator=gen),
                torch.randn(200, 300, device="cuda", generator=gen), torch.randn(60, 700, device="cuda", generator=gen))

    def work(given):
        tokens, grad, wide, small = given
        weight, momentum = wide.clone(), torch.zeros_like(wide)
        for _ in range(rounds):
            tgs_gpu.muon_step(weight, wide, momentum, lr=0.1)
            g = tgs_gpu.embedding_grad(tokens, grad, V)
            o = tgs_gpu.newton_schulz(small)
        return weight, momentum, g, o

    given = [inputs(i) for i in range(2)]
    want = [work(x) for x in given]
    torch.cuda.synchronize()
    got = in_threads(2, lambda i: work(given[i]))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.gpu
def test_a_graph_outlives_the_workspace_of_its_stream(tgs_gpu):
    """Captured on the stream that was warmed up, without a workspace of the
    caller's; then a larger call there replaces the stream's own."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(300, 400, device="cuda", generator=gen)
    tokens = torch.randint(0, 900, (9_000,), device="cuda", generator=gen)
    grad = torch.randn(9_000, 40, device="cuda", generator=gen)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        o, g = tgs_gpu.newton_schulz(x), tgs_gpu.embedding_grad(tokens, grad, 900)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        tgs_gpu.newton_schulz(x, out=o)
        tgs_gpu.embedding_grad(tokens, grad, 900, out=g)
    with torch.cuda.stream(stream):
        tgs_gpu.newton_schulz(torch.randn(900, 1300, device="cuda", generator=gen))
        tgs_gpu.embedding_grad(torch.randint(0, 900, (200_000,), device="cuda", generator=gen),
                               torch.randn(200_000, 40, device="cuda", generator=gen), 900)
        others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in [1 << 16, 1 << 20, 1 << 22] * 20]
    stream.synchronize()
    for seed in (4, 5, 6):
        gen.manual_seed(seed)
        x.normal_(generator=gen)
        grad.normal_(generator=gen)
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, tgs_gpu.newton_schulz(x)) and torch.equal(g, tgs_gpu.embedding_grad(tokens, grad, 900))
        assert all(bool((t == 7).all()) for t in others)


@pytest.mark.gpu
def test_every_call_refuses_a_workspace_in_host_memory(tgs_gpu):
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    ids, x, v = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(4, 8, device="cuda"), torch.ones(64, device="cuda")
    lam = torch.ones(1, device="cuda")
    for call in (lambda: tgs_gpu.embedding_lookup(ids, x, ws=ws), lambda: tgs_gpu.embedding_grad(ids, x, 4, ws=ws),
                 lambda: tgs_gpu.newton_schulz(x, ws=ws), lambda: tgs_gpu.muon_step(x, x.clone(), x.clone(), lr=0.1, ws=ws),
                 lambda: tgs_gpu.topk_ef_step(v, v.clone(), 3, ws=ws),
                 lambda: tgs_gpu.topk_ef_step_segmented(v, v.clone(), [0, 64], [3], ws=ws),
                 lambda: tgs_gpu.threshold_ef_step(v, v.clone(), 0.5, 64, ws=ws),
                 lambda: tgs_gpu.threshold_ef_step_dev(v, v.clone(), lam, 64, ws=ws),
                 lambda: tgs_gpu.threshold_estimate(v, v.clone(), ids, 1, ws=ws),
                 lambda: tgs_gpu.estimated_threshold_ef_step(v, v.clone(), ids, 1, 64, ws=ws),
                 lambda: tgs_gpu.rtopk_ef_step(v, v.clone(), 8, 3, 1, 1, ws=ws),
                 lambda: tgs_gpu.gtopk_merge(ids[:3].view(1, 3), v[:3].view(1, 3), 64, ws=ws)):
        with pytest.raises(ValueError, match="ws is on cpu"):
            call()
    assert x.eq(1).all() and v.eq(1).all()
