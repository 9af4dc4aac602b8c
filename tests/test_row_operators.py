"""The row operators together, as a training step runs them: hidden states,
norm, logits, losses, and back; on other streams, in graphs, from two threads."""
import pytest
import torch

from _rows import scores


def inputs(T, D, V, K, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sigma=1.0):
        return (sigma * torch.randn(*shape, device="cuda", generator=gen)).to(dtype)

    return dict(x=normal(T, D), w=1 + 0.1 * normal(D).float(), b=0.1 * normal(D).float(), head=normal(D, V, sigma=D**-0.5),
                tokens=torch.randint(-1, V, (T,), device="cuda", generator=gen),
                at=torch.randint(-1, V, (T, K), device="cuda", generator=gen, dtype=torch.int32), teacher=normal(T, K),
                weights=torch.rand(T, device="cuda", generator=gen))


def chain(tgs, i, out=None):
    """One step by the operators' own calls; ``out`` holds results to write to where the calls take them."""
    y, mean, rstd = tgs.layer_norm(i["x"], i["w"], i["b"], return_stats=True)
    logits = y @ i["head"]
    r = tgs.token_logprobs(logits, i["tokens"], top=4, entropy=True)
    g = tgs.token_logprobs_grad(logits, i["tokens"], r.stats, i["weights"], r.entropy, i["weights"], 1.0)
    loss, stats = tgs.distillation_loss(logits, i["at"], i["teacher"], 2.0, return_stats=True)
    d = tgs.distillation_grad(logits, i["at"], i["teacher"], stats, i["weights"], 2.0)
    both, step = tgs.distillation_loss_and_grad(logits, i["at"], i["teacher"], i["weights"], 2.0)
    back = ((g + d) @ i["head"].T.contiguous())
    gx, gw, gb = tgs.layer_norm_grad(back, i["x"], mean, rstd, i["w"])
    return (y, mean, rstd, *r, g, loss, stats, d, both, step, gx, gw, gb)


SIZES = [(5, 64, 300, 4), (33, 200, 30_000, 16), (1100, 130, 2000, 40)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,V,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_step_against_autograd_in_64_bits(tgs_gpu, T, D, V, K, dtype):
    i = inputs(T, D, V, K, dtype, 1)
    x, w, b, head = (i[n].clone().requires_grad_() for n in ("x", "w", "b", "head"))
    logits = tgs_gpu.layer_norm(x, w, b, out_dtype=dtype) @ head
    r = tgs_gpu.token_logprobs(logits, i["tokens"], entropy=True)
    kl = tgs_gpu.distillation_loss(logits, i["at"], i["teacher"], 2.0)
    loss = (i["weights"] * (kl - r.logprobs - 0.1 * r.entropy)).mean()
    got = torch.autograd.grad(loss, (x, w, b, head))

    xd, wd, bd, hd = (i[n].double().cpu().requires_grad_() for n in ("x", "w", "b", "head"))
    y = torch.nn.functional.layer_norm(xd, (D,), wd, bd)
    z = y @ hd
    tokens, at = i["tokens"].cpu(), i["at"].long().cpu()
    lp = torch.log_softmax(z, -1)
    real = tokens >= 0
    ent = -(lp.exp() * lp).sum(-1)
    t = (i["teacher"].double().cpu() / 2).masked_fill(at < 0, -torch.inf)
    live = (at >= 0).any(-1)
    q = torch.softmax(t[live], -1)
    lp2 = torch.log_softmax(z / 2, -1)[live].gather(-1, at[live].clamp(min=0))
    d = torch.zeros(T, dtype=torch.float64)
    d[live] = (torch.special.xlogy(q, q) - torch.where(q > 0, q * lp2, 0.0)).sum(-1)
    wt = i["weights"].double().cpu()
    want_loss = (wt * (d - real * (lp.gather(-1, tokens.clamp(min=0)[:, None])[:, 0] + 0.1 * ent))).mean()
    want = torch.autograd.grad(want_loss, (xd, wd, bd, hd))
    # torch's own products round their results: to bf16 2^-8 of each logit (of size 4) and of each gradient
    eps = 2.0**-20 if dtype == torch.float32 else 2.0**-8
    assert abs(loss.item() - want_loss.item()) <= 8 * eps * max(1.0, abs(want_loss.item()))
    for a, c in zip(got, want):
        assert (a.double().cpu() - c).norm() <= 8 * eps * c.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,V,K", SIZES)
def test_the_same_bits_every_time_and_on_another_stream(tgs_gpu, T, D, V, K):
    i = inputs(T, D, V, K, torch.bfloat16, 2)
    want = chain(tgs_gpu, i)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = [chain(tgs_gpu, i) for _ in range(3)]
    stream.synchronize()
    for results in got:
        for a, b in zip(results, want):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,V,K", SIZES)
def test_two_graphs_and_eager_work_between_their_replays(tgs_gpu, T, D, V, K):
    """Two captured steps and the eager one, on inputs that change from replay to replay."""
    given = [inputs(T, D, V, K, torch.bfloat16, 3 + n) for n in range(2)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for i in given:
            chain(tgs_gpu, i)
    stream.synchronize()
    graphs, results = [], []
    for i in given:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            results.append(chain(tgs_gpu, i))
    for seed in (11, 12, 13):
        for n, i in enumerate(given):
            for name, value in inputs(T, D, V, K, torch.bfloat16, 10 * seed + n).items():
                i[name].copy_(value)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        bigger = inputs(2 * T, D, V, K, torch.bfloat16, seed)  # an eager call that outgrows the kept workspace
        chain(tgs_gpu, bigger)
        torch.cuda.synchronize()
        for i, got in zip(given, results):
            for a, b in zip(got, chain(tgs_gpu, i)):
                assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_captured_backward_pass(tgs_gpu):
    i = inputs(40, 96, 500, 8, torch.float32, 5)
    x, w, b = (i[n].requires_grad_() for n in ("x", "w", "b"))

    def step():
        logits = tgs_gpu.layer_norm(x, w, b) @ i["head"]
        r = tgs_gpu.token_logprobs(logits, i["tokens"], entropy=True)
        loss = (tgs_gpu.distillation_loss(logits, i["at"], i["teacher"]) - r.logprobs - 0.1 * r.entropy) * i["weights"]
        return torch.autograd.grad(loss, (x, w, b), torch.ones_like(loss))

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = step()
    for seed in (6, 7, 8):
        with torch.no_grad():
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(got, step()):
            assert torch.equal(a, c)


@pytest.mark.gpu
def test_two_threads_on_one_stream(tgs_gpu):
    from test_workspaces import in_threads
    given = [inputs(33, 200, 30_000, 16, torch.bfloat16, 20 + n) for n in range(2)]
    want = [chain(tgs_gpu, i) for i in given]
    torch.cuda.synchronize()
    got = in_threads(2, lambda n: [chain(tgs_gpu, given[n]) for _ in range(10)][-1])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.gpu
def test_one_workspace_for_calls_of_all_kinds(tgs_gpu):
    """A workspace moves between these operators and the sparsifier's."""
    logits = scores(6, 40_000, torch.float32, 1)
    tokens = torch.arange(6, device="cuda")
    n, k = 300_000, 400
    ws = torch.zeros(max(tgs_gpu.topk_workspace_bytes(n, k), tgs_gpu.token_logprobs_workspace_bytes(6, 40_000, torch.float32, 9)),
                     dtype=torch.uint8, device="cuda")
    g = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    want = tgs_gpu.topk_ef_step(g, torch.zeros_like(g), k)
    first = tgs_gpu.token_logprobs(logits, tokens, top=9, entropy=True)
    for _ in range(3):
        got = tgs_gpu.topk_ef_step(g, torch.zeros_like(g), k, ws=ws)
        r = tgs_gpu.token_logprobs(logits, tokens, top=9, entropy=True, ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(a, b) for a, b in zip(r, first))
        tgs_gpu.check_device_error(ws)


@pytest.mark.gpu
def test_an_out_that_requires_a_gradient_is_refused(tgs_gpu):
    """Written behind autograd's back it would keep a graph of the values that it held before."""
    T, D, V, K = 6, 40, 50, 3
    i = inputs(T, D, V, K, torch.float32, 9)
    z = scores(T, V, torch.float32, 1)
    f, st = torch.ones(T, device="cuda"), torch.zeros(T, 2, device="cuda")
    for make in (lambda *shape: torch.zeros(shape, device="cuda").requires_grad_(),
                 lambda *shape: torch.zeros(shape, device="cuda").requires_grad_() * 2):
        row, out = make(T, D), make(T, V)
        for call in (lambda: tgs_gpu.layer_norm(i["x"], out=row),
                     lambda: tgs_gpu.layer_norm_grad(i["x"], i["x"], f, f, out=row),
                     lambda: tgs_gpu.token_logprobs_grad(z, i["tokens"], st, f, out=out),
                     lambda: tgs_gpu.distillation_grad(z, i["at"], i["teacher"], st, f, out=out),
                     lambda: tgs_gpu.distillation_loss_and_grad(z, i["at"], i["teacher"], f, out=out)):
            with pytest.raises(RuntimeError, match="out requires a gradient"):
                call()
            assert not out.any() and not row.any()
            with torch.no_grad():
                call()
            with torch.no_grad():
                row.zero_(), out.zero_()
