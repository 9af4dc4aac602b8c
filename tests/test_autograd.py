"""What autograd sees of the training step's operators."""
import pytest
import torch

U = 2.0**-24
FLOATS = (torch.float32, torch.bfloat16, torch.float16)


def normal(*shape, seed, dtype=torch.float32):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=gen).to(dtype)


def tokens_of(V, *shape, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-V // 8, V, shape, device="cuda", generator=gen)


def definition(tokens, table, scale):
    rows = table[tokens.clamp(min=0)] * scale
    return torch.where((tokens >= 0)[..., None], rows, torch.zeros_like(rows))


@pytest.mark.gpu
@pytest.mark.parametrize("table_dtype", FLOATS)
@pytest.mark.parametrize("out_dtype", [None, *FLOATS])
@pytest.mark.parametrize("shape", [(7, 30), (6, 1000)])
def test_a_lookup_gives_its_table_a_gradient(tgs_gpu, table_dtype, out_dtype, shape):
    V, D, scale = 90, 24, 0.37
    tokens = tokens_of(V, *shape, seed=1)
    table = normal(V, D, seed=2, dtype=table_dtype).requires_grad_()
    rows = tgs_gpu.embedding_lookup(tokens, table, scale=scale, out_dtype=out_dtype)
    assert rows.requires_grad and rows.dtype == (out_dtype or table_dtype)
    g = normal(*rows.shape, seed=3, dtype=rows.dtype)
    rows.backward(g)
    assert table.grad.dtype == table_dtype
    exact = table.detach().double().requires_grad_()
    definition(tokens, exact, scale).backward(g.double())
    count = torch.bincount(tokens[tokens >= 0], minlength=V)[:, None]
    size = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(
        0, tokens[tokens >= 0], g[tokens >= 0].double().abs()) * scale
    # fp32 sums of `count` terms and a few joining, scale and its product, the rounding to the table's type
    tol = size * (count + 8) * U + exact.grad.abs() * (U + torch.finfo(table_dtype).eps / 2) * 1.01
    tol += torch.finfo(table_dtype).tiny * torch.finfo(table_dtype).eps / 2
    assert ((table.grad.double() - exact.grad).abs() <= tol).all()


@pytest.mark.gpu
def test_gradients_and_differences(tgs_gpu):
    """The lookup is linear: <g, lookup(E + dE) - lookup(E)> is <grad, dE>; and a broadcast gradient."""
    V, D = 50, 17
    tokens, E, dE = tokens_of(V, 40, 5, seed=4), normal(V, D, seed=5).requires_grad_(), normal(V, D, seed=6)
    rows = tgs_gpu.embedding_lookup(tokens, E, scale=2.0)
    g = normal(40, 5, D, seed=7)
    (grad,) = torch.autograd.grad(rows, E, g)
    moved = tgs_gpu.embedding_lookup(tokens, E.detach() + dE, scale=2.0) - rows.detach()
    left, right = (g.double() * moved.double()).sum(), (grad.double() * dE.double()).sum()
    bound = (g.double().abs() * (moved.double().abs() + 4 * rows.detach().double().abs())).sum() * 4 * U
    assert (left - right).abs() <= bound + (grad.double().abs() * dE.double().abs()).sum() * 20 * U
    tgs_gpu.embedding_lookup(tokens, E).sum().backward()  # its gradient is one number, broadcast
    assert torch.equal(E.grad, torch.bincount(tokens[tokens >= 0], minlength=V)[:, None].float().expand(V, D))


@pytest.mark.gpu
def test_gradients_of_gradients(tgs_gpu):
    """embedding_grad is linear in the gradient that it sums, and its own gradient is a lookup."""
    V, D = 30, 9
    tokens = tokens_of(V, 200, seed=8)
    g = normal(200, D, seed=9).requires_grad_()
    s = tgs_gpu.embedding_grad(tokens, g, V, scale=0.5)
    w = normal(V, D, seed=10)
    (dg,) = torch.autograd.grad(s, g, w)
    assert torch.equal(dg, definition(tokens, w, 0.5))
    table = normal(V, D, seed=11).requires_grad_()
    h = normal(200, D, seed=12).requires_grad_()
    (dt,) = torch.autograd.grad(tgs_gpu.embedding_lookup(tokens, table), table, h, create_graph=True)
    (dh,) = torch.autograd.grad(dt, h, w)
    assert torch.equal(dh, definition(tokens, w, 1.0))


@pytest.mark.gpu
def test_what_has_no_gradient_says_so(tgs_gpu):
    tokens, table = tokens_of(8, 5, seed=1), normal(8, 6, seed=2).requires_grad_()
    with pytest.raises(RuntimeError, match="out"):
        tgs_gpu.embedding_lookup(tokens, table, out=torch.empty(5, 6, device="cuda"))
    with pytest.raises(RuntimeError, match="out"):
        tgs_gpu.embedding_grad(tokens, normal(5, 6, seed=3).requires_grad_(), 8, out=torch.zeros(8, 6, device="cuda"),
                               accumulate=True)
    with pytest.raises(RuntimeError, match="out"):
        tgs_gpu.newton_schulz(table, out=torch.empty(8, 6, device="cuda"))
    o = tgs_gpu.newton_schulz(table)
    with pytest.raises(NotImplementedError, match="newton_schulz"):
        o.sum().backward()
    with torch.no_grad():  # and without a graph everything is as before
        want = tgs_gpu.newton_schulz(table.detach())
        assert not tgs_gpu.newton_schulz(table).requires_grad and torch.equal(o.detach(), want)
        assert not tgs_gpu.embedding_lookup(tokens, table, out=torch.empty(5, 6, device="cuda")).requires_grad


@pytest.mark.gpu
def test_what_is_written_in_place_is_seen(tgs_gpu):
    """A graph that saved a tensor must not go back through values that a later call has overwritten."""
    x, g, w = normal(4, 6, seed=1), normal(6, 5, seed=2), normal(6, 5, seed=3).requires_grad_()
    loss = (x.requires_grad_() @ w).sum()
    with torch.no_grad():
        tgs_gpu.muon_step(w, g, torch.zeros_like(g), lr=0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    for write in (lambda t: tgs_gpu.newton_schulz(g, out=t),
                  lambda t: tgs_gpu.embedding_lookup(torch.arange(6, device="cuda"), g, out=t),
                  lambda t: tgs_gpu.embedding_grad(torch.arange(6, device="cuda"), g, 6, out=t),
                  lambda t: tgs_gpu.muon_step(torch.ones_like(g), g, t, lr=0.1)):
        t = normal(6, 5, seed=4)
        before = t._version
        write(t)
        assert t._version > before
    with torch.inference_mode():
        t = normal(6, 5, seed=4)
        tgs_gpu.muon_step(t, g, torch.zeros_like(g), lr=0.1)
