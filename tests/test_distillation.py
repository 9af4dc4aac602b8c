"""Distillation from a teacher's top logits and its gradient, against their
definitions in 64 bits (tolerances in ``_rows``)."""
import ctypes
import math

import pytest
import torch

from _rows import FLOATS, U, Softmax, assert_close, rounded, scores

EINVAL, EWORKSPACE = -1, -2


def make_teacher(logits, K, dtype, ids, seed, empty=0.2, masked=0.1):
    """(indices, scores): distinct tokens in no order, some slots empty, some rows without any."""
    gen = torch.Generator().manual_seed(seed)
    T, V = logits.shape
    at = torch.rand(T, min(V, 4096), generator=gen).argsort(1)[:, :K] * max(1, V // 4096)
    values = logits.float().cpu().gather(1, at) + torch.randn(T, K, generator=gen)
    at[torch.rand(T, K, generator=gen) < empty] = -1
    at[torch.rand(T, generator=gen) < masked] = -5
    return at.to(ids).cuda(), values.to(dtype).cuda()


def exact(logits, indices, teacher, temperature):
    """(loss, its error in fp32, sum of q at every token, its relative error, places with a distribution to follow)."""
    s = Softmax(logits, temperature)
    V = logits.shape[-1]
    at = indices.long().cpu()
    on = (at >= 0) & (at < V)
    t = torch.where(on, teacher.double().cpu(), -math.inf)
    top = t.max(-1, keepdim=True).values
    live = top > -math.inf
    d = torch.where(live, (t - top) / temperature, -math.inf)
    total = d.exp().sum(-1, keepdim=True)
    lq = torch.where(live, d - total.log(), -math.inf)
    q = torch.where(live, lq.exp(), 0.0)
    at = torch.where(on, at, 0)
    lp, ds = s.lp.gather(-1, at), s.d.gather(-1, at)
    terms = torch.where(q > 0, q * (lq - lp), 0.0)
    size = torch.where(q > 0, -d, 0.0)
    K = at.shape[-1]
    # q: its exponent's three roundings and the one by log2(e), the exponential, K / 256 + 12 additions, the division
    mean = (q * size).sum(-1, keepdim=True)
    rel = U * (5 * size + 5 * mean + K / 256 + 12 + 8)
    both = torch.where(q > 0, lq.abs(), 0.0) + torch.where((q > 0) & torch.isfinite(lp), lp.abs(), 0.0)
    off = U * (4 * size + 5 * mean + K / 256 + 12 + 4 * torch.where(q > 0, lq.abs(), 0.0)) + s.tol_lp(ds, torch.where(torch.isfinite(lp), lp, 0.0))
    tol = (q * (off + both * (rel + U * (K / 256 + 16)))).sum(-1)
    qs = torch.zeros_like(s.p).scatter_add_(-1, at, q)
    return s, terms.sum(-1), tol, qs, rel.max(-1, keepdim=True).values + U * K, live[..., 0]


def check_loss(tgs, logits, indices, teacher, temperature=1.0, ws=None):
    loss, stats = tgs.distillation_loss(logits, indices, teacher, temperature, return_stats=True, ws=ws)
    s, want, tol, _, _, live = exact(logits, indices, teacher, temperature)
    assert loss.dtype == torch.float32
    assert_close(loss, torch.where(live, want, 0.0), tol * live, "loss")
    lse = stats[..., 0].double().cpu() / temperature + stats[..., 1].double().cpu()
    assert_close(torch.where(live, lse, 0.0), torch.where(live, (s.m / temperature + s.log_s)[..., 0], 0.0),
                 s.tol_log_s[..., 0], "stats")
    assert torch.equal(loss, tgs.distillation_loss(logits, indices, teacher, temperature))
    return loss, stats


def check_grad(got, logits, indices, teacher, g, temperature=1.0):
    s, _, _, qs, rel, live = exact(logits, indices, teacher, temperature)
    a = g.double().cpu()[..., None] / temperature
    on = live[..., None] & ~s.empty
    want = torch.where(on, a * (s.p - qs), 0.0)
    tol = a.abs() * (s.p * (s.relative() + 3 * U) + qs * (rel + 3 * U)) + U * want.abs()
    assert got.dtype == logits.dtype
    assert_close(got, want, on * (tol + rounded(want, logits.dtype) + 2.0**-120), "grad")


def check(tgs, logits, indices, teacher, temperature=1.0, ws=None):
    """The loss, its gradient and both at once."""
    loss, stats = check_loss(tgs, logits, indices, teacher, temperature, ws)
    g = torch.randn(loss.shape, generator=torch.Generator().manual_seed(4)).cuda()
    grad = tgs.distillation_grad(logits, indices, teacher, stats, g, temperature, ws=ws)
    check_grad(grad, logits, indices, teacher, g, temperature)
    both, step = tgs.distillation_loss_and_grad(logits, indices, teacher, g, temperature, ws=ws)
    # its sums may take another order
    _, want, tol, _, _, live = exact(logits, indices, teacher, temperature)
    assert_close(both, torch.where(live, want, 0.0), tol * live, "loss with its gradient")
    check_grad(step, logits, indices, teacher, g, temperature)
    return loss, stats, g, grad, step


# ------------------------------------------------------------------- CPU --
BASE = dict(z=0x1000000, zt=0, T=16, V=100, ld=100, i=0x2000000, it=4, t=0x2100000, tt=0, K=8, tau=1.0)
WS = dict(ws=0x6000000, wsn=1 << 20)


def call(lib, which, **kw):
    a = dict(BASE, **WS, loss=0x3000000, st=0x3100000, g=0x3200000, out=0x5000000, lo=100)
    a.update(kw)
    p = ctypes.c_void_p
    head = [p(a["z"]), a["zt"], a["T"], a["V"], a["ld"], p(a["i"]), a["it"], p(a["t"]), a["tt"], a["K"], a["tau"]]
    tail = [p(a["ws"]), a["wsn"], None]
    if which == "loss":
        return lib.tgs_distillation_loss(*head, p(a["loss"]), p(a["st"]), *tail)
    if which == "grad":
        return lib.tgs_distillation_grad(*head, p(a["st"]), p(a["g"]), p(a["out"]), a["lo"], *tail)
    return lib.tgs_distillation_loss_and_grad(*head, p(a["g"]), p(a["loss"]), p(a["out"]), a["lo"], *tail)


@pytest.fixture
def lib():
    import top_gradient_sparsification_amd as tgs
    return tgs.library()


@pytest.mark.parametrize("which", ["loss", "grad", "both"])
@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=2**31), dict(V=0), dict(V=2**31), dict(ld=99), dict(zt=4), dict(it=0), dict(tt=3), dict(K=0),
    dict(K=1025), dict(tau=0.0), dict(tau=float("nan")), dict(tau=1e7), dict(z=None), dict(i=None), dict(t=None),
    dict(ws=None), dict(ws=0x6000004), dict(z=0x1000002), dict(i=0x2000004), dict(t=0x2100002),
])
def test_refusals_before_any_launch(lib, which, kw):
    assert call(lib, which, **kw) == EINVAL, lib.tgs_last_error()
    assert b"distillation" in lib.tgs_last_error()


def test_refusals_of_each(lib):
    for kw in (dict(loss=None), dict(loss=0x1000100), dict(loss=0x3100000), dict(loss=0x6000000), dict(st=0x2000000)):
        assert call(lib, "loss", **kw) == EINVAL, kw
    for kw in (dict(st=None), dict(g=None), dict(out=None), dict(lo=99), dict(out=0x1000100), dict(out=0x2000000),
               dict(out=0x1000000, lo=101), dict(out=0x3200000), dict(out=0x3100000)):
        assert call(lib, "grad", **kw) == EINVAL, kw
    for kw in (dict(loss=None), dict(out=None), dict(lo=99), dict(out=0x2100000), dict(loss=0x3200000), dict(loss=0x5000100)):
        assert call(lib, "both", **kw) == EINVAL, kw
    need = lib.tgs_distillation_workspace_bytes(16, 100_000, 0)
    assert need > 32768
    big = dict(V=100_000, ld=100_000, lo=100_000, z=0x10000000, out=0x20000000, wsn=need - 1)
    assert call(lib, "loss", **big) == EWORKSPACE and call(lib, "both", **big) == EWORKSPACE
    assert call(lib, "grad", wsn=32767) == EWORKSPACE
    for bad in ((-1, 10, 0), (1, 0, 0), (1, 10, 3), (2**31, 8, 0)):
        assert lib.tgs_distillation_workspace_bytes(*bad) == 0


def test_binding_refusals_on_the_cpu():
    import top_gradient_sparsification_amd as tgs
    z, i, t = torch.zeros(4, 10), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(TypeError, match="GPU tensor"):
        tgs.distillation_loss(z, i, t)
    with pytest.raises(TypeError, match="logits must be one of"):
        tgs.distillation_loss_and_grad(z.double(), i, t)


def test_the_definitions_agree_with_differences():
    gen = torch.Generator().manual_seed(3)
    z = 2 * torch.randn(4, 9, generator=gen, dtype=torch.float64)
    at = torch.tensor([[0, 3, 8], [2, 2, -1], [-1, -1, -1], [5, 9, 1]])
    t = torch.randn(4, 3, generator=gen, dtype=torch.float64)
    t[0, 1] = -math.inf
    _, loss, tol, qs, _, live = exact(z, at, t, 1.7)
    assert live.tolist() == [True, True, False, True] and loss[2] == 0 and qs[0, 3] == 0
    assert torch.allclose(qs.sum(1), live.double()) and abs(qs[1, 2] - 1) < 1e-12 and qs[3, 5] + qs[3, 1] == qs[3].sum()
    h = 1e-6
    for j in (0, 2, 5):
        step = torch.zeros_like(z)
        step[:, j] = h
        up, down = (exact(z + x * step, at, t, 1.7) for x in (1, -1))
        want = torch.where(live, (up[0].p[:, j] + down[0].p[:, j]) / 2 - qs[:, j], 0.0) / 1.7
        assert ((up[1] - down[1]) / (2 * h) - want).abs().max() < 1e-7
    with pytest.raises(AssertionError):
        assert_close(loss + 1e-4, loss, tol)


# ------------------------------------------------------------------- GPU --
@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 2, 9, 64, 130, 512, 513, 1000, 4097, 10_000, 50_001, 128_000])
def test_vocabularies(tgs_gpu, V):
    for dtype, T, K, ids, tt, tau in ((torch.float32, 3, 1, torch.int32, torch.float32, 1.0),
                                      (torch.bfloat16, 40, 16, torch.int64, torch.bfloat16, 2.0),
                                      (torch.float16, 5, 65, torch.int32, torch.float16, 0.7)):
        logits = scores(T, V, dtype, V)
        indices, teacher = make_teacher(logits, min(K, V), tt, ids, V, masked=0.2 if T > 5 else 0.0)
        check(tgs_gpu, logits, indices, teacher, tau)


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,K", [(2500, 1000, 8), (1100, 5001, 33), (300, 20_000, 64), (4000, 3, 2), (9000, 130, 5)])
def test_many_rows(tgs_gpu, T, V, K):
    for dtype in FLOATS:
        logits = scores(T, V, dtype, T)
        check(tgs_gpu, logits, *make_teacher(logits, K, torch.float32, torch.int32, T))


@pytest.mark.gpu
@pytest.mark.parametrize("K", [2, 255, 256, 257, 700, 1024])
def test_slots(tgs_gpu, K):
    for T, V in ((6, 5000), (1100, 1500)):
        for ids in (torch.int32, torch.int64):
            logits = scores(T, V, torch.bfloat16, K)
            check(tgs_gpu, logits, *make_teacher(logits, K, torch.bfloat16, ids, K))


@pytest.mark.gpu
@pytest.mark.parametrize("V", [9000, 16_000, 16_001, 32_768, 32_775, 60_000, 60_001])
def test_rows_read_twice_by_one_workgroup(tgs_gpu, V):
    """Rows kept in LDS whole and in part, by 256, 512 and 1,024 threads, from and to lines and between them."""
    T = 520
    for dtype, pad, K in ((torch.bfloat16, 0, 9), (torch.float32, 3, 70)):
        logits = scores(T, V, dtype, V, pad=pad)
        indices, teacher = make_teacher(logits, K, torch.float32, torch.int32, V)
        g = torch.randn(T, generator=torch.Generator().manual_seed(3)).cuda()
        loss, grad = tgs_gpu.distillation_loss_and_grad(logits, indices, teacher, g, 1.5)
        _, want, tol, _, _, live = exact(logits, indices, teacher, 1.5)
        assert_close(loss, torch.where(live, want, 0.0), tol * live, "loss")
        check_grad(grad, logits, indices, teacher, g, 1.5)
        again, out = tgs_gpu.distillation_loss_and_grad(logits, indices, teacher, g, 1.5, out=logits)
        assert torch.equal(again, loss) and torch.equal(logits, grad)


@pytest.mark.gpu
def test_most_slots_beside_a_row_in_lds(tgs_gpu):
    logits = scores(515, 60_000, torch.bfloat16, 1)
    indices, teacher = make_teacher(logits, 1024, torch.bfloat16, torch.int64, 1)
    loss, grad = tgs_gpu.distillation_loss_and_grad(logits, indices, teacher)
    _, want, tol, _, _, live = exact(logits, indices, teacher, 1.0)
    assert_close(loss, torch.where(live, want, 0.0), tol * live, "loss")
    check_grad(grad, logits, indices, teacher, torch.ones(515))


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(9, 100), (9, 3000), (9, 60_000), (1100, 3000)])
def test_an_index_in_several_slots(tgs_gpu, T, V):
    for dtype in FLOATS:
        logits = scores(T, V, dtype, 1)
        indices, teacher = make_teacher(logits, 48, torch.float32, torch.int64, 2, masked=0.0)
        indices[:, 5] = indices[:, 1] = indices[:, 40] = V - 1
        indices[3] = 7
        indices[4, ::2] = indices[4, 1::2]
        check(tgs_gpu, logits, indices, teacher, 1.5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("T,V,pad", [(7, 1001, 23), (1300, 777, 1), (3, 50_001, 47), (40, 100, 3), (33, 30_000, 1)])
def test_rows_apart_and_in_place(tgs_gpu, dtype, T, V, pad):
    logits = scores(T, V, dtype, 5, pad=pad)
    rows = logits.as_strided((T, V + pad), (V + pad, 1))
    indices, teacher = make_teacher(logits, 20, torch.float32, torch.int32, 5)
    loss, stats, g, grad, step = check(tgs_gpu, logits, indices, teacher)
    wide = torch.full((T, V + pad + 2), 5.0, dtype=dtype, device="cuda")
    tgs_gpu.distillation_grad(logits, indices, teacher, stats, g, out=wide[:, 2:V + 2])
    assert torch.equal(wide[:, 2:V + 2], grad) and (wide[:, :2] == 5).all() and (wide[:, V + 2:] == 5).all()
    kept, version = rows.clone(), logits._version
    assert tgs_gpu.distillation_grad(logits, indices, teacher, stats, g, out=logits) is logits
    assert torch.equal(logits, grad) and torch.isnan(rows[:, V:]).all() and logits._version > version
    rows.copy_(kept)
    again, out = tgs_gpu.distillation_loss_and_grad(logits, indices, teacher, g, out=logits)
    assert out is logits and torch.equal(logits, step) and torch.equal(again, loss) and torch.isnan(rows[:, V:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(8, 60), (8, 4000), (8, 70_001), (1030, 4000)])
@pytest.mark.parametrize("dtype", FLOATS)
def test_masks_and_infinities(tgs_gpu, dtype, T, V):
    logits = scores(T, V, dtype, 2).clone()
    indices, teacher = make_teacher(logits, 10, torch.float32, torch.int32, 2, empty=0.0, masked=0.0)
    indices[:, 0], indices[:, 1] = 0, V - 1
    logits[0] = -math.inf                             # no distribution: loss inf, gradient 0
    logits[1] = torch.finfo(dtype).min                # uniform
    logits[2, 1:] = -math.inf                         # q > 0 where p = 0: loss inf
    teacher[3, 2:] = -math.inf                        # slots without probability
    teacher[4] = -math.inf                            # none has any: masked
    indices[5] = -1                                   # no slots: masked
    logits[5] = math.nan                              # of which nothing is needed
    teacher[6] = torch.finfo(torch.float32).min       # equal scores
    logits[7, ::2] = -math.inf
    indices[7], teacher[7, 5:] = torch.arange(10, dtype=torch.int32), -math.inf
    indices[7, :5] = 2 * torch.arange(5, dtype=torch.int32) + 1
    loss, stats = tgs_gpu.distillation_loss(logits, indices, teacher, return_stats=True)
    g = torch.ones(T, device="cuda")
    grad = tgs_gpu.distillation_grad(logits, indices, teacher, stats, g)
    both, step = tgs_gpu.distillation_loss_and_grad(logits, indices, teacher)
    assert torch.equal(both, loss) and not grad[5].any() and not step[5].any() and loss[5] == 0
    assert loss[0] == math.inf and loss[2] == math.inf and loss[4] == 0 and not grad[4].any() and not grad[0].any()
    assert torch.isfinite(loss[[1, 3, 6, 7]]).all() and torch.isfinite(grad.float()).all()
    keep = torch.tensor([i for i in range(T) if i != 5], device="cuda")
    check(tgs_gpu, logits[keep], indices[keep], teacher[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(6, 60), (6, 4000), (6, 70_001), (1030, 4000)])
def test_nan_and_infinity_stay_in_their_rows(tgs_gpu, T, V):
    logits = scores(T, V, torch.float32, 4)
    indices, teacher = make_teacher(logits, 12, torch.float32, torch.int64, 4, empty=0.3, masked=0.0)
    want, wstep = tgs_gpu.distillation_loss_and_grad(logits, indices, teacher)
    bad, worse = logits.clone(), teacher.clone()
    indices[1:5, 0] = 3
    bad[1, V // 2], bad[2, 0] = math.nan, math.inf
    worse[3, 0], worse[4, 0] = math.nan, math.inf
    loss, stats = tgs_gpu.distillation_loss(bad, indices, worse, return_stats=True)
    grad = tgs_gpu.distillation_grad(bad, indices, worse, stats, torch.ones_like(loss))
    both, step = tgs_gpu.distillation_loss_and_grad(bad, indices, worse)
    for x in (loss, both, grad, step):
        assert torch.isnan(x[1:5]).all()
    keep = [0, 5] + list(range(6, T))
    assert torch.equal(loss[keep], want[keep]) and torch.equal(both[keep], want[keep]) and torch.equal(step[keep], wstep[keep])


@pytest.mark.gpu
def test_bad_indices_are_reported_and_empty(tgs_gpu):
    for T, V in ((4, 100), (4, 90_000), (1200, 700)):
        logits = scores(T, V, torch.float32, 8)
        indices, teacher = make_teacher(logits, 6, torch.float32, torch.int64, 8, masked=0.0)
        indices[1, 2], indices[2] = V, 2**40
        indices[0, 0] = -2**40
        need = tgs_gpu.distillation_workspace_bytes(T, V, torch.float32)
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        check(tgs_gpu, logits, indices, teacher, ws=ws)
        with pytest.raises(ValueError, match="index"):
            tgs_gpu.check_device_error(ws)
        tgs_gpu.check_device_error(ws)
        assert not ws[:32768].any()


@pytest.mark.gpu
def test_offsets_past_32_bits(tgs_gpu):
    V, T = 50_001, 44_000
    logits = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    logits[-1100:] = scores(1100, V, torch.bfloat16, 9)
    indices = torch.full((T, 4), -1, dtype=torch.int32, device="cuda")
    teacher = torch.zeros(T, 4, device="cuda")
    indices[-1100:], teacher[-1100:] = make_teacher(logits[-1100:], 4, torch.float32, torch.int32, 9)
    w = torch.rand(T, device="cuda")
    want, wgrad = tgs_gpu.distillation_loss_and_grad(logits[-1100:], indices[-1100:], teacher[-1100:], w[-1100:])
    loss, stats = tgs_gpu.distillation_loss(logits, indices, teacher, return_stats=True)
    part = tgs_gpu.distillation_grad(logits, indices, teacher, stats, w)
    assert torch.equal(part[-1100:].float(), tgs_gpu.distillation_grad(
        logits[-1100:], indices[-1100:], teacher[-1100:], stats[-1100:], w[-1100:]).float())
    del part
    assert torch.equal(loss[-1100:], tgs_gpu.distillation_loss(logits[-1100:], indices[-1100:], teacher[-1100:]))
    both, _ = tgs_gpu.distillation_loss_and_grad(logits, indices, teacher, w, out=logits)
    assert torch.equal(both[-1100:], want) and not both[:-1100].any() and not loss[:-1100].any()
    assert torch.equal(logits[-1100:], wgrad) and not logits[:-1100].any()


@pytest.mark.gpu
def test_more_rows_than_a_launch_takes(tgs_gpu):
    T, V = 2**22 + 1000, 3  # the two-in-one call's launches are cut for its largest workgroups
    gen = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(T, V, device="cuda", generator=gen)
    indices = torch.randint(-1, V, (T, 2), device="cuda", generator=gen)
    teacher = torch.randn(T, 2, device="cuda", generator=gen)
    tail = slice(T - 2000, T)
    loss, grad = tgs_gpu.distillation_loss_and_grad(logits, indices, teacher)
    want, wgrad = tgs_gpu.distillation_loss_and_grad(logits[tail], indices[tail], teacher[tail])
    assert torch.equal(loss[tail], want) and torch.equal(grad[tail], wgrad)
    check(tgs_gpu, logits[tail], indices[tail], teacher[tail])


@pytest.mark.gpu
def test_gradients_flow(tgs_gpu):
    z = scores(24, 300, torch.float32, 3).clone()
    indices, teacher = make_teacher(z, 12, torch.float32, torch.int32, 3)
    z, indices, teacher = z.view(4, 6, 300), indices.view(4, 6, 12), teacher.view(4, 6, 12)
    z.requires_grad_()
    loss, stats = tgs_gpu.distillation_loss(z, indices, teacher, 1.4, return_stats=True)
    assert loss.requires_grad and not stats.requires_grad
    w = torch.linspace(0, 1, 24, device="cuda").view(4, 6)
    (got,) = torch.autograd.grad((w * loss).sum(), z)
    assert torch.equal(got, tgs_gpu.distillation_grad(z.detach(), indices, teacher, stats, w, 1.4))
    (mean,) = torch.autograd.grad(tgs_gpu.distillation_loss(z, indices, teacher).mean(), z)
    # the directional derivative in 64 bits
    v = torch.randn(z.shape, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    zd, h = z.detach().double().cpu(), 1e-6
    up, down = (exact(zd + s * h * v, indices, teacher, 1.0)[1].mean() for s in (1, -1))
    want = (up - down) / (2 * h)
    assert abs((mean.double().cpu() * v).sum() - want) < 1e-4 * abs(want) + 1e-5
    with pytest.raises(RuntimeError, match="detach teacher_logits"):
        tgs_gpu.distillation_loss(z, indices, teacher.clone().requires_grad_())
    _, step = tgs_gpu.distillation_loss_and_grad(z, indices, teacher)
    with pytest.raises(NotImplementedError, match="distillation_loss_and_grad has no gradient"):
        step.sum().backward()
    with pytest.raises(RuntimeError, match="out="):
        tgs_gpu.distillation_loss_and_grad(z, indices, teacher, out=torch.empty_like(z))


@pytest.mark.gpu
def test_shapes_and_binding_refusals(tgs_gpu):
    z = scores(6, 40, torch.float32, 1)
    i, t = make_teacher(z, 3, torch.float32, torch.int32, 1)
    f, st = torch.zeros(6, device="cuda"), torch.zeros(6, 2, device="cuda")
    assert tgs_gpu.distillation_loss(z[1], i[1], t[1]).shape == ()
    loss, grad = tgs_gpu.distillation_loss_and_grad(z[:0], i[:0], t[:0], f[:0])
    assert loss.shape == (0,) and grad.shape == (0, 40)
    assert tgs_gpu.distillation_grad(z[:0], i[:0], t[:0], st[:0], f[:0]).shape == (0, 40)
    for call_, error in ((lambda: tgs_gpu.distillation_loss(z, i[:5], t), "teacher_indices must have"),
                         (lambda: tgs_gpu.distillation_loss(z, i, t[:, :2].contiguous()), "teacher_logits must have shape"),
                         (lambda: tgs_gpu.distillation_loss(z, i.float(), t), "teacher_indices must be one of"),
                         (lambda: tgs_gpu.distillation_loss(z, i[:, :0].contiguous(), t[:, :0].contiguous()), "K=0"),
                         (lambda: tgs_gpu.distillation_loss(z, i, t, temperature=-1.0), "temperature"),
                         (lambda: tgs_gpu.distillation_loss(z.T, i, t), "contiguous along"),
                         (lambda: tgs_gpu.distillation_grad(z, i, t, st[:5], f), "stats must have shape"),
                         (lambda: tgs_gpu.distillation_grad(z, i, t, st, f[:5]), "grad_loss must have shape"),
                         (lambda: tgs_gpu.distillation_loss_and_grad(z, i, t, f.half()), "weights must be one of"),
                         (lambda: tgs_gpu.distillation_loss_and_grad(z, i, t, out=z[:, :20]), "out must have shape"),
                         (lambda: tgs_gpu.distillation_loss(z, i, t, ws=torch.zeros(64, dtype=torch.uint8)), "ws is on cpu"),
                         (lambda: tgs_gpu.distillation_loss(z, i, t, ws=torch.zeros(64, dtype=torch.uint8, device="cuda")), "need")):
        with pytest.raises((ValueError, TypeError, MemoryError), match=error):
            call_()


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(6, 60), (6, 4000), (6, 70_001), (1030, 4000)])
@pytest.mark.parametrize("dtype", FLOATS)
def test_rows_of_nan_alone(tgs_gpu, dtype, T, V):
    """Such a row's gradient is NaN as its loss is, and not the zeros of a row of -inf: from the
    separate calls and from the one that makes both, in one workgroup and in slices."""
    logits = scores(T, V, dtype, 4)
    indices, teacher = make_teacher(logits, 12, torch.float32, torch.int64, 4, empty=0.3, masked=0.0)
    bad = logits.clone()
    bad[1] = math.nan
    bad[2], bad[2, V // 2] = -math.inf, math.nan
    bad[4] = -math.inf
    indices[5], bad[5] = -1, math.nan            # masked: nothing of it is needed
    want, stats = tgs_gpu.distillation_loss(logits, indices, teacher, return_stats=True)
    ok = tgs_gpu.distillation_grad(logits, indices, teacher, stats, torch.ones_like(want))
    loss, stats = tgs_gpu.distillation_loss(bad, indices, teacher, return_stats=True)
    grad = tgs_gpu.distillation_grad(bad, indices, teacher, stats, torch.ones_like(loss))
    both, step = tgs_gpu.distillation_loss_and_grad(bad, indices, teacher)
    keep = torch.tensor([0, 3, 5] + list(range(6, T)), device="cuda")
    for x in (loss, both, grad, step):
        assert torch.isnan(x[1:3]).all()
    assert loss[4] == math.inf and both[4] == math.inf and loss[5] == 0 and both[5] == 0
    assert (grad[4:6] == 0).all() and (step[4:6] == 0).all()
    assert torch.equal(loss[keep], want[keep]) and torch.equal(grad[keep], ok[keep])
    teacher[4, 0], indices[4, 0] = math.nan, 1   # a teacher's NaN goes to such a row too
    loss, stats = tgs_gpu.distillation_loss(bad, indices, teacher, return_stats=True)
    grad = tgs_gpu.distillation_grad(bad, indices, teacher, stats, torch.ones_like(loss))
    both, step = tgs_gpu.distillation_loss_and_grad(bad, indices, teacher)
    for x in (loss, both, grad, step):
        assert torch.isnan(x[4]).all()
    assert torch.equal(loss[keep], want[keep]) and torch.equal(grad[keep], ok[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(3, 50), (3, 70_001), (1030, 9000)])
def test_scores_further_apart_than_the_type_reaches(tgs_gpu, T, V):
    """x - m is no fp32 number, (x - m) / temperature is one."""
    for dtype in (torch.float32, torch.bfloat16):
        low = torch.finfo(dtype).min
        logits = scores(T, V, dtype, 3).clone()
        indices, teacher = make_teacher(logits, 5, torch.float32, torch.int32, 3, masked=0.0)
        logits[0, 7], logits[0, 9] = low, -low
        indices[0, 0], teacher[0, 0] = 7, 3.0
        for tau in (2.5, 1e6):
            loss = check(tgs_gpu, logits, indices, teacher, tau)[0]
            assert torch.isfinite(loss[0]) and loss[0] > 1e31


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("V", [65_537, 65_539, 65_543, 65_545])
def test_last_slices_of_a_few_scores(tgs_gpu, dtype, V):
    """Rows in slices of 4,096 or 8,192 scores, of which the last holds less than a vector or little more; and
    enough slots for longer ones."""
    for K in (7, 700):
        logits = scores(5, V, dtype, 7).clone()
        indices, teacher = make_teacher(logits, K, torch.float32, torch.int64, 7, masked=0.0)
        indices[:, 0] = V - 1
        logits[1, 65_536:] = 30.0
        logits[2, :65_000] = -math.inf
        indices[2, 1:] = -1
        check(tgs_gpu, logits, indices, teacher, 0.8)
