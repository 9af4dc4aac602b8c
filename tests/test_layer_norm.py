"""Layer norm and its gradients, against their definitions in 64 bits.

Tolerances count roundings of fp32 (U = 2^-24 each) and the last rounding to
the result's type.  ``depth`` is the most additions that a value goes through:
32 in a thread, 10 and more to join the threads, D / 4,096 where a row is read
in a loop.
"""
import ctypes

import pytest
import torch

from _rows import FLOATS, U, assert_close, half_step, rounded, tiny

EINVAL, EWORKSPACE = -1, -2


def depth(D):
    return 48 + D / 1024


def exact_norm(x, weight, bias, eps):
    """(y, error that fp32 allows, mean, rstd) with one rounding of y still to count."""
    x = x.detach().double().cpu()
    one = torch.ones(x.shape[-1], dtype=torch.float64)
    w = one if weight is None else weight.detach().double().cpu()
    b = 0 * one if bias is None else bias.detach().double().cpu()
    mean = x.mean(-1, keepdim=True)
    var = ((x - mean) ** 2).mean(-1, keepdim=True)
    rstd = (var + eps).rsqrt()
    xh = (x - mean) * rstd
    y = xh * w + b
    k = depth(x.shape[-1])
    off = (k + 1) * U * x.abs().mean(-1, keepdim=True)  # of the mean
    # var's sum and division, the mean's error squared, then eps, root and division
    scale = U * ((k + 3) / 2 + 4) + off**2 / (2 * (var + eps))
    tol = w.abs() * (rstd * off + xh.abs() * (scale + 3 * U)) + U * y.abs()
    return y, tol, (mean, off + U * mean.abs()), (rstd, rstd * scale)


def exact_grad(g, x, mean, rstd, weight):
    """x's, weight's and bias's gradients with the errors that fp32 allows, before the last rounding."""
    g, x, mean, rstd = (t.detach().double().cpu() for t in (g, x, mean, rstd))
    D, T = x.shape[-1], x.shape[:-1].numel()
    g, x, mean, rstd = g.reshape(T, D), x.reshape(T, D), mean.reshape(T, 1), rstd.reshape(T, 1)
    w = torch.ones(D, dtype=torch.float64) if weight is None else weight.detach().double().cpu()
    xh, gw = (x - mean) * rstd, g * w
    m0, m1 = gw.mean(-1, keepdim=True), (gw * xh).mean(-1, keepdim=True)
    a0, a1 = gw.abs().mean(-1, keepdim=True), (gw * xh).abs().mean(-1, keepdim=True)
    gx = rstd * (gw - m0 - xh * m1)
    k = depth(D)
    tol = rstd * U * ((k + 3) * a0 + xh.abs() * ((k + 6) * a1 + 4 * m1.abs()) + 3 * gw.abs() + 2 * m0.abs()) + 3 * U * gx.abs()
    # a workgroup's rows, at least a 64th of all; its waves, the partial rows in 16 parts
    rows = T / 64 + 64
    gwt, gb = (g * xh).sum(0), g.sum(0)
    tw, tb = U * (rows + 3) * (g * xh).abs().sum(0), U * rows * g.abs().sum(0)
    return (gx, tol), (gwt, tw), (gb, tb)


def make(T, D, dtype, seed, mean=0.3, scale=1.5):
    gen = torch.Generator().manual_seed(seed)
    return (mean + scale * torch.randn(T, D, generator=gen)).to(dtype).cuda()


def params(D, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    return ((1 + 0.3 * torch.randn(D, generator=gen)).to(dtype).cuda(),
            (0.2 * torch.randn(D, generator=gen)).to(dtype).cuda())


def check(tgs, x, w, b, out_dtype=None, eps=1e-5, grad=True):
    """Forward and backward of one call against the definitions; returns the results."""
    y, mean, rstd = tgs.layer_norm(x, w, b, eps=eps, out_dtype=out_dtype, return_stats=True)
    want, tol, (em, tm), (er, tr) = exact_norm(x, w, b, eps)
    assert y.dtype == (out_dtype or x.dtype) and y.shape == x.shape
    assert_close(y, want, tol + rounded(want, y.dtype), "y")
    assert_close(mean[..., None], em, tm, "mean")
    assert_close(rstd[..., None], er, tr + U * er, "rstd")
    if not grad:
        return y
    gen = torch.Generator().manual_seed(17)
    g = (0.1 * torch.randn(y.shape, generator=gen)).to(y.dtype).cuda()
    gx, gw, gb = tgs.layer_norm_grad(g, x, mean, rstd, w)
    (wx, tx), (ww, tw), (wb, tb) = exact_grad(g, x, mean, rstd, w)
    assert gx.dtype == x.dtype and gx.shape == x.shape
    assert_close(gx.reshape(wx.shape), wx, tx + rounded(wx, gx.dtype), "grad x")
    assert_close(gw, ww, tw + rounded(ww, gw.dtype), "grad weight")
    assert_close(gb, wb, tb + rounded(wb, gb.dtype), "grad bias")
    assert gw.dtype == gb.dtype == (torch.float32 if w is None else w.dtype)
    return y, g, gx, gw, gb


# ------------------------------------------------------------------- CPU --
def forward_call(lib, **kw):
    a = dict(x=0x100000, xt=0, T=16, D=8, w=0x200000, b=0x210000, wt=0, eps=1e-5, out=0x300000, ot=0, mean=0x400000,
             rstd=0x410000)
    a.update(kw)
    p = ctypes.c_void_p
    return lib.tgs_layer_norm(p(a["x"]), a["xt"], a["T"], a["D"], p(a["w"]), p(a["b"]), a["wt"], a["eps"], p(a["out"]),
                              a["ot"], p(a["mean"]), p(a["rstd"]), None)


def grad_call(lib, **kw):
    a = dict(g=0x500000, gt=0, x=0x100000, xt=0, T=16, D=8, w=0x200000, wt=0, out=0x300000, mean=0x400000,
             rstd=0x410000, gw=0x420000, gb=0x430000, pt=0, ws=0x1000000, wsn=1 << 24)
    a.update(kw)
    p = ctypes.c_void_p
    return lib.tgs_layer_norm_grad(p(a["g"]), a["gt"], p(a["x"]), a["xt"], a["T"], a["D"], p(a["mean"]), p(a["rstd"]),
                                   p(a["w"]), a["wt"], p(a["out"]), p(a["gw"]), p(a["gb"]), a["pt"], p(a["ws"]),
                                   a["wsn"], None)


@pytest.fixture
def lib():
    import top_gradient_sparsification_amd as tgs
    return tgs.library()


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=2**31), dict(D=0), dict(D=2**24 + 1), dict(xt=3), dict(xt=9), dict(wt=4), dict(x=None),
    dict(out=None), dict(x=0x100002), dict(out=0x300001), dict(w=0x200002), dict(mean=0x400002),
    dict(out=0x100010), dict(out=0x200000), dict(mean=0x100100), dict(rstd=0x300010),
])
def test_refusals_before_any_launch(lib, kw):
    assert forward_call(lib, **kw) == EINVAL, lib.tgs_last_error()
    assert b"layer_norm" in lib.tgs_last_error()
    if kw in (dict(rstd=0x300010), dict(mean=0x100100)):
        kw = dict(out=0x410000)  # the gradient reads the statistics, its inputs may overlap
    assert grad_call(lib, **kw) == EINVAL, lib.tgs_last_error()
    assert b"layer_norm_grad" in lib.tgs_last_error()


def test_refusals_of_each(lib):
    for eps in (-1.0, float("nan"), float("inf")):
        assert forward_call(lib, eps=eps) == EINVAL
    assert forward_call(lib, ot=4) == EINVAL
    assert forward_call(lib, rstd=0x400010) == EINVAL
    assert forward_call(lib, out=0x100000, ot=1) == EINVAL  # in place, of another type
    assert grad_call(lib, gt=3) == EINVAL
    assert grad_call(lib, pt=3) == EINVAL
    assert grad_call(lib, g=None) == EINVAL
    assert grad_call(lib, mean=None) == EINVAL
    assert grad_call(lib, rstd=None) == EINVAL
    assert grad_call(lib, ws=None) == EINVAL
    assert grad_call(lib, ws=0x1000010) == EINVAL
    assert grad_call(lib, gw=0x430000) == EINVAL       # over the bias's
    assert grad_call(lib, gw=0x1000100) == EINVAL      # in the workspace
    assert grad_call(lib, out=0x500000, gt=1) == EINVAL  # in place of a gradient of another type
    assert grad_call(lib, gb=0x400000) == EINVAL
    need = lib.tgs_layer_norm_grad_workspace_bytes(16, 8)
    assert need >= 32768 and grad_call(lib, wsn=need - 1) == EWORKSPACE
    for T, D in ((1, 2**24), (10**6, 2**20), (10**6, 40_000), (10**6, 16_384), (10**6, 512), (2**31 - 1, 1)):
        assert 32768 < lib.tgs_layer_norm_grad_workspace_bytes(T, D) <= 32768 + max(2**25, 8 * D)
    for bad in ((-1, 8), (2**31, 8), (8, 0), (8, 2**24 + 1)):
        assert lib.tgs_layer_norm_grad_workspace_bytes(*bad) == 0


def test_binding_refusals_on_the_cpu():
    import top_gradient_sparsification_amd as tgs
    x, s = torch.zeros(4, 8), torch.zeros(4)
    with pytest.raises(TypeError, match="GPU tensor"):
        tgs.layer_norm(x)
    with pytest.raises(TypeError, match="x must be one of"):
        tgs.layer_norm(x.double())
    with pytest.raises(TypeError, match="GPU tensor"):
        tgs.layer_norm_grad(x, x, s, s)


def test_the_definitions_agree_with_differences():
    gen = torch.Generator().manual_seed(5)
    x, w, b, g = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((3, 7), (7,), (7,), (3, 7)))
    _, _, (mean, _), (rstd, _) = exact_norm(x, w, b, 1e-5)
    (gx, _), (gw, _), (gb, _) = exact_grad(g, x, mean[:, 0], rstd[:, 0], w)

    def loss(x, w, b):
        return (exact_norm(x, w, b, 1e-5)[0] * g).sum()

    h = 1e-6
    for t, got in ((x, gx), (w, gw), (b, gb)):
        for i in range(t.numel()):
            step = torch.zeros_like(t)
            step.view(-1)[i] = h
            up, down = (loss(*(p + s * step if p is t else p for p in (x, w, b))) for s in (1, -1))
            assert abs((up - down) / (2 * h) - got.reshape(-1)[i]) < 1e-7
    with pytest.raises(AssertionError):
        assert_close(gx + 1e-3, gx, torch.full_like(gx, 1e-6))


# ------------------------------------------------------------------- GPU --
WIDTHS = [1, 2, 3, 7, 8, 9, 31, 64, 65, 130, 255, 256, 257, 500, 513, 1001, 1024, 1500, 2048, 2049, 4096, 4100, 8191,
          8192, 8200, 16384, 16391, 40001]


@pytest.mark.gpu
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(tgs_gpu, D):
    for dtype, wt, T in ((torch.float32, torch.float32, 5), (torch.bfloat16, torch.float32, 37),
                         (torch.float16, torch.float16, 3)):
        x = make(T, D, dtype, D)
        check(tgs_gpu, x, *params(D, wt, D + 1))


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", FLOATS)
@pytest.mark.parametrize("dtype", FLOATS)
def test_types(tgs_gpu, dtype, out_dtype):
    for D in (24, 130, 1001, 3000, 9001):
        for wt in FLOATS:
            check(tgs_gpu, make(9, D, dtype, D), *params(D, wt, 3), out_dtype=out_dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("T,D", [(1, 4096), (2, 8), (33, 64), (1000, 40), (5000, 130), (517, 131), (3001, 2048), (1029, 5000),
                                 (700, 16384), (150, 20000)])
def test_rows(tgs_gpu, T, D):
    for dtype in (torch.float32, torch.bfloat16):
        check(tgs_gpu, make(T, D, dtype, T), *params(D, torch.float32, 2))


@pytest.mark.gpu
def test_without_weight_or_bias_and_shapes(tgs_gpu):
    x = make(24, 200, torch.bfloat16, 1).view(2, 3, 4, 200)
    w, b = params(200, torch.bfloat16, 1)
    for ww, bb in ((None, None), (w, None), (None, b)):
        check(tgs_gpu, x, ww, bb)
    _, mean, rstd = tgs_gpu.layer_norm(x, w, b, return_stats=True)
    gx, gw, gb = tgs_gpu.layer_norm_grad(x, x, mean, rstd, w, params=False)
    assert gw is None and gb is None
    same, gw, gb = tgs_gpu.layer_norm_grad(x, x, mean, rstd, w, param_dtype=torch.float32)
    assert torch.equal(gx, same) and gw.dtype == gb.dtype == torch.float32
    assert tgs_gpu.layer_norm(x[0, 0, 0], w, b).shape == (200,)
    empty = x[:0]
    assert tgs_gpu.layer_norm(empty, w, b).shape == (0, 3, 4, 200)
    gx, gw, gb = tgs_gpu.layer_norm_grad(empty, empty, mean[:0], rstd[:0], w)
    assert gx.shape == empty.shape and not gw.any() and not gb.any()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [40, 300, 2048, 6000, 16384, 17000])
def test_in_place(tgs_gpu, D):
    x, (w, b) = make(19, D, torch.float32, D), params(D, torch.float32, 4)
    y, mean, rstd = tgs_gpu.layer_norm(x, w, b, return_stats=True)
    at = x.clone()
    version = at._version
    assert tgs_gpu.layer_norm(at, w, b, out=at) is at and torch.equal(at, y) and at._version > version
    g = make(19, D, torch.float32, 6)
    want = tgs_gpu.layer_norm_grad(g, x, mean, rstd, w)
    for place in (x.clone(), g.clone()):
        given = (g, place) if torch.equal(place, x) else (place, x)
        got = tgs_gpu.layer_norm_grad(*given, mean, rstd, w, out=place)
        assert got[0] is place
        for a, c in zip(got, want):
            assert torch.equal(a, c)


@pytest.mark.gpu
def test_rows_far_from_zero_and_constant_rows(tgs_gpu):
    for D in (64, 1000, 5000, 20000):
        x = make(7, D, torch.float32, D, mean=1000.0, scale=1.0)
        x[1] = 3.25           # no variance: xh = 0 and y = bias
        x[2] = make(1, D, torch.float32, 9, scale=1e-4)[0]
        x[3] = 1e18 * make(1, D, torch.float32, 8)[0]
        w, b = params(D, torch.float32, 2)
        check(tgs_gpu, x, w, b, grad=False)
        assert torch.equal(tgs_gpu.layer_norm(x, w, b)[1], b)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [8, 130, 2048, 4096, 17000])
def test_a_bad_row_stays_alone(tgs_gpu, D):
    x = make(12, D, torch.float32, 3)
    w, b = params(D, torch.float32, 2)
    want, mean, rstd = tgs_gpu.layer_norm(x, w, b, return_stats=True)
    bad = x.clone()
    bad[5, D // 2], bad[9, 0] = float("nan"), float("inf")
    got, bm, br = tgs_gpu.layer_norm(bad, w, b, return_stats=True)
    rows = torch.tensor([5, 9], device="cuda")
    keep = torch.ones(12, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[rows]).any(1).all()
    gx, _, _ = tgs_gpu.layer_norm_grad(x, bad, bm, br, w)
    ok, _, _ = tgs_gpu.layer_norm_grad(x, x, mean, rstd, w)
    assert torch.equal(gx[keep], ok[keep]) and torch.isnan(gx[5]).all()


@pytest.mark.gpu
def test_offsets_past_32_bits(tgs_gpu):
    """2.2e9 values: the last rows against a call on them alone."""
    D, T = 2048, 1_075_000
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    x[:-4000] = 1.0
    x[-4000:] = make(4000, D, torch.bfloat16, 1)
    w, b = params(D, torch.bfloat16, 2)
    y, mean, rstd = tgs_gpu.layer_norm(x, w, b, return_stats=True)
    part, pm, pr = tgs_gpu.layer_norm(x[-4000:], w, b, return_stats=True)
    assert torch.equal(y[-4000:], part) and torch.equal(mean[-4000:], pm) and torch.equal(rstd[-4000:], pr)
    assert torch.equal(y[:4], b.expand(4, D))
    gx, gw, gb = tgs_gpu.layer_norm_grad(y, x, mean, rstd, w, param_dtype=torch.float32)
    px, _, _ = tgs_gpu.layer_norm_grad(part, x[-4000:], pm, pr, w)
    assert torch.equal(gx[-4000:], px)


@pytest.mark.gpu
def test_very_long_rows(tgs_gpu):
    D = 300_001
    x = make(40, D, torch.bfloat16, 1)
    check(tgs_gpu, x, *params(D, torch.float32, 2))


@pytest.mark.gpu
@pytest.mark.parametrize("T,D", [(517, 131), (1024, 256), (1025, 256), (4096, 100), (8192, 60), (8193, 60), (64, 257)])
def test_either_side_of_the_one_launch_rule(tgs_gpu, T, D):
    """The gradient twice on one workspace of the caller's: its counter is left as it was found."""
    for dtype in (torch.float32, torch.bfloat16):
        x, (w, b) = make(T, D, dtype, 3), params(D, torch.float32, 4)
        first = check(tgs_gpu, x, w, b)
        ws = torch.zeros(tgs_gpu.layer_norm_grad_workspace_bytes(T, D), dtype=torch.uint8, device="cuda")
        _, mean, rstd = tgs_gpu.layer_norm(x, w, b, return_stats=True)
        for _ in range(3):
            for got, want in zip(tgs_gpu.layer_norm_grad(first[1], x, mean, rstd, w, ws=ws), first[2:]):
                assert torch.equal(got, want)
            assert not ws[:32768].any()


@pytest.mark.gpu
def test_gradients_flow(tgs_gpu):
    x, (w, b) = make(40, 96, torch.float32, 1).view(5, 8, 96), params(96, torch.float32, 2)
    x, w, b = (t.requires_grad_() for t in (x, w, b))
    y = tgs_gpu.layer_norm(x, w, b)
    g = make(40, 96, torch.float32, 5).view(5, 8, 96)
    got = torch.autograd.grad(y, (x, w, b), g)
    _, mean, rstd = tgs_gpu.layer_norm(x.detach(), w.detach(), b.detach(), return_stats=True)
    for a, c in zip(got, tgs_gpu.layer_norm_grad(g, x.detach(), mean, rstd, w.detach())):
        assert torch.equal(a, c)
    (only,) = torch.autograd.grad(tgs_gpu.layer_norm(x.detach(), w, b.detach()).sum(), w)  # an expanded gradient
    assert only.shape == w.shape
    # the directional derivative in 64 bits
    v = make(40, 96, torch.float32, 7).view(5, 8, 96).double().cpu()
    h = 1e-6
    up, down = (exact_norm(x.detach().double().cpu() + s * h * v, w, b, 1e-5)[0] for s in (1, -1))
    want = ((up - down) / (2 * h) * g.double().cpu()).sum()
    assert abs((got[0].double().cpu() * v).sum() - want) < 1e-4 * want.abs() + 1e-4
    y, mean, _ = tgs_gpu.layer_norm(x, w, b, return_stats=True)
    assert y.requires_grad and not mean.requires_grad
    with pytest.raises(RuntimeError, match="out="):
        tgs_gpu.layer_norm(x, w, b, out=torch.empty_like(x))
    back = tgs_gpu.layer_norm_grad(g, x, mean, mean, w)
    with pytest.raises(NotImplementedError, match="layer_norm_grad has no gradient"):
        back[0].sum().backward()
    (gx,) = torch.autograd.grad(tgs_gpu.layer_norm(x, w, b).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()
    with torch.no_grad():
        assert not tgs_gpu.layer_norm(x, w, b).requires_grad


@pytest.mark.gpu
def test_binding_refusals(tgs_gpu):
    x = make(6, 32, torch.float32, 1)
    w, b = params(32, torch.float32, 1)
    s = torch.zeros(6, device="cuda")
    for call, error in ((lambda: tgs_gpu.layer_norm(x[:, :16]), "contiguous"),
                        (lambda: tgs_gpu.layer_norm(x, w[:16]), "weight must have shape"),
                        (lambda: tgs_gpu.layer_norm(x, w, b.half()), "bias must be one of"),
                        (lambda: tgs_gpu.layer_norm(x, out=x[:3]), "out must have shape"),
                        (lambda: tgs_gpu.layer_norm(x, out_dtype=torch.int32), "out_dtype"),
                        (lambda: tgs_gpu.layer_norm(x, eps=-1.0), "eps"),
                        (lambda: tgs_gpu.layer_norm(x[:, :0].contiguous()), "D=0"),
                        (lambda: tgs_gpu.layer_norm(x, out=x.view(-1)[:192].view(6, 32).half()[:5]), "shape"),
                        (lambda: tgs_gpu.layer_norm_grad(x[:5], x, s, s), "grad must have shape"),
                        (lambda: tgs_gpu.layer_norm_grad(x, x, s[:5], s), "mean must have shape"),
                        (lambda: tgs_gpu.layer_norm_grad(x, x, s, s.half()), "rstd must be one of"),
                        (lambda: tgs_gpu.layer_norm_grad(x, x, s, s, param_dtype=torch.int64), "param_dtype"),
                        (lambda: tgs_gpu.layer_norm_grad(x, x, s, s, ws=torch.zeros(99, dtype=torch.uint8)), "ws is on cpu"),
                        (lambda: tgs_gpu.layer_norm_grad(x, x, s, s, ws=torch.zeros(256, dtype=torch.uint8, device="cuda")),
                         "need")):
        with pytest.raises((ValueError, TypeError, MemoryError), match=error):
            call()


def test_tolerances_are_tight():
    """What a mean of one rounding less, or a single bf16 sum, would give lies outside them."""
    gen = torch.Generator().manual_seed(0)
    x = 0.3 + torch.randn(64, 2048, generator=gen)
    y, tol, _, _ = exact_norm(x, None, None, 1e-5)
    assert (tol < 2e-5 * (1 + y.abs())).all()
    coarse = (x - x.bfloat16().float().mean(-1, keepdim=True)).double() * y.std() / (x.double() - x.double().mean(-1, keepdim=True)).std()
    with pytest.raises(AssertionError):
        assert_close(coarse, y, tol)
    assert half_step(torch.float32) == U and tiny(torch.float32) == 2.0**-150


@pytest.mark.gpu
@pytest.mark.parametrize("D", [7, 64, 130, 1001, 5000, 16384, 20_001, 300_001, 1 << 20, 1 << 24])
def test_rows_of_one_value(tgs_gpu, D):
    """y = bias, whatever the value and however many of it are summed.

    The mean is the value itself: the first one is off by k roundings at most (k < 700 for D = 2^24), each value's
    distance to it is exact, and those distances' mean, off by 650 U of itself at most, brings it within 0.03 of
    a step of the value."""
    w, b = params(D, torch.float32, 2)
    other = make(1, D, torch.float32, 3)
    for dtype in (torch.float32, torch.bfloat16):
        alone = tgs_gpu.layer_norm(other.to(dtype), w, b)
        for value in (0.0, 0.1, 1000.1, -3.3e-21, 7e15, 2e38, torch.finfo(dtype).min):
            for eps in (1e-5, 2.0**-125):
                x = torch.full((3, D), value, device="cuda")
                x[1] = other
                x = x.to(dtype)
                y, mean, rstd = tgs_gpu.layer_norm(x, w, b, eps=eps, out_dtype=torch.float32, return_stats=True)
                assert torch.equal(y[::2], b.expand(2, D)), (value, eps)
                assert torch.equal(mean[::2], x[::2, 0].float()), (value, eps)
                # the root and the division, and eps itself as a float
                want = torch.full((2,), eps**-0.5, dtype=torch.float64)
                assert_close(rstd[::2], want, 3 * U * want, "rstd")
                if eps == 1e-5:
                    assert torch.equal(tgs_gpu.layer_norm(x, w, b)[1], alone[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [7, 64, 130, 1001, 5000, 20000, 33000])
def test_rows_whose_squares_fall_below_the_range(tgs_gpu, D, dtype):
    """Without an eps, or with one as small, rows of the smallest values are normed like any other."""
    w, b = params(D, torch.float32, 2)
    for size in (1e-15, 1e-18, 1e-22, 1e-25, 1e-30, 1e-37):
        x = size * make(9, D, torch.float32, D)
        x[1:4] = make(3, D, torch.float32, 5)          # beside rows of ordinary ones
        check(tgs_gpu, x.to(dtype), w, b, eps=0.0)
        check(tgs_gpu, x.to(dtype), w, b, eps=2.0**-125)
    x = (1e-41 * make(3, D, torch.float32, D).cpu()).cuda()  # rstd is no fp32 number, the results are
    want, tol, _, _ = exact_norm(x, w, b, 0.0)
    assert_close(tgs_gpu.layer_norm(x, w, b, eps=0.0), want, tol + rounded(want, torch.float32), "y")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [7, 130, 1001, 5000, 33000])
def test_gradients_of_rows_wider_than_the_type(tgs_gpu, D, dtype):
    """x - mean is no fp32 number, (x - mean) rstd is one."""
    x = make(9, D, torch.float32, D)
    x[2:7] = torch.where(x[2:7] > 0.9, 3.2e38, -3.2e38)
    check(tgs_gpu, x.to(dtype), *params(D, torch.float32, 3))
