"""Newton-Schulz orthogonalisation and the Muon step.

The oracle is the definition in 64 bits.  Tolerances are relative 2-norms over
a matrix, derived from the roundings:
* 16-bit results: in each of the (at most 10 here) steps three operands are
  rounded to fp16 (half step 2^-11, rms 0.4 of that), independently; the
  parts so rounded are at most 1.5 times the result.  sqrt(3 * 10) * 0.4 *
  2^-11 * 1.5 < 2^-9.  The final rounding adds at most eps / 2.
* fp32 results: operands hold 22 bits and sums are fp32: each of the (at most
  30) products is off by about 2^-22, times sqrt(30) and a gain of at most 3:
  2^-18.
Two things raise what the steps leave: directions in which the input is empty
(what is rounded into them grows by the first coefficient a step while the
strong directions stay: up to 140 in four steps, of which a share of about
1 / sqrt(rows) counts; 16 is allowed), and more than five steps of the quintic
(its slope between steps reaches 1.6 near 0.87).
"""
import ctypes
import math

import numpy as np
import pytest
import torch

U = 2.0**-24
QUINTIC = (3.4445, -4.7750, 2.0315)
FLOATS = (torch.float32, torch.bfloat16, torch.float16)
EINVAL, EWORKSPACE = -1, -2


def tolerance(dtype, gain=1.0):
    return gain * 2.0**-18 if dtype == torch.float32 else gain * 2.0**-9 + torch.finfo(dtype).eps / 2


def exact(x, steps=5, coefficients=QUINTIC, eps=1e-7):
    a, b, c = coefficients
    y = x.double()
    y = y / (y.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    tall = y.shape[-2] > y.shape[-1]
    if tall:
        y = y.mT
    for _ in range(steps):
        g = y @ y.mT
        y = a * y + (b * g + c * (g @ g)) @ y
    return y.mT if tall else y


def distance(got, want):
    """The largest relative 2-norm of the difference over the stack."""
    d = (got.double().cpu() - want).flatten(-2).norm(dim=-1)
    return float((d / want.flatten(-2).norm(dim=-1)).max())


def matrices(shape, seed, noise=0.3, dtype=torch.float32):
    """Gradient-like: a few strong directions and noise."""
    rng = np.random.default_rng(seed)
    *b, m, n = shape
    r = max(1, min(m, n) // 16)
    u = rng.standard_normal((*b, m, r)) / np.arange(1, r + 1)
    x = u @ rng.standard_normal((*b, r, n)) + noise * rng.standard_normal(shape)
    return torch.from_numpy((x / math.sqrt(m * n)).astype(np.float32)).to(dtype)


# ------------------------------------------------------------------- CPU --
def abi():
    import top_gradient_sparsification_amd as tgs
    return tgs.library()


def ns_call(lib, **kw):
    a = dict(x=0x100000, dt=0, batch=1, rows=64, cols=64, steps=5, a=3.0, b=-4.0, c=2.0, eps=1e-7, out=0x200000,
             ws=0x1000000, wsn=1 << 30)
    a.update(kw)
    p = ctypes.c_void_p
    return lib.tgs_newton_schulz(p(a["x"]), a["dt"], a["batch"], a["rows"], a["cols"], a["steps"], a["a"], a["b"],
                                 a["c"], a["eps"], p(a["out"]), p(a["ws"]), a["wsn"], None)


def muon_call(lib, **kw):
    a = dict(w=0x200000, wt=0, x=0x100000, dt=0, mom=0x300000, batch=1, rows=64, cols=64, lr=0.02, beta=0.9, nest=1,
             wd=0.0, steps=5, a=3.0, b=-4.0, c=2.0, eps=1e-7, ws=0x1000000, wsn=1 << 30)
    a.update(kw)
    p = ctypes.c_void_p
    return lib.tgs_muon_step(p(a["w"]), a["wt"], p(a["x"]), a["dt"], p(a["mom"]), a["batch"], a["rows"], a["cols"],
                             a["lr"], a["beta"], a["nest"], a["wd"], a["steps"], a["a"], a["b"], a["c"], a["eps"],
                             p(a["ws"]), a["wsn"], None)


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=65536), dict(rows=0), dict(cols=0), dict(rows=65537), dict(cols=65537), dict(dt=3),
    dict(dt=-1), dict(steps=0), dict(steps=65), dict(a=float("nan")), dict(b=float("inf")), dict(c=float("-inf")),
    dict(eps=-1e-3), dict(eps=float("nan")), dict(x=None), dict(x=0x100002), dict(ws=None), dict(ws=0x1000080),
    dict(a=1e10), dict(a=10.0, b=0.0, c=0.0, steps=20),  # singular values would pass 2^30
    dict(x=0x1000000 + 4096),                            # in the workspace
])
def test_refusals_before_any_launch(kw):
    lib = abi()
    assert ns_call(lib, **kw) == EINVAL, lib.tgs_last_error()
    assert b"newton_schulz" in lib.tgs_last_error()
    assert muon_call(lib, **kw) == EINVAL, lib.tgs_last_error()
    assert b"muon_step" in lib.tgs_last_error()


def test_refusals_of_each():
    lib = abi()
    assert ns_call(lib, out=None) == EINVAL
    assert ns_call(lib, out=0x100100) == EINVAL  # over x, and not x itself
    for kw in (dict(w=None), dict(mom=None), dict(mom=0x300002), dict(wt=4), dict(lr=float("nan")),
               dict(beta=float("inf")), dict(wd=float("nan")), dict(w=0x100100), dict(mom=0x100100),
               dict(mom=0x200100), dict(mom=0x1000000 + 4096)):
        assert muon_call(lib, **kw) == EINVAL, kw
    for dt in range(3):
        need = lib.tgs_newton_schulz_workspace_bytes(2, 100, 300, dt)
        assert need >= 32768 and lib.tgs_muon_workspace_bytes(2, 100, 300, dt) == need
        assert ns_call(lib, batch=2, rows=100, cols=300, dt=dt, wsn=need - 1) == EWORKSPACE
        assert muon_call(lib, batch=2, rows=100, cols=300, dt=dt, wt=dt, wsn=need - 1) == EWORKSPACE
    for bad in ((0, 4, 4, 0), (1, 0, 4, 0), (1, 4, 70_000, 0), (1, 4, 4, 3)):
        assert lib.tgs_newton_schulz_workspace_bytes(*bad) == 0


def test_binding_refusals_on_the_cpu():
    import top_gradient_sparsification_amd as tgs
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError, match="GPU tensor"):
        tgs.newton_schulz(x)
    with pytest.raises(TypeError, match="x must be one of"):
        tgs.newton_schulz(x.double())
    with pytest.raises(TypeError, match="GPU tensor"):
        tgs.muon_step(x, x, x, lr=0.1)


def test_the_oracle_on_closed_forms():
    # a multiple of an orthogonal matrix: every singular value takes the scalar recurrence
    q = torch.linalg.qr(torch.from_numpy(np.random.default_rng(0).standard_normal((6, 6))))[0]
    s = 1.0 / math.sqrt(6)
    a, b, c = QUINTIC
    for _ in range(5):
        s = s * (a + b * s**2 + c * s**4)
    assert torch.allclose(exact(7.0 * q, eps=0.0), s * q, atol=1e-12)
    assert torch.allclose(exact(q[:, :2] * 3, eps=0.0), exact((q[:, :2] * 3).mT, eps=0.0).mT, atol=1e-14)
    assert distance(exact(q) * (1 + 1e-3), exact(q)) > 9e-4  # the measure sees a planted mistake


# ------------------------------------------------------------------- GPU --
SHAPES = [(1, 1), (1, 9), (9, 1), (3, 5), (33, 31), (64, 64), (65, 63), (127, 129), (40, 700), (1000, 24),
          (130, 1030), (300, 200), (513, 520), (530, 1100), (1100, 530), (3, 20, 36), (5, 70, 33), (2, 520, 640),
          # shorter side up to 64: one workgroup a matrix, then chunks of columns
          (64, 512), (513, 64), (30, 1024), (1025, 20), (32, 257), (129, 33), (16, 128), (1, 5000), (64, 8192),
          (8192, 31), (40, 40, 2000), (130, 1500, 17), (7, 64, 600)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", FLOATS)
def test_orthogonalise_sizes_and_types(tgs_gpu, shape, dtype):
    x = matrices(shape, seed=sum(shape), dtype=dtype)
    b, m, n = (1, *shape)[-3:]
    ws = torch.full((tgs_gpu.newton_schulz_workspace_bytes(b, m, n, dtype),), 0xFF, dtype=torch.uint8, device="cuda")
    dev = x.cuda()
    got = tgs_gpu.newton_schulz(dev, ws=ws)  # scratch holds NaN bits
    assert got.dtype == dtype and got.shape == x.shape
    assert torch.equal(dev.cpu(), x)
    assert distance(got, exact(x)) <= tolerance(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("coefficients,steps", [
    ((1.5, -0.5, 0.0), 10), ((1.875, -1.25, 0.375), 7), ((2.0, -1.5, 0.5), 1), ((1.0, 0.0, 0.0), 2),
    ((0.5, 0.25, 0.0), 3), (QUINTIC, 1), (QUINTIC, 2), (QUINTIC, 10)])
def test_coefficients_and_steps(tgs_gpu, dtype, coefficients, steps):
    x = matrices((90, 150), seed=steps, dtype=dtype)
    got = tgs_gpu.newton_schulz(x.cuda(), steps=steps, coefficients=coefficients)
    gain = 1.6**max(0, steps - 5) if coefficients == QUINTIC else 1.0
    assert distance(got, exact(x, steps, coefficients)) <= tolerance(dtype, gain)


@pytest.mark.gpu
@pytest.mark.parametrize("noise", [0.0, 0.1, 1.0])
@pytest.mark.parametrize("shape", [(96, 160), (530, 600)])
@pytest.mark.parametrize("dtype", FLOATS)
def test_spectra(tgs_gpu, noise, shape, dtype):
    """From rank-deficient to nearly white."""
    x = matrices(shape, seed=5, noise=noise, dtype=dtype)
    assert distance(tgs_gpu.newton_schulz(x.cuda()), exact(x)) <= tolerance(dtype, 16.0 if noise == 0.0 else 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 1e30])
def test_scale_of_the_input_does_not_matter(tgs_gpu, scale):
    x = matrices((70, 90), seed=1)
    got = tgs_gpu.newton_schulz((x * scale).cuda(), eps=0.0)
    assert distance(got, exact(x * scale, eps=0.0)) <= tolerance(torch.float32)
    # eps against a small norm
    got = tgs_gpu.newton_schulz((x * 1e-6).cuda(), eps=1e-6)
    assert distance(got, exact(x * 1e-6, eps=1e-6)) <= tolerance(torch.float32)


@pytest.mark.gpu
def test_zeros_nans_and_neighbours_in_a_batch(tgs_gpu):
    x = matrices((4, 50, 70), seed=2)
    x[1] = 0
    x[2, 3, 4] = float("nan")
    x[3, 49, 0] = float("inf")
    for dtype in FLOATS:
        y = x.to(dtype)
        got = tgs_gpu.newton_schulz(y.cuda()).cpu()
        assert distance(got[:1], exact(y[:1])) <= tolerance(dtype)
        assert (got[1] == 0).all()
        assert got[2].isnan().all() and got[3].isnan().all()
    # a column of zeros, and rows that repeat
    z = matrices((60, 80), seed=3)
    z[:, 5] = 0
    z[7] = z[8]
    got = tgs_gpu.newton_schulz(z.cuda())
    assert (got[:, 5] == 0).all() and distance(got, exact(z)) <= tolerance(torch.float32)


@pytest.mark.gpu
def test_views_in_place_and_refusals(tgs_gpu):
    x = matrices((40, 33), seed=4)
    flat = torch.zeros(1 + x.numel())
    flat[1:] = x.flatten()
    dev = flat.cuda()[1:].view(40, 33)  # 4-byte aligned only
    want = tgs_gpu.newton_schulz(x.cuda())
    assert torch.equal(tgs_gpu.newton_schulz(dev), want)
    assert tgs_gpu.newton_schulz(dev, out=dev) is dev and torch.equal(dev, want)
    assert tgs_gpu.newton_schulz(dev[:0]).shape == (0, 33)
    with pytest.raises(ValueError, match="contiguous"):
        tgs_gpu.newton_schulz(dev.t())
    with pytest.raises(ValueError, match="shape"):
        tgs_gpu.newton_schulz(dev.flatten())
    with pytest.raises(ValueError, match="shape"):
        tgs_gpu.newton_schulz(dev, out=dev[:3])
    with pytest.raises(TypeError):
        tgs_gpu.newton_schulz(dev, out=dev.half())
    with pytest.raises(ValueError, match="2\\^30"):
        tgs_gpu.newton_schulz(dev, coefficients=(1e9, 0.0, 0.0))
    with pytest.raises(ValueError, match="one shape"):
        tgs_gpu.muon_step(dev, dev[:3], dev, lr=0.1)
    with pytest.raises(TypeError):
        tgs_gpu.muon_step(dev, dev, dev.half(), lr=0.1)
    with pytest.raises(ValueError, match="overlap"):
        tgs_gpu.muon_step(dev, dev, dev.clone(), lr=0.1)


def matrices_gpu(shape, seed, noise=0.3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    b, m, n = shape
    r = max(1, min(m, n) // 16)
    u = torch.randn(b, m, r, device="cuda", generator=gen) / torch.arange(1, r + 1, device="cuda")
    x = torch.bmm(u, torch.randn(b, r, n, device="cuda", generator=gen))
    return (x + noise * torch.randn(shape, device="cuda", generator=gen)) / math.sqrt(m * n)


def distance_gpu(got, want):
    d = (got.double() - want).flatten(-2).norm(dim=-1)
    return float((d / want.flatten(-2).norm(dim=-1)).max())


# a size for every way a product is cut: whole matrices in one workgroup's LDS, tiles of 64
# (with long stages, shared), 128 (with a long ring), 192 and 256, hanging over or not
CUTS = [(1, 128, 128), (3, 65, 384), (2, 384, 66), (5, 100, 256), (300, 70, 90), (1, 129, 129), (1, 393, 393),
        (2, 129, 2029), (1, 2029, 129), (1, 200, 8000), (1, 129, 899), (33, 129, 129), (100, 129, 409), (64, 409, 129),
        (64, 129, 829), (33, 261, 261), (64, 261, 541), (64, 393, 393), (16, 556, 556), (8, 686, 1316),
        (16, 1206, 1346), (1, 6036, 1466), (3, 2246, 2246), (5, 2246, 2246)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", CUTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_cut_of_the_products(tgs_gpu, shape, dtype):
    x = matrices_gpu(shape, seed=sum(shape)).to(dtype)
    ws = torch.full((tgs_gpu.newton_schulz_workspace_bytes(*shape, dtype),), 0xFF, dtype=torch.uint8, device="cuda")
    got = tgs_gpu.newton_schulz(x, ws=ws)  # scratch holds NaN bits
    assert distance_gpu(got, exact(x)) <= tolerance(dtype)
    assert torch.equal(tgs_gpu.newton_schulz(x, ws=ws), got)  # whatever order workgroups arrive in


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 128, 128), (3, 100, 70), (1, 300, 90), (2, 1315, 687), (1, 1466, 6036),
                                   (1, 2246, 2246), (1, 8000, 200)])
@pytest.mark.parametrize("weight_dtype", [torch.bfloat16, torch.float32])
def test_muon_step_of_every_cut(tgs_gpu, shape, weight_dtype):
    lr, beta, wd = 0.02, 0.95, 0.1
    w = (0.02 * matrices_gpu(shape, 1, noise=1.0) * math.sqrt(shape[1] * shape[2])).to(weight_dtype)
    g, m = matrices_gpu(shape, 2).bfloat16(), 5 * matrices_gpu(shape, 3)
    want_w, want_m, moved = muon_exact(w, g, m, lr, beta, True, wd)
    old_w, old_m = w.double(), m.double()
    tgs_gpu.muon_step(w, g, m, lr, beta=beta, weight_decay=wd)
    assert ((m.double() - want_m).abs() <= (beta * old_m.abs() + want_m.abs()) * 1.01 * U).all()
    off = (w.double() - want_w).flatten(-2).norm(dim=-1)
    inner = 2.0**-18 if weight_dtype == torch.float32 else 2.0**-9
    tol = moved.flatten(-2).norm(dim=-1) * (inner + 2 * U) + old_w.flatten(-2).norm(dim=-1) * 2 * U + (
        want_w.flatten(-2).norm(dim=-1) * (U + torch.finfo(weight_dtype).eps / 2))
    assert (off <= tol).all()


@pytest.mark.gpu
def test_a_nan_stays_in_its_matrix_of_a_stack(tgs_gpu):
    for shape in ((3, 128, 100), (3, 200, 150), (3, 129, 2029)):
        for dtype in (torch.bfloat16, torch.float32):
            x = matrices_gpu(shape, 7).to(dtype)
            x[1, 5, 6] = float("nan")
            got = tgs_gpu.newton_schulz(x)
            assert got[1].isnan().all()
            for i in (0, 2):
                assert torch.equal(got[i], tgs_gpu.newton_schulz(x[i:i + 1])[0]) or distance_gpu(
                    got[i:i + 1], exact(x[i:i + 1])) <= tolerance(dtype)


def muon_exact(w, g, m, lr, beta, nesterov, wd):
    g, m = g.double(), m.double()
    m = beta * m + g
    o = exact(g + beta * m if nesterov else m)
    s = math.sqrt(max(1.0, w.shape[-2] / w.shape[-1]))
    return w.double() * (1 - lr * wd) - lr * s * o, m, lr * s * o


@pytest.mark.gpu
@pytest.mark.parametrize("weight_dtype", FLOATS)
@pytest.mark.parametrize("grad_dtype", FLOATS)
@pytest.mark.parametrize("shape,nesterov", [((33, 50), True), ((129, 40), False), ((2, 70, 90), True),
                                            ((3, 2000, 30), True), ((50, 700), True),
                                            ((530, 700), False)])
def test_muon_step(tgs_gpu, weight_dtype, grad_dtype, shape, nesterov):
    lr, beta, wd = 0.02, 0.95, 0.1
    w = matrices(shape, seed=1, noise=1.0, dtype=weight_dtype)
    g = matrices(shape, seed=2, dtype=grad_dtype)
    m = 5 * matrices(shape, seed=3)
    want_w, want_m, moved = muon_exact(w, g, m, lr, beta, nesterov, wd)
    dw, dg, dm = w.cuda(), g.cuda(), m.cuda()
    assert tgs_gpu.muon_step(dw, dg, dm, lr, beta=beta, nesterov=nesterov, weight_decay=wd) is dw
    assert torch.equal(dg.cpu(), g)
    # beta to fp32, one fused multiply-add
    assert ((dm.cpu().double() - want_m).abs() <= (beta * m.double().abs() + want_m.abs()) * 1.01 * U).all()
    # the move is as exact as an orthogonalisation in fp32 or 16 bits; lr, keep, gain and the sum are
    # rounded to fp32 (four roundings), the weight to its type
    off = (dw.cpu().double() - want_w).flatten(-2).norm(dim=-1)
    inner = 2.0**-18 if weight_dtype == torch.float32 else 2.0**-9
    tol = moved.flatten(-2).norm(dim=-1) * (inner + 2 * U) + (
        w.double().flatten(-2).norm(dim=-1) * 2 * U + want_w.flatten(-2).norm(dim=-1) * (
            U + torch.finfo(weight_dtype).eps / 2))
    assert (off <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shape,dtype", [((2, 60, 40), torch.bfloat16), ((520, 700), torch.float32)])
def test_same_bits_every_run_on_any_stream_and_in_a_graph(tgs_gpu, shape, dtype):
    w, g, m = (matrices(shape, seed=s, dtype=d).cuda() for s, d in ((1, dtype), (2, dtype), (3, torch.float32)))
    want = tgs_gpu.newton_schulz(g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert torch.equal(tgs_gpu.newton_schulz(g), want)
    side.synchronize()
    b, rows, cols = (1, *shape)[-3:]
    ws = torch.zeros(tgs_gpu.muon_workspace_bytes(b, rows, cols, dtype), dtype=torch.uint8, device="cuda")
    w2, m2, o2 = w.clone(), m.clone(), torch.empty_like(g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tgs_gpu.muon_step(w2, g, m2, lr=0.05, ws=ws)
        tgs_gpu.newton_schulz(g, out=o2, ws=ws)
    for seed in (4, 5, 6):
        g.copy_(matrices(shape, seed=seed, dtype=dtype))
        graph.replay()
        torch.cuda.synchronize()
        tgs_gpu.muon_step(w, g, m, lr=0.05)
        assert torch.equal(w2, w) and torch.equal(m2, m)
        assert torch.equal(o2, tgs_gpu.newton_schulz(g))
