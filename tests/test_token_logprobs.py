"""Log probabilities of given tokens, with entropy and top alternatives, and
the logits' gradient, against their definitions in 64 bits (tolerances in
``_rows``)."""
import ctypes
import math

import pytest
import torch

from _rows import FLOATS, U, Softmax, assert_close, rounded, scores

EINVAL, EWORKSPACE = -1, -2
LOWEST = {t: torch.finfo(t).min for t in FLOATS}


def make_tokens(logits, masked, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    T, V = logits.shape[0], logits.shape[-1]
    t = torch.randint(V, (T,), generator=gen)
    t[torch.rand(T, generator=gen) < masked] = -1
    return t.to(dtype).cuda()


def check_forward(tgs, logits, tokens, temperature=1.0, top=0, entropy=True, ws=None):
    r = tgs.token_logprobs(logits, tokens, temperature=temperature, top=top, entropy=entropy, ws=ws)
    s = Softmax(logits, temperature)
    t = tokens.long().cpu()
    real = (t >= 0) & (t < logits.shape[-1])
    at = torch.where(real, t, 0)[..., None]
    lp, d = s.lp.gather(-1, at)[..., 0], s.d.gather(-1, at)[..., 0]
    assert_close(r.logprobs, torch.where(real, lp, 0.0), s.tol_lp(d[..., None], lp[..., None])[..., 0] * real, "logprobs")
    if entropy:
        want = torch.where(real & ~s.empty[..., 0], s.entropy, 0.0)
        assert_close(r.entropy, want, s.tol_entropy * real, "entropy")
    else:
        assert r.entropy is None
    if top:
        order = torch.argsort(logits.double().cpu(), dim=-1, descending=True, stable=True)[..., :top]
        assert r.top_indices.dtype == torch.int32
        assert torch.equal(r.top_indices.cpu().long(), torch.where(real[..., None], order, -1))
        lp, d = s.lp.gather(-1, order), s.d.gather(-1, order)
        assert_close(r.top_logprobs, torch.where(real[..., None], lp, 0.0), s.tol_lp(d, lp) * real[..., None], "top")
    else:
        assert r.top_indices is None and r.top_logprobs is None
    lse = r.stats[..., 0].double().cpu() / temperature + r.stats[..., 1].double().cpu()
    want = (s.m / temperature + s.log_s)[..., 0]
    assert_close(torch.where(real, lse, 0.0), torch.where(real, want, 0.0), s.tol_log_s[..., 0], "stats")
    return r


def check_backward(tgs, logits, tokens, r, temperature=1.0, use=(True, True), seed=3, out=None):
    gen = torch.Generator().manual_seed(seed)
    shape = tokens.shape
    g = torch.randn(shape, generator=gen).cuda() if use[0] else None
    ge = (0.3 * torch.randn(shape, generator=gen)).cuda() if use[1] else None
    s = Softmax(logits, temperature)
    t = tokens.long().cpu()
    real = ((t >= 0) & (t < logits.shape[-1]))[..., None] & ~s.empty
    hot = torch.zeros_like(s.p).scatter_(-1, t.clamp(min=0, max=logits.shape[-1] - 1)[..., None], 1.0)
    rel = s.relative()
    want, tol = torch.zeros_like(s.p), torch.zeros_like(s.p)
    if use[0]:
        a = g.double().cpu()[..., None]
        want = a * (hot - s.p)
        tol = a.abs() * (s.p * (rel + 2 * U) + 2 * U * hot)
    if use[1]:
        a, lp, h = ge.double().cpu()[..., None], torch.where(s.p > 0, s.lp, 0.0), s.entropy[..., None]
        want = want - a * s.p * (lp + h)
        off = s.tol_lp(s.d, s.lp) + U * s.size + s.tol_entropy[..., None] + U * (lp + h).abs()
        tol = tol + a.abs() * s.p * ((lp + h).abs() * (rel + 4 * U) + off)
        if use[0]:
            tol = tol + U * s.p * (g.double().cpu()[..., None].abs() + a.abs() * (lp + h).abs())
    want, tol = want / temperature, (tol / temperature + 4 * U * want.abs() / temperature)
    given = out
    out = tgs.token_logprobs_grad(logits, tokens, r.stats, g, r.entropy, ge, temperature, out=out)
    assert given is None or out is given
    assert out.dtype == logits.dtype
    # exponentials below fp32's normal numbers are flushed to 0
    assert_close(out, torch.where(real, want, 0.0), real * (tol + rounded(want, logits.dtype) + 2.0**-120), "grad")
    return out, g, ge


# ------------------------------------------------------------------- CPU --
def forward_call(lib, **kw):
    a = dict(z=0x1000000, zt=0, T=16, V=100, ld=100, t=0x2000000, tt=3, tau=1.0, lp=0x3000000, st=0x3100000, e=0x3200000,
             top=2, ti=0x3300000, tl=0x3400000, ws=0x4000000, wsn=1 << 20)
    a.update(kw)
    p = ctypes.c_void_p
    return lib.tgs_token_logprobs(p(a["z"]), a["zt"], a["T"], a["V"], a["ld"], p(a["t"]), a["tt"], a["tau"], p(a["lp"]),
                                  p(a["st"]), p(a["e"]), a["top"], p(a["ti"]), p(a["tl"]), p(a["ws"]), a["wsn"], None)


def grad_call(lib, **kw):
    a = dict(z=0x1000000, zt=0, T=16, V=100, ld=100, t=0x2000000, tt=3, tau=1.0, st=0x3100000, g=0x3000000, e=0x3200000,
             ge=0x3300000, out=0x5000000, lo=100, ws=0x4000000, wsn=1 << 20)
    a.update(kw)
    p = ctypes.c_void_p
    return lib.tgs_token_logprobs_grad(p(a["z"]), a["zt"], a["T"], a["V"], a["ld"], p(a["t"]), a["tt"], a["tau"],
                                       p(a["st"]), p(a["g"]), p(a["e"]), p(a["ge"]), p(a["out"]), a["lo"], p(a["ws"]),
                                       a["wsn"], None)


@pytest.fixture
def lib():
    import top_gradient_sparsification_amd as tgs
    return tgs.library()


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=2**31), dict(V=0), dict(V=2**31), dict(ld=99), dict(ld=2**31), dict(zt=3), dict(tt=0),
    dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")), dict(tau=1e-7), dict(z=None),
    dict(t=None), dict(st=None), dict(ws=None), dict(ws=0x4000010), dict(z=0x1000002), dict(t=0x2000002),
    dict(st=0x3100002), dict(t=0x2000004, tt=4),
])
def test_refusals_before_any_launch(lib, kw):
    assert forward_call(lib, **kw) == EINVAL, lib.tgs_last_error()
    assert b"token_logprobs:" in lib.tgs_last_error()
    assert grad_call(lib, **kw) == EINVAL, lib.tgs_last_error()
    assert b"token_logprobs_grad:" in lib.tgs_last_error()


def test_refusals_of_each(lib):
    for kw in (dict(top=-1), dict(top=65), dict(V=3, ld=3, top=4), dict(lp=None), dict(ti=None), dict(tl=None),
               dict(lp=0x1000100), dict(st=0x3000010), dict(e=0x3300000), dict(ti=0x2000000), dict(tl=0x4000100)):
        assert forward_call(lib, **kw) == EINVAL, kw
    for kw in (dict(g=None, ge=None), dict(e=None), dict(lo=99), dict(out=None), dict(out=0x1000100),
               dict(out=0x1000000, lo=101), dict(out=0x3000000), dict(out=0x2000000), dict(out=0x4000000)):
        assert grad_call(lib, **kw) == EINVAL, kw
    need = lib.tgs_token_logprobs_workspace_bytes(16, 100_000, 0, 2)
    assert need > 32768
    assert forward_call(lib, V=100_000, ld=100_000, lp=0x3F00000, z=0x10000000, wsn=need - 1) == EWORKSPACE
    assert grad_call(lib, wsn=100) == EWORKSPACE
    for bad in ((-1, 10, 0, 0), (1, 0, 0, 0), (1, 10, 3, 0), (1, 10, 0, 11), (1, 1000, 0, 65), (1, 10, 0, -1), (2**31, 8, 0, 0)):
        assert lib.tgs_token_logprobs_workspace_bytes(*bad) == 0, bad


def test_rows_that_the_binding_takes_and_refuses():
    import top_gradient_sparsification_amd as tgs

    class Gpu(torch.Tensor):
        is_cuda = True

    def rows(t):
        return tgs._spaced_rows(t.as_subclass(Gpu), "logits", FLOATS)

    x = torch.zeros(4, 6, 10)
    assert rows(x) == (24, 10, 10) and rows(x[..., :7]) == (24, 7, 10) and rows(x[:, 2:3, :7]) == (4, 7, 60)
    assert rows(x[0, 0]) == (1, 10, 10) and rows(x[0, 0, 2:5]) == (1, 3, 3) and rows(x[..., :1]) == (24, 1, 10)
    assert rows(x[:0]) == (0, 10, 10) and rows(x[..., 3:3])[:2] == (0, 0) and rows(x[1:3, :, 2:9]) == (12, 7, 10)
    for bad, error in ((x[:, :5, :7], "fixed number"), (x.transpose(1, 2), "contiguous along"), (x[:, ::2, ::2], "contiguous along"),
                       (x[:1, :1].expand(4, 1, 10)[:, 0], "overlap"), (x.transpose(0, 1)[..., :7], "fixed number")):
        with pytest.raises(ValueError, match=error):
            rows(bad)
    with pytest.raises(TypeError, match="GPU tensor"):
        tgs.token_logprobs(x, torch.zeros(4, 6, dtype=torch.int64))
    with pytest.raises(TypeError, match="must be one of"):
        tgs.token_logprobs(x.long(), torch.zeros(4, 6, dtype=torch.int64))


def test_the_definitions_agree_with_differences():
    gen = torch.Generator().manual_seed(2)
    z = 2 * torch.randn(3, 6, generator=gen, dtype=torch.float64)
    z[1, 2] = -math.inf
    s = Softmax(z, 0.7)
    assert (s.p.sum(-1) - 1).abs().max() < 1e-12 and s.p[1, 2] == 0
    h = 1e-6
    for j in (0, 4):
        step = torch.zeros_like(z)
        step[:, j] = h
        up, down = Softmax(z + step, 0.7), Softmax(z - step, 0.7)
        d_lp = (up.lp[:, 0] - down.lp[:, 0]) / (2 * h)
        assert ((float(j == 0) - s.p[:, j]) / 0.7 - d_lp).abs().max() < 1e-7
        d_h = (up.entropy - down.entropy) / (2 * h)
        assert (-s.p[:, j] * (s.lp[:, j] + s.entropy) / 0.7 - d_h).abs().max() < 1e-7
    wrong = s.entropy + 1e-4
    with pytest.raises(AssertionError):
        assert_close(wrong, s.entropy, s.tol_entropy)
    assert (s.tol_log_s < 1e-5).all() and (s.tol_entropy < 2e-5).all()


# ------------------------------------------------------------------- GPU --
VOCABULARIES = [1, 2, 3, 7, 8, 63, 64, 65, 511, 512, 513, 1000, 2047, 2048, 4097, 8191, 10_000, 50_001, 128_000]


@pytest.mark.gpu
@pytest.mark.parametrize("V", VOCABULARIES)
def test_vocabularies(tgs_gpu, V):
    for dtype, T, ids, top, tau in ((torch.float32, 3, torch.int32, 5, 1.0), (torch.bfloat16, 40, torch.int64, 64, 0.7),
                                    (torch.float16, 1, torch.int64, 20, 2.0)):
        logits = scores(T, V, dtype, V)
        tokens = make_tokens(logits, 0.2 if T > 3 else 0.0, ids, V)
        r = check_forward(tgs_gpu, logits, tokens, tau, min(top, V))
        check_backward(tgs_gpu, logits, tokens, r, tau)


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(2500, 1000), (1100, 5001), (300, 20_000), (4000, 3), (20_000, 130), (2100, 513)])
def test_many_rows(tgs_gpu, T, V):
    for dtype in FLOATS:
        logits = scores(T, V, dtype, T)
        tokens = make_tokens(logits, 0.3, torch.int64, T)
        r = check_forward(tgs_gpu, logits, tokens, 1.0, min(V, 7))
        check_backward(tgs_gpu, logits, tokens, r)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("T,V", [(5, 50_001), (1500, 1001), (9, 200)])
def test_each_output_alone(tgs_gpu, dtype, T, V):
    logits, tokens = scores(T, V, dtype, 1), None
    tokens = make_tokens(logits, 0.1, torch.int32, 1)
    full = check_forward(tgs_gpu, logits, tokens, 1.3, 9, True)
    for top in (0, 1, 9):
        for entropy in (False, True):
            r = check_forward(tgs_gpu, logits, tokens, 1.3, top, entropy)
            assert torch.equal(r.logprobs, full.logprobs) and torch.equal(r.stats, full.stats)
    for use in ((True, False), (False, True)):
        check_backward(tgs_gpu, logits, tokens, full, 1.3, use)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("T,V,pad", [(7, 1001, 23), (1300, 777, 1), (3, 50_001, 47), (40, 100, 3)])
def test_rows_apart_and_in_place(tgs_gpu, dtype, T, V, pad):
    """Padded rows, read and written between NaNs that stay where they are."""
    logits = scores(T, V, dtype, 5, pad=pad)
    rows = logits.as_strided((T, V + pad), (V + pad, 1))
    assert torch.isnan(rows[:, V:]).all()
    tokens = make_tokens(logits, 0.1, torch.int64, 5)
    r = check_forward(tgs_gpu, logits, tokens, 1.0, 5)
    out, g, ge = check_backward(tgs_gpu, logits, tokens, r)
    wide = torch.full((T, V + pad + 2), 5.0, dtype=dtype, device="cuda")
    check_backward(tgs_gpu, logits, tokens, r, out=wide[:, 2:V + 2])
    assert torch.equal(wide[:, 2:V + 2], out) and (wide[:, :2] == 5).all() and (wide[:, V + 2:] == 5).all()
    version = logits._version
    tgs_gpu.token_logprobs_grad(logits, tokens, r.stats, g, r.entropy, ge, out=logits)
    assert torch.equal(logits, out) and torch.isnan(rows[:, V:]).all() and logits._version > version


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(6, 40), (6, 700), (6, 9000), (6, 70_001), (1030, 9000)])
@pytest.mark.parametrize("dtype", FLOATS)
def test_masks_of_minus_infinity_and_the_lowest_value(tgs_gpu, dtype, T, V):
    logits = scores(T, V, dtype, 2).clone()
    logits[0] = -math.inf                       # nothing left
    logits[1] = LOWEST[dtype]                   # a score like any other: uniform
    logits[2, 1:] = -math.inf                   # one score left
    logits[3, :V // 2] = LOWEST[dtype]
    logits[4, V // 3:] = -math.inf
    logits[5, ::2] = -math.inf
    tokens = make_tokens(logits, 0.0, torch.int64, 2)
    tokens[2] = 0
    tokens[4] = V - 1                           # probability 0
    top = min(V, 30)
    for tau in (1.0, 0.5):
        r = check_forward(tgs_gpu, logits, tokens, tau, top)
        check_backward(tgs_gpu, logits, tokens, r, tau)
    assert r.logprobs[0] == -math.inf and r.entropy[0] == 0 and r.top_indices[0].tolist() == list(range(top))
    assert (r.top_logprobs[0] == -math.inf).all()
    assert r.logprobs[2] == 0 and r.entropy[2] == 0 and r.logprobs[4] == -math.inf
    assert r.top_indices[2, 0] == 0 and r.top_indices[2, 1:].tolist() == list(range(1, top))


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(5, 30), (5, 600), (5, 30_000), (1030, 3000)])
def test_nan_and_infinity_stay_in_their_rows(tgs_gpu, T, V):
    logits = scores(T, V, torch.float32, 4)
    tokens = make_tokens(logits, 0.0, torch.int64, 4)
    want = tgs_gpu.token_logprobs(logits, tokens, top=10, entropy=True)
    bad = logits.clone()
    bad[1, V // 2] = math.nan
    bad[3, V - 1] = math.inf
    bad[3, 4] = -math.nan
    got = tgs_gpu.token_logprobs(bad, tokens, top=10, entropy=True)
    keep = torch.tensor([0, 2, 4], device="cuda")
    for a, b in zip(got, want):
        assert torch.equal(a[keep], b[keep])
    for row in (1, 3):
        assert torch.isnan(got.logprobs[row]) and torch.isnan(got.entropy[row]) and torch.isnan(got.top_logprobs[row]).all()
    # a NaN ranks above all, infinity next
    best = logits[1].clone()
    best[V // 2] = math.inf
    order = torch.sort(best, descending=True, stable=True).indices[:10]
    assert got.top_indices[1].tolist() == order.tolist()
    assert got.top_indices[3, :2].tolist() == [4, V - 1]
    grad = tgs_gpu.token_logprobs_grad(bad, tokens, got.stats, want.logprobs, got.entropy, want.entropy)
    ok = tgs_gpu.token_logprobs_grad(logits, tokens, want.stats, want.logprobs, want.entropy, want.entropy)
    assert torch.equal(grad[keep], ok[keep]) and torch.isnan(grad[1]).all() and torch.isnan(grad[3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(3, 50), (3, 5000), (3, 128_000), (1100, 700), (1100, 6000)])
def test_ties_go_to_the_lower_index(tgs_gpu, T, V):
    gen = torch.Generator().manual_seed(1)
    logits = torch.randint(-3, 4, (T, V), generator=gen).to(torch.bfloat16).cuda()
    logits[0] = 0.0
    logits[0, 1::3] = -0.0                      # equal to +0
    logits[1] = 2.5
    tokens = make_tokens(logits, 0.0, torch.int32, 1)
    r = check_forward(tgs_gpu, logits, tokens, 1.0, min(V, 64))
    assert r.top_indices[0].tolist() == r.top_indices[1].tolist() == list(range(min(V, 64)))


@pytest.mark.gpu
def test_orders_made_against_the_selection(tgs_gpu):
    """Largest scores that a few threads hold together, in rows that one
    workgroup reads and in rows of many slices: more of them than a list takes."""
    V = 131_072
    gen = torch.Generator().manual_seed(6)
    for dtype in (torch.bfloat16, torch.float32):
        E = 8 if dtype == torch.bfloat16 else 4
        z = torch.randn(1100, V, generator=gen).to(dtype)
        owner = (torch.arange(V) // E) % 256
        z[0, owner < 16] += 20
        z[1] = torch.arange(V).float() / V * 16
        z[2] = -z[1]
        z[3, owner == 3] += 30
        logits = z.cuda()
        tokens = torch.full((1100,), -1, device="cuda")
        tokens[:4] = torch.tensor([5, 77, 0, V - 1])
        r = tgs_gpu.token_logprobs(logits, tokens, top=64)
        order = torch.argsort(z[:4].double(), dim=-1, descending=True, stable=True)[:, :64]
        assert torch.equal(r.top_indices[:4].cpu().long(), order)
        assert (r.top_indices[4:] == -1).all()
    # every slice of a single row holds the same 64 scores, then 64 of one slice alone
    row = torch.randn(1, V, generator=gen)
    for s in range(64):
        row[0, s * 2048 + 64 * (s % 7):][:64] = 1000 - torch.arange(64).float()
    check_forward(tgs_gpu, row.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"), 1.0, 64)
    row[0, 90_000:90_064] += 5000
    check_forward(tgs_gpu, row.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"), 1.0, 64)


@pytest.mark.gpu
def test_rising_and_falling_scores(tgs_gpu):
    """A reference score that has to be replaced many times, and one that never is."""
    V = 40_000
    for T in (2, 1100):
        z = torch.zeros(T, V)
        z[0] = torch.linspace(-3000, 3000, V)
        z[1] = torch.linspace(3000, -3000, V)
        for dtype in (torch.float32, torch.bfloat16):
            logits = z.to(dtype).cuda()
            tokens = torch.full((T,), -1, device="cuda")
            tokens[0], tokens[1] = V - 3, 2
            r = check_forward(tgs_gpu, logits, tokens, 1.0, 5)
            check_backward(tgs_gpu, logits, tokens, r)


@pytest.mark.gpu
def test_bad_tokens_are_reported_and_masked(tgs_gpu):
    for T, V in ((4, 100), (4, 90_000), (1200, 700)):
        logits = scores(T, V, torch.float32, 8)
        tokens = make_tokens(logits, 0.0, torch.int64, 8)
        tokens[2] = V
        tokens[1] = 2**40
        tokens[0] = -2**40
        ws = torch.zeros(tgs_gpu.token_logprobs_workspace_bytes(T, V, torch.float32, 3), dtype=torch.uint8, device="cuda")
        r = check_forward(tgs_gpu, logits, tokens, 1.0, 3, ws=ws)
        with pytest.raises(ValueError, match="index"):
            tgs_gpu.check_device_error(ws)
        tgs_gpu.check_device_error(ws)
        check_backward(tgs_gpu, logits, tokens, r)
        tgs_gpu.token_logprobs_grad(logits, tokens, r.stats, r.logprobs, ws=ws)
        with pytest.raises(ValueError, match="index"):
            tgs_gpu.check_device_error(ws)
        assert not ws[4:32768].any()


@pytest.mark.gpu
def test_offsets_past_32_bits(tgs_gpu):
    """2.2e9 scores: the last rows against a call on them alone."""
    V, T = 50_001, 44_000
    logits = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    logits[-1100:] = scores(1100, V, torch.bfloat16, 9)
    tokens = torch.full((T,), -1, device="cuda")
    tokens[-1100:] = make_tokens(logits[-1100:], 0.1, torch.int64, 9)
    tokens[0] = 7
    r = tgs_gpu.token_logprobs(logits, tokens, top=3, entropy=True)
    part = tgs_gpu.token_logprobs(logits[-1100:], tokens[-1100:], top=3, entropy=True)
    for a, b in zip(r, part):
        assert torch.equal(a[-1100:], b)
    assert abs(r.logprobs[0].item() + math.log(V)) < 1e-5
    want = tgs_gpu.token_logprobs_grad(logits[-1100:], tokens[-1100:], part.stats, part.logprobs)
    tgs_gpu.token_logprobs_grad(logits, tokens, r.stats, r.logprobs, out=logits)
    assert torch.equal(logits[-1100:], want) and not logits[1:-1100].any()


@pytest.mark.gpu
def test_more_rows_than_a_launch_takes(tgs_gpu):
    """2^26 workgroups of a wave are a launch: the rows behind them."""
    T, V = 2**26 + 1000, 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(T, V, device="cuda", generator=gen).to(torch.bfloat16)
    tokens = torch.randint(-1, V, (T,), device="cuda", generator=gen, dtype=torch.int32)
    r = tgs_gpu.token_logprobs(logits, tokens, entropy=True)
    g = tgs_gpu.token_logprobs_grad(logits, tokens, r.stats, r.logprobs)
    tail = slice(T - 2000, T)
    part = check_forward(tgs_gpu, logits[tail], tokens[tail])
    for a, b in zip((r.logprobs, r.entropy, r.stats), (part.logprobs, part.entropy, part.stats)):
        assert torch.equal(a[tail], b)
    assert torch.equal(g[tail], tgs_gpu.token_logprobs_grad(logits[tail], tokens[tail], part.stats, part.logprobs))


@pytest.mark.gpu
def test_gradients_flow(tgs_gpu):
    z = scores(24, 300, torch.float32, 3).reshape(4, 6, 300).clone().requires_grad_()
    tokens = make_tokens(z.detach().reshape(24, 300), 0.2, torch.int64, 3).view(4, 6)
    r = tgs_gpu.token_logprobs(z, tokens, temperature=0.8, top=4, entropy=True)
    assert r.logprobs.shape == (4, 6) and r.top_indices.shape == (4, 6, 4)
    assert r.logprobs.requires_grad and r.entropy.requires_grad and not r.top_logprobs.requires_grad
    weights = torch.linspace(-1, 1, 24, device="cuda").view(4, 6)
    (got,) = torch.autograd.grad((weights * r.logprobs).sum() + 0.1 * r.entropy.sum(), z)
    plain = tgs_gpu.token_logprobs(z.detach(), tokens, temperature=0.8, entropy=True)
    want = tgs_gpu.token_logprobs_grad(z.detach(), tokens, plain.stats, weights, plain.entropy,
                                       torch.full_like(weights, 0.1), 0.8)
    assert torch.equal(got, want)
    (got,) = torch.autograd.grad(tgs_gpu.token_logprobs(z, tokens).logprobs.sum(), z)
    assert torch.isfinite(got).all() and (got[tokens < 0] == 0).all()
    (got,) = torch.autograd.grad(tgs_gpu.token_logprobs(z, tokens, entropy=True).entropy.sum(), z)
    # the directional derivative in 64 bits
    v = torch.randn(z.shape, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    h = 1e-6
    zd = z.detach().double().cpu()
    real = (tokens >= 0).cpu()
    up, down = (Softmax(zd + s * h * v, 1.0).entropy[real].sum() for s in (1, -1))
    want = (up - down) / (2 * h)
    assert abs((got.double().cpu() * v).sum() - want) < 1e-4 * abs(want) + 1e-4
    back = tgs_gpu.token_logprobs_grad(z, tokens, plain.stats, weights, temperature=0.8)
    with pytest.raises(NotImplementedError, match="token_logprobs_grad has no gradient"):
        back.sum().backward()
    with pytest.raises(RuntimeError, match="out="):
        tgs_gpu.token_logprobs_grad(z, tokens, plain.stats, weights, out=torch.empty_like(z))


@pytest.mark.gpu
def test_shapes_and_binding_refusals(tgs_gpu):
    z = scores(6, 40, torch.float32, 1)
    t = make_tokens(z, 0.0, torch.int64, 1)
    one = tgs_gpu.token_logprobs(z[2], t[2], top=2, entropy=True)
    assert one.logprobs.shape == () and one.top_indices.shape == (2,) and one.stats.shape == (2,)
    none = tgs_gpu.token_logprobs(z[:0], t[:0], top=2, entropy=True)
    assert none.logprobs.shape == (0,) and none.top_indices.shape == (0, 2)
    assert tgs_gpu.token_logprobs_grad(z[:0], t[:0], none.stats, none.logprobs).shape == (0, 40)
    f = torch.zeros(6, device="cuda")
    st = torch.zeros(6, 2, device="cuda")
    for call, error in ((lambda: tgs_gpu.token_logprobs(z, t[:5]), "tokens must have shape"),
                        (lambda: tgs_gpu.token_logprobs(z, t.float()), "tokens must be one of"),
                        (lambda: tgs_gpu.token_logprobs(z, t, top=65), "top=65"),
                        (lambda: tgs_gpu.token_logprobs(z, t, top=41), "top=41"),
                        (lambda: tgs_gpu.token_logprobs(z, t, top=-1), "top=-1"),
                        (lambda: tgs_gpu.token_logprobs(z, t, temperature=0.0), "temperature"),
                        (lambda: tgs_gpu.token_logprobs(z[:, :0], t), "invalid sizes"),
                        (lambda: tgs_gpu.token_logprobs(z.T, t), "contiguous along"),
                        (lambda: tgs_gpu.token_logprobs(z, t, ws=torch.zeros(64, dtype=torch.uint8)), "ws is on cpu"),
                        (lambda: tgs_gpu.token_logprobs_grad(z, t, st), "must be given"),
                        (lambda: tgs_gpu.token_logprobs_grad(z, t, st, grad_entropy=f), "needs entropy"),
                        (lambda: tgs_gpu.token_logprobs_grad(z, t, st[:5], f), "stats must have shape"),
                        (lambda: tgs_gpu.token_logprobs_grad(z, t, st, f.half()), "grad_logprobs must be one of"),
                        (lambda: tgs_gpu.token_logprobs_grad(z, t, st, f, out=z[:5]), "out must have shape"),
                        (lambda: tgs_gpu.token_logprobs_grad(z, t, st, f, out=z.half()), "out must be one of"),
                        (lambda: tgs_gpu.token_logprobs_grad(z, t, st, f, ws=torch.zeros(64, dtype=torch.uint8)), "ws is on cpu")):
        with pytest.raises((ValueError, TypeError), match=error):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(6, 40), (6, 700), (6, 9000), (6, 70_001), (1030, 9000)])
@pytest.mark.parametrize("dtype", FLOATS)
def test_rows_of_nan_alone(tgs_gpu, dtype, T, V):
    """Such a row's gradient is NaN as its loss is, and not the zeros of a row of -inf; by every route."""
    logits = scores(T, V, dtype, 6)
    tokens = make_tokens(logits, 0.0, torch.int64, 6)
    top = min(V, 20)
    g = torch.randn(T, generator=torch.Generator().manual_seed(3)).cuda()
    want = tgs_gpu.token_logprobs(logits, tokens, top=top, entropy=True)
    bad = logits.clone()
    bad[1] = math.nan
    bad[2], bad[2, V // 2] = -math.inf, math.nan
    bad[4] = -math.inf
    r = tgs_gpu.token_logprobs(bad, tokens, top=top, entropy=True)
    for x in (r.logprobs, r.entropy, r.top_logprobs):
        assert torch.isnan(x[1:3]).all()
    assert r.top_indices[1].tolist() == list(range(top))
    assert r.top_indices[2].tolist() == [V // 2] + [i for i in range(top) if i != V // 2][:top - 1]
    keep = torch.tensor([0, 3] + list(range(5, T)), device="cuda")
    for ge in (None, 0.1 * g):
        grad = tgs_gpu.token_logprobs_grad(bad, tokens, r.stats, g, r.entropy, ge)
        ok = tgs_gpu.token_logprobs_grad(logits, tokens, want.stats, g, want.entropy, ge)
        assert torch.isnan(grad[1:3]).all() and (grad[4] == 0).all() and torch.equal(grad[keep], ok[keep])
    leaf = bad.clone().requires_grad_()
    (-tgs_gpu.token_logprobs(leaf, tokens).logprobs).sum().backward()
    assert torch.isnan(leaf.grad[1:3]).all() and (leaf.grad[4] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(3, 50), (3, 30_000), (1030, 9000)])
def test_scores_further_apart_than_the_type_reaches(tgs_gpu, T, V):
    """x - m is no fp32 number, (x - m) / temperature is one."""
    for dtype in (torch.float32, torch.bfloat16):
        logits = scores(T, V, dtype, 3).clone()
        logits[0, 7], logits[0, 9] = LOWEST[dtype], -LOWEST[dtype]
        logits[1, 1], logits[1, 2:] = -LOWEST[dtype], LOWEST[dtype]
        tokens = make_tokens(logits, 0.0, torch.int32, 3)
        tokens[0], tokens[1] = 7, 5
        for tau in (2.5, 1e6):
            r = check_forward(tgs_gpu, logits, tokens, tau, min(V, 10))
            check_backward(tgs_gpu, logits, tokens, r, tau)
            assert torch.isfinite(r.logprobs[:2]).all() and (r.logprobs[:2] < -1e32).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("V", [65_537, 65_539, 65_543, 65_545])
def test_last_slices_of_a_few_scores(tgs_gpu, dtype, V):
    """Rows in slices of 4,096 or 8,192 scores, of which the last holds less than a vector or little more."""
    logits = scores(5, V, dtype, 7, pad=3).clone()
    logits[1, 65_536:] = 30.0
    logits[2, :65_536] = -math.inf
    logits[3, 65_536:] = -math.inf
    tokens = make_tokens(logits, 0.0, torch.int64, 7)
    tokens[1:4] = V - 1
    for top in (1, 12, 64):
        r = check_forward(tgs_gpu, logits, tokens, 0.8, top)
    check_backward(tgs_gpu, logits, tokens, r, 0.8)
