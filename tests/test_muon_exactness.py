"""How exact the Newton-Schulz products are, type by type.

r is the 2-norm error of the exact result rounded to the type, taken from the
oracle itself; a result whose error before the rounding is d r is off by
sqrt(1 + d^2) r, and r varies by some per cent over the few entries of a small
matrix.
* fp16 and fp32 results: operands of 22 bits, 2^-18 in all before the rounding.
* bf16 results: single fp16 operands, diagonals apart, d <= 1/2 for matrices like
  gradients: 1.12 r, here 1.15 r.  Rounding X, A and P whole to fp16 gives 1.24 r
  and more.  Matrices of low rank: those here, of 128 and more, up to 2.8e-3
  before the rounding (2 r); whole operands give 14 r and more.  With a shorter
  side of 33 to 64 the update takes X's low parts too: those here d <= 0.65, 1.19
  r, allowed 1.25 r; without them 2 r to 10 r.  Up to 32 bf16 is as exact as fp16.
"""
import math

import numpy as np
import pytest
import torch

from test_muon import QUINTIC, distance, exact, matrices

SHAPES = [(64, 64), (40, 700), (128, 128), (96, 160), (300, 200), (530, 600)]


def low_rank(m, n, rank, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, rank)) @ rng.standard_normal((rank, n)) / math.sqrt(m * n)
    return torch.from_numpy(x.astype(np.float32))


def rounding(want, dtype):
    return distance(want.to(dtype), want)


def bound(want, dtype, factor=1.15):
    return factor * rounding(want, dtype) if dtype == torch.bfloat16 else 1.05 * rounding(want, dtype) + 2.0**-18


def rounded(v, scale):
    return (v * scale).half().float() / scale


def half_products(x, apart, low=False, steps=5):
    """The iteration with fp16 operands: diagonals of A and P and X held apart in fp32, or all rounded whole;
    `low`: X's low parts in the update too."""
    a, b, c = QUINTIC
    y = (x.double() / (x.double().norm() + 1e-7)).float()
    y = y.T.contiguous() if y.shape[0] > y.shape[1] else y
    for _ in range(steps):
        h = rounded(y, 8192.0)
        g = h @ h.T
        d = g.diagonal().clone() if apart else torch.zeros(len(g))
        e = rounded(g - d.diag(), 8192.0)
        square = e @ e
        p = (c * (d[:, None] + d[None, :]) + b) * e + c * square
        dp = c * (d * d + square.diagonal()) + b * d if apart else torch.zeros(len(g))
        p = rounded(p - p.diagonal().diag() if apart else p, 2048.0)
        y = (a + dp)[:, None] * (y if apart else h) + p @ (y if low else h)
    return y.T if x.shape[0] > x.shape[1] else y


@pytest.mark.parametrize("shape", [(64, 64), (128, 128), (300, 200)])
@pytest.mark.parametrize("noise", [0.1, 0.3, 1.0])
def test_the_bounds_tell_the_schemes_apart(shape, noise):
    x = matrices(shape, seed=sum(shape), noise=noise)
    for dtype in (torch.bfloat16, torch.float16):
        want = exact(x.to(dtype))
        apart, whole = (half_products(x.to(dtype), s).to(dtype) for s in (True, False))
        assert distance(whole, want) > bound(want, dtype)
        # single products with the diagonals apart are enough for bf16, not for fp16
        assert (distance(apart, want) <= bound(want, dtype)) == (dtype == torch.bfloat16)
    z = low_rank(*shape, 8, 3).bfloat16()
    want = exact(z)
    single, low, whole = (distance(half_products(z, *s).bfloat16(), want) for s in ((True,), (True, True), (False,)))
    r = rounding(want, torch.bfloat16)
    assert low <= 1.15 * r < single and 2 * r < whole and (single <= 2 * r) == (min(shape) > 64)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("noise", [0.1, 0.3, 1.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rounding_is_what_16_bit_results_lose(tgs_gpu, shape, noise, dtype):
    for s in (shape, shape[::-1]):
        x = matrices(s, seed=sum(s), noise=noise, dtype=dtype)
        want = exact(x)
        assert distance(tgs_gpu.newton_schulz(x.cuda()), want) <= bound(want, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(64, 64), (128, 128), (300, 400)])
@pytest.mark.parametrize("rank", [2, 8, 32])
def test_low_rank_in_bf16(tgs_gpu, shape, rank):
    x = low_rank(*shape, rank, 3).bfloat16()
    want = exact(x)
    assert distance(tgs_gpu.newton_schulz(x.cuda()), want) <= bound(want, torch.bfloat16, 2.0)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(64, 64), (33, 50), (64, 700), (700, 40), (2000, 64), (20, 1500)])
@pytest.mark.parametrize("rank", [1, 4, 16])
def test_low_rank_in_bf16_of_a_short_side(tgs_gpu, shape, rank):
    x = low_rank(*shape, rank, 3).bfloat16()
    want = exact(x)
    assert distance(tgs_gpu.newton_schulz(x.cuda()), want) <= bound(want, torch.bfloat16, 1.25)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 5), (5, 1), (2, 7), (8, 8), (16, 40), (32, 300), (1500, 20), (31, 1025), (64, 3, 9)])
@pytest.mark.parametrize("rank", [1, 2, None])
def test_a_side_of_up_to_32_loses_nothing_but_the_rounding(tgs_gpu, shape, rank):
    *b, m, n = shape
    for seed in range(8):
        x = torch.stack([matrices((m, n), seed + 9 * i, 1.0) if rank is None else low_rank(m, n, min(rank, m, n), seed + 9 * i)
                         for i in range(b[0] if b else 1)]).bfloat16()
        want = exact(x)
        assert distance(tgs_gpu.newton_schulz(x.cuda()), want) <= 1.05 * rounding(want, torch.bfloat16) + 2.0**-18


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(20, 30), (64, 512), (500, 40), (64, 8192), (3, 3000, 30), (70, 90), (300, 200)])
@pytest.mark.parametrize("ratio", [1e-8, 1e-12, 1e-16])
def test_a_norm_far_below_eps(tgs_gpu, shape, ratio):
    """X stays tiny and every step multiplies it by the first coefficient, near enough."""
    x = matrices(shape, seed=sum(shape)) * (1e-3 * ratio)
    got = tgs_gpu.newton_schulz(x.cuda(), eps=1e-3)
    assert distance(got, exact(x, eps=1e-3)) <= 2.0**-18
