"""The embedding gradient's two routes, few places in one launch and many by a
sort, held to the same results."""
import numpy as np
import pytest
import torch

from test_embedding import EINVAL, FLOATS, U, abi, assert_grad, grad_call, lookup_call, make_tokens

ONE_LAUNCH = 32768  # bytes of workspace: the header alone


def needs(tgs, T, V, D, grad_dtype, out_dtype):
    return tgs.embedding_grad_workspace_bytes(T, V, D, grad_dtype, out_dtype)


def test_more_threads_than_a_launch_may_have_are_refused():
    """2^24 workgroups of 256 make 2^32 threads: refused before anything is enqueued."""
    lib, far = abi(), dict(tokens=1 << 44, out=3 << 44, ws=5 << 44, wsn=1 << 50)
    assert lookup_call(lib, table=2 << 44, T=2**31 - 1, D=64, **far) == EINVAL
    assert b"too large" in lib.tgs_last_error()
    assert grad_call(lib, grad=2 << 44, T=2**31 - 1, D=1024, **far) == EINVAL
    assert b"too large" in lib.tgs_last_error()


@pytest.mark.gpu
def test_more_sums_to_join_than_workgroups(tgs_gpu):
    """Over 2^30 places of one column: the kernel that joins partial sums has more of them than a launch has
    workgroups of 256.  All sums are counts below 2^24, so exact."""
    T, V, part = (1 << 30) + 12_345, 1 << 20, 1 << 26
    gen = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32, generator=gen)
    want = torch.zeros(V, dtype=torch.int64, device="cuda")
    for t in tokens.split(part):
        want += torch.bincount(t, minlength=V)
    grad = torch.ones(T, 1, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(needs(tgs_gpu, T, V, 1, torch.bfloat16, torch.float32), dtype=torch.uint8, device="cuda")
    got = tgs_gpu.embedding_grad(tokens, grad, V, ws=ws)
    assert torch.equal(got[:, 0].long(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("T,one", [(300, True), (5_000, False)])
@pytest.mark.parametrize("out_dtype", FLOATS)
def test_rows_without_places_are_plus_zero(tgs_gpu, T, one, out_dtype):
    V, D = 700, 33
    assert (needs(tgs_gpu, T, V, D, torch.float32, out_dtype) == ONE_LAUNCH) == one
    rng = np.random.default_rng(T)
    tokens = make_tokens(T, V, 0.1, torch.int64, rng)
    grad = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32))
    got = tgs_gpu.embedding_grad(tokens.cuda(), grad.cuda(), V, scale=-0.37, out_dtype=out_dtype).cpu()
    assert_grad(got, tokens, grad, V, -0.37)
    empty = torch.ones(V, dtype=torch.bool)
    empty[tokens[tokens >= 0]] = False
    assert empty.any() and not torch.signbit(got[empty]).any()
    # masked places only, and no places
    for t in (torch.full((T,), -1), torch.empty(0, dtype=torch.int64)):
        none = tgs_gpu.embedding_grad(t.cuda(), grad[:t.numel()].cuda(), V, scale=-2.0, out_dtype=out_dtype)
        assert not none.any() and not torch.signbit(none).any()


@pytest.mark.gpu
@pytest.mark.parametrize("grad_dtype", FLOATS)
@pytest.mark.parametrize("out_dtype", FLOATS)
@pytest.mark.parametrize("D", [1, 5, 130, 264])
def test_sorted_types_and_widths(tgs_gpu, grad_dtype, out_dtype, D):
    """Every type, written and accumulated: masked places, tokens within a chunk and over many."""
    T, V = 5_003, 311
    assert needs(tgs_gpu, T, V, D, grad_dtype, out_dtype) > ONE_LAUNCH
    rng = np.random.default_rng(D)
    for ids, scale, acc in ((torch.int32, -0.37, False), (torch.int64, 1.0, True)):
        tokens = make_tokens(T, V, 0.1, ids, rng)
        grad = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(grad_dtype)
        base = torch.from_numpy(rng.standard_normal((V, D)).astype(np.float32)).to(out_dtype) if acc else None
        out = base.cuda() if acc else None
        got = tgs_gpu.embedding_grad(tokens.cuda(), grad.cuda(), V, scale=scale, out_dtype=out_dtype, out=out,
                                     accumulate=acc)
        assert got.dtype == out_dtype
        assert_grad(got, tokens, grad, V, scale, base)


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,D,one", [(1025, 128_000, 130, True), (1_100, 128_000, 130, False), (2_048, 1_000, 33, True),
                                       (2_049, 1_000, 33, False), (1, 300_000, 3, False), (700, 64, 4_099, True)])
@pytest.mark.parametrize("out_dtype", FLOATS)
def test_either_side_of_the_rule(tgs_gpu, T, V, D, one, out_dtype):
    assert (needs(tgs_gpu, T, V, D, torch.bfloat16, out_dtype) == ONE_LAUNCH) == one
    rng = np.random.default_rng(T)
    tokens = make_tokens(T, V, 0.05, torch.int64, rng)
    grad = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).bfloat16()
    got = tgs_gpu.embedding_grad(tokens.cuda(), grad.cuda(), V, scale=0.5, out_dtype=out_dtype)
    assert_grad(got, tokens, grad, V, 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T,D", [(70_001, 2_003), (70_001, 2_048), (262_147, 257), (262_147, 256)])
def test_eight_fp16_gradients_a_lane(tgs_gpu, T, D, accumulate):
    """Sizes that take eight 16-bit gradients a lane into fp32 rows, and one that does not; the oracle runs on the GPU."""
    V = 3_000
    gen = torch.Generator(device="cuda").manual_seed(D)
    tokens = torch.randint(-100, V, (T,), device="cuda", generator=gen)
    grad = torch.randn(T, D, device="cuda", generator=gen).half()
    base = torch.randn(V, D, device="cuda", generator=gen) if accumulate else torch.zeros(V, D, device="cuda")
    real = tokens >= 0
    total, size = (torch.zeros(V, D, dtype=torch.float64, device="cuda") for _ in range(2))
    total.index_add_(0, tokens[real], grad[real].double())
    size.index_add_(0, tokens[real], grad[real].double().abs())
    count = torch.bincount(tokens[real], minlength=V).double()[:, None]
    got = tgs_gpu.embedding_grad(tokens, grad, V, out=base.clone(), accumulate=accumulate)
    want = total + base.double()
    assert ((got.double() - want).abs() <= size * (count + 8) * U * 1.01 + want.abs() * 2 * U).all()
