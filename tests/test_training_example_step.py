"""The training example's Muon steps against the definition."""
import math

import pytest
import torch

from test_gpu_training_example import example  # noqa: F401 - a fixture
from test_muon import U, exact


@pytest.mark.gpu
def test_matrices_move_by_out_over_in(example):  # noqa: F811
    """The update is lr sqrt(max(1, out / in)) times the orthogonalised momentum, however a matrix is stored."""
    model = example.Model(vocab=300, dim=72, density=0.1)
    tokens, targets = next(example.batches(300, 7, 19))
    before = [w.detach().double().cpu() for w, _ in model.matrices]
    model.step(tokens, targets, lr_table=1.0, lr_matrices=0.05)
    assert [tuple(w.shape) for w in before] == [(72, 72), (72, 300)]  # [in, out]
    for (w, _), old, (n_in, n_out) in zip(model.matrices, before, ((72, 72), (72, 300))):
        g = w.grad.double().cpu()
        want = 0.05 * math.sqrt(max(1.0, n_out / n_in)) * exact(g + 0.95 * g)
        off = (old - w.detach().double().cpu() - want).norm()
        assert off <= want.norm() * (2.0**-18 + 4 * U) + old.norm() * 2 * U
