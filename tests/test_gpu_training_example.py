"""The training example: the operators together, as a training loop calls them."""
import importlib.util
import math
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(tgs_gpu):
    spec = importlib.util.spec_from_file_location("train_language_model",
                                                  os.path.join(ROOT, "examples", "train_language_model.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.gpu
def test_the_loss_falls(example):
    losses = example.train(steps=60, vocab=512, dim=96, density=0.02, sequences=48, length=33, report=0)
    assert abs(losses[0] - math.log(512)) < 0.5
    assert all(math.isfinite(x) for x in losses) and sum(losses[-5:]) / 5 < 0.6 * losses[0]


@pytest.mark.gpu
def test_gradients_through_the_lookup(example):
    """The example's gradients against the same model in 64 bits, through torch's own indexing."""
    model = example.Model(vocab=300, dim=72, density=0.1)
    tokens, targets = next(example.batches(300, 7, 19))
    model.loss(tokens, targets).backward()
    table, hidden, output = (t.detach().double().requires_grad_() for t in (model.table, model.hidden, model.output))
    h = torch.tanh((table[tokens] * model.scale).flatten(0, 1) @ hidden)
    real = targets.flatten() >= 0
    torch.nn.functional.cross_entropy(h[real] @ output, targets.flatten()[real]).backward()
    for got, want in ((model.table, table), (model.hidden, hidden), (model.output, output)):
        # fp32 products of up to 300 terms and the softmax on the way: sqrt(300) * 8 roundings
        assert (got.grad.double() - want.grad).norm() <= math.sqrt(300) * 8 * 2.0**-24 * want.grad.norm()
