"""The training example's norm and its distillation: they run, and their gradients."""
import math

import pytest
import torch

from test_gpu_training_example import example  # noqa: F401 - a fixture


@pytest.mark.gpu
@pytest.mark.parametrize("distill", [False, True])
def test_gradients_with_norm_and_teacher(example, distill):  # noqa: F811
    """Every parameter's gradient against the same model in 64 bits, through torch's own operators."""
    model, first = example.Model(vocab=300, dim=72, density=0.1, norm=True), example.Model(300, 40, 0.1, seed=5)
    with torch.no_grad():
        model.gain.add_(0.1 * torch.randn_like(model.gain))
        model.shift.add_(0.1 * torch.randn_like(model.shift))
    tokens, targets = next(example.batches(300, 7, 19))
    told = first.alternatives(tokens, targets, 8) if distill else None
    loss = model.loss(tokens, targets, told)
    names = ("table", "gain", "shift", "hidden", "output")
    got = torch.autograd.grad(loss, [getattr(model, n) for n in names])

    table, gain, shift, hidden, output = leaves = [getattr(model, n).detach().double().requires_grad_() for n in names]
    x = torch.nn.functional.layer_norm(table[tokens] * model.scale, (72,), gain, shift).flatten(0, 1)
    real = targets.flatten() >= 0
    lp = torch.log_softmax(torch.tanh(x @ hidden) @ output, -1)[real]
    if distill:
        at, t = told[0][real].long(), told[1][real].double()
        assert (told[0][~real] == -1).all()
        q = torch.softmax(t, -1)
        want_loss = (q * (q.log() - lp.gather(1, at))).sum() / real.sum()
    else:
        want_loss = -lp.gather(1, targets.flatten()[real][:, None]).sum() / real.sum()
    assert abs(loss.item() - want_loss.item()) < 1e-4 * (1 + want_loss.item())
    for name, a, c in zip(names, got, torch.autograd.grad(want_loss, leaves)):
        # fp32 products of up to 300 terms, the norm and the softmax on the way: sqrt(300) * 16 roundings
        assert (a.double() - c).norm() <= math.sqrt(300) * 16 * 2.0**-24 * c.norm(), name


@pytest.mark.gpu
def test_it_trains_with_norm_and_distils(example):  # noqa: F811
    first = example.Model(512, 64, 0.02, norm=True)
    sizes = dict(vocab=512, density=0.02, sequences=16, length=33, report=0)
    assert all(math.isfinite(x) for x in example.train(steps=8, dim=64, model=first, **sizes))
    assert all(math.isfinite(x) for x in example.train(steps=8, dim=32, norm=True, teacher=first, **sizes))
