"""Forward-mode derivatives: no operator of the training step has them, so that
a call raises instead of handing back a result without a tangent, which torch
reads as a derivative of zero."""
import pytest
import torch
from torch.autograd import forward_ad

CALLS = {
    "embedding_lookup": lambda t, s, i: lambda tgs: tgs.embedding_lookup(i, t),
    "embedding_grad": lambda t, s, i: lambda tgs: tgs.embedding_grad(i, t[:3], 5),
    "newton_schulz": lambda t, s, i: lambda tgs: tgs.newton_schulz(t),
    "muon_step": lambda t, s, i: lambda tgs: tgs.muon_step(s.clone(), t, torch.zeros_like(s), lr=0.1),
    "layer_norm": lambda t, s, i: lambda tgs: tgs.layer_norm(t),
    "layer_norm weight": lambda t, s, i: lambda tgs: tgs.layer_norm(s, t[0]),
    "layer_norm bias": lambda t, s, i: lambda tgs: tgs.layer_norm(s, None, t[0]),
    "layer_norm out": lambda t, s, i: lambda tgs: tgs.layer_norm(s, out=t),
    "layer_norm_grad": lambda t, s, i: lambda tgs: tgs.layer_norm_grad(t, s, s[:, 0].clone(), s[:, 0].clone()),
    "token_logprobs": lambda t, s, i: lambda tgs: tgs.token_logprobs(t[:3], i),
    "token_logprobs_grad": lambda t, s, i: lambda tgs: tgs.token_logprobs_grad(s[:3], i, s[:3, :2].clone(), t[:3, 0].clone()),
    "distillation_loss": lambda t, s, i: lambda tgs: tgs.distillation_loss(t[:3], i[:, None], s[:3, :1].clone()),
    "distillation_loss teacher": lambda t, s, i: lambda tgs: tgs.distillation_loss(s[:3], i[:, None], t[:3, :1].clone()),
    "distillation_grad": lambda t, s, i: lambda tgs: tgs.distillation_grad(
        s[:3], i[:, None], s[:3, :1].clone(), s[:3, :2].clone(), t[:3, 0].clone()),
    "distillation_loss_and_grad": lambda t, s, i: lambda tgs: tgs.distillation_loss_and_grad(
        s[:3], i[:, None], s[:3, :1].clone(), t[:3, 0].clone()),
}


def refused(tgs, call, device):
    s = torch.randn(6, 4, device=device)
    i = torch.tensor([0, 2, 1], device=device)
    for mode in (torch.enable_grad, torch.no_grad):
        with forward_ad.dual_level(), mode():
            t = forward_ad.make_dual(torch.randn(6, 4, device=device), torch.ones(6, 4, device=device))
            with pytest.raises(NotImplementedError, match="forward-mode"):
                CALLS[call](t, s, i)(tgs)
    return s, i


@pytest.mark.parametrize("call", ["embedding_lookup", "embedding_grad", "newton_schulz", "layer_norm", "token_logprobs",
                                  "distillation_loss"])  # which look at the dual tensor first
def test_dual_tensors_are_refused(call):
    import top_gradient_sparsification_amd as tgs
    refused(tgs, call, "cpu")


@pytest.mark.gpu
@pytest.mark.parametrize("call", CALLS)
def test_dual_tensors_are_refused_on_the_gpu(tgs_gpu, call):
    s, i = refused(tgs_gpu, call, "cuda")
    with forward_ad.dual_level():       # others are not
        inside = CALLS[call](s, s, i)(tgs_gpu)
    outside = CALLS[call](s, s, i)(tgs_gpu)
    first = lambda r: r if isinstance(r, torch.Tensor) else r[0]  # noqa: E731
    if call != "layer_norm out":        # which overwrites s
        assert torch.equal(first(inside), first(outside))


@pytest.mark.gpu
def test_function_transforms_raise(tgs_gpu):
    x = torch.randn(6, 8, device="cuda")
    for transform in (lambda f: torch.func.jvp(f, (x,), (x,)), lambda f: torch.func.vmap(f)(x)):
        with pytest.raises((RuntimeError, NotImplementedError, TypeError)):
            transform(lambda t: tgs_gpu.layer_norm(t))
