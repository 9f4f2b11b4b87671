"""Autograd of the attention on the GPU: what a gradient of its gradients does."""
import pytest
import torch

from exact_head_attention_gb300 import exattn

pytestmark = pytest.mark.gpu


def _leaves(n):
    g = torch.Generator().manual_seed(1)
    return [torch.randn((1, 2, 128, 64), generator=g).to(torch.bfloat16).cuda().requires_grad_() for _ in range(n)]


@pytest.mark.parametrize("which", ["attention", "student", "teacher"])
def test_second_gradients_raise(which):
    """A penalty on gradients, beside another term that has its own: raised, not left out; first gradients as ever."""
    x = _leaves(3 if which == "attention" else 4)

    def loss():
        if which == "attention":
            return exattn.attention(*x, causal=True, dq_mode="deterministic").float().sum()
        return exattn.attention_kl(*x, causal=True, train=which, dq_mode="deterministic").sum()

    trained = x if which == "attention" else x[2:] if which == "student" else x[:2]
    first = torch.autograd.grad(loss(), trained, create_graph=True)
    for a, b in zip(first, torch.autograd.grad(loss(), trained)):
        assert torch.equal(a, b)
    with pytest.raises(RuntimeError, match="once"):
        (sum(g.float().square().sum() for g in first) + x[0].float().square().sum()).backward()
