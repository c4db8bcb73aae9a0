"""What the binding of the training-step operators keeps to: autograd's checks, streams, bound storage."""
import pytest
import torch

from memory_aware_device_gb300 import build as nbuild
from memory_aware_device_gb300 import train

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()


def test_second_derivatives_of_gate_are_refused():
    """Its gradient has no derivative: a penalty on it raises instead of adding nothing."""
    x = torch.randn(16, 8, device="cuda", requires_grad=True)
    y = (train.gate(x, 2).weights[:, 0] ** 2 * x[:, 0] ** 2).sum()
    grad, = torch.autograd.grad(y, x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (grad ** 2).sum().backward()
    plain, = torch.autograd.grad((train.gate(x, 2).weights[:, 0] ** 2 * x[:, 0] ** 2).sum(), x)
    assert torch.equal(plain, grad.detach())
