"""The gated recurrence example end to end: every new operator together, its gradients against differences of its own loss,
training that learns, and streaming that agrees with the scan."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _needs_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from padding_free_variable_gb300 import build
    build.build()


def test_learns_and_streams():
    import gated_recurrence as ex
    lengths = [40, 0, 7, 90, 1, 64]
    stack, xp, losses = ex.train(lengths, width=48, layers=2, steps=25)
    assert losses[-1] < 0.6 * losses[0]
    # both run the same fp32 arithmetic but for the projection's summation order (three bf16 pieces against fp32)
    assert ex.compare_streaming(stack, xp, lengths) < 2e-3


def test_gradients_of_the_whole_stack():
    import gated_recurrence as ex
    from padding_free_variable_gb300 import ops
    lengths = [9, 30, 2, 17]
    plan = ops.Plan(lengths)
    stack = ex.GatedRecurrenceStack(plan, 32, 2, seed=3)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(plan.rows, 32, generator=g, device="cuda")
    c = torch.randn(plan.rows, 32, generator=g, device="cuda")
    stack.forward(x)
    grads = stack.backward(c)
    params = stack.parameters()
    way = [torch.randn(p.shape, generator=g, device="cuda") * p.abs().mean().clamp_min(0.05) for p in params]

    def loss(e):
        for p, w in zip(params, way):
            p += e * w
        out = (stack.forward(x).double() * c.double()).sum().item()
        for p, w in zip(params, way):
            p -= e * w
        return out

    want = sum((a.double() * w.double()).sum().item() for a, w in zip(grads, way))
    size = sum((a.double() * w.double()).abs().sum().item() for a, w in zip(grads, way))
    # central difference: fp32 forward noise over the step, and the step squared
    got = (loss(1e-2) - loss(-1e-2)) / 2e-2
    assert abs(got - want) < 0.02 * size
