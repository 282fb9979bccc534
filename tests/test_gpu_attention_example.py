"""The linear attention example end to end: the operators together, gradients against differences of their own loss, and
streaming that agrees with whole sequences."""
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


def test_trains_and_streams():
    import linear_attention as ex
    lengths = [40, 0, 7, 90, 1, 64]
    stack, xp, losses = ex.train(lengths, heads=3, size=16, layers=2, steps=5)
    assert len(losses) == 5 and all(v == v and v < float("inf") for v in losses)
    # both run fp32 arithmetic; the projection adds three bf16 pieces' products where torch adds fp32 ones
    assert ex.compare_streaming(stack, xp, lengths) < 2e-3


def test_gradients_of_the_whole_stack():
    import linear_attention as ex
    from padding_free_variable_gb300 import ops
    plan = ops.Plan([9, 30, 2, 17])
    stack = ex.LinearAttentionStack(plan, 2, 16, 2, seed=3)
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
