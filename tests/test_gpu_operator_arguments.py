"""Tensors and streams of another device than the call's, in every argument of the gated linear recurrence's and the block
norms' calls: refused before a launch."""
import types

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from padding_free_variable_gb300 import build
    build.build()


def calls():
    """(function, its keyword arguments) of each call."""
    from padding_free_variable_gb300 import ops
    lens, H = [4, 2], 16
    plan, n = ops.Plan(lens), 6
    t = lambda *s: torch.randn(s, device="cuda")  # noqa: E731
    shape = ops.glr_shape(H, 1, False, "gated")
    ws = torch.zeros(ops.glr_workspace_bytes(plan, shape), dtype=torch.uint8, device="cuda")
    gates = {k: t(n, 1, H) for k in "fzi"}
    yield ops.glr_forward, dict(plan=plan, shape=shape, **gates, h0=t(1, 2, H), y=t(n, 1, H), h_n=t(1, 2, H), workspace=ws)
    yield ops.glr_backward, dict(plan=plan, shape=shape, **gates, workspace=ws, dy=t(n, 1, H), dh_n=t(1, 2, H), df=t(n, 1, H),
                                 dz=t(n, 1, H), di=t(n, 1, H), dh0=t(1, 2, H))
    yield ops.glr_step, dict(shape=shape, **gates, state_in=t(9, H), state_out=t(9, H), y=t(n, 1, H),
                             slots=torch.arange(n, dtype=torch.int32, device="cuda"))
    norm = ops.block_norm_shape(H, "layer")
    p = {k: t(H) for k in ("w_post", "b_post", "scale", "w_pre", "b_pre")}
    rows = {k: t(n, H) for k in ("x", "y", "gate")}
    yield ops.block_norm_forward, dict(shape=norm, **rows, params=p, x_out=t(n, H), n=t(n, H), stats=t(n, 4))
    scratch = torch.zeros(ops.block_norm_scratch_bytes(norm, n), dtype=torch.uint8, device="cuda")
    yield ops.block_norm_backward, dict(shape=norm, **rows, params=p, stats=t(n, 4), dx_out=t(n, H), dn=t(n, H), dx=t(n, H),
                                        dy=t(n, H), dgate=t(n, H), grads={k: t(H) for k in p}, scratch=scratch)


def test_every_tensor_has_to_be_on_the_device():
    seen = 0
    for fn, args in calls():
        fn(**args)      # as it is: taken
        for name, v in args.items():
            bad = [v.cpu()] if isinstance(v, torch.Tensor) else [{**v, k: t.cpu()} for k, t in v.items()] if isinstance(v, dict) else []
            for b in bad:
                with pytest.raises(ValueError):
                    fn(**{**args, name: b})
                seen += 1
    torch.cuda.synchronize()
    assert seen == 7 + 10 + 7 + 11 + 20


def test_the_device_has_to_be_the_current_one(monkeypatch):
    all_calls = list(calls())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for fn, args in all_calls:
        with pytest.raises(ValueError, match="current CUDA device"):
            fn(**args)


def test_streams_of_another_device():
    for fn, args in calls():
        with pytest.raises(ValueError, match="stream"):
            fn(**args, stream=types.SimpleNamespace(cuda_stream=0, device_index=1))
        fn(**args, stream=torch.cuda.Stream())
        torch.cuda.synchronize()
