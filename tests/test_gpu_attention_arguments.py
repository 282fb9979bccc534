"""Tensors and streams of another device than the call's, in every argument of the calls of linear attention and of the norms
of queries and keys: refused before a launch."""
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
    plan, n, H, a, b = ops.Plan([4, 2]), 6, 2, 16, 8
    t = lambda *s: torch.randn(s, device="cuda")  # noqa: E731
    shape = ops.la_shape(H, a, b)
    rows = lambda: {"q": t(n, 1, H, a), "k": t(n, 1, H, a), "v": t(n, 1, H, b)}  # noqa: E731
    ld, st = -t(1, H).abs(), lambda m: t(1, m, H, a, b)  # noqa: E731
    yield ops.la_forward, dict(plan=plan, shape=shape, **rows(), log_decay=ld, s0=st(2), y=t(n, 1, H, b), s_n=st(2))
    yield ops.la_backward, dict(plan=plan, shape=shape, **rows(), log_decay=ld, s0=st(2), dy=t(n, 1, H, b), ds_n=st(2),
                                **{"d" + k: v for k, v in rows().items()}, ds0=st(2))
    yield ops.la_step, dict(shape=shape, **rows(), log_decay=ld, state_in=t(9, H, a, b), state_out=t(9, H, a, b), y=t(n, 1, H, b),
                            slots=torch.arange(n, dtype=torch.int32, device="cuda"))
    norm = ops.qk_norm_shape(H, H, a, "rms", 8)
    common = dict(shape=norm, q=t(n, H, a), k=t(n, H, a), wq=t(a), wk=t(a), table=ops.rotary_table(ops.rotary_frequencies(8)),
                  positions=torch.arange(n, dtype=torch.int32, device="cuda"))
    yield ops.qk_norm_forward, dict(**common, q_out=t(n, H, a), k_out=t(n, H, a))
    scratch = torch.zeros(ops.qk_norm_scratch_bytes(norm, n), dtype=torch.uint8, device="cuda")
    yield ops.qk_norm_backward, dict(**common, dq_out=t(n, H, a), dk_out=t(n, H, a), dq=t(n, H, a), dk=t(n, H, a), dwq=t(a), dwk=t(a),
                                     scratch=scratch)


def test_every_tensor_has_to_be_on_the_device():
    seen = 0
    for fn, args in calls():
        fn(**args)      # as it is: taken
        for name, v in args.items():
            if isinstance(v, torch.Tensor):
                with pytest.raises(ValueError):
                    fn(**{**args, name: v.cpu()})
                seen += 1
    torch.cuda.synchronize()
    assert seen == 7 + 11 + 8 + 8 + 13


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
