"""The Python calls of the gated linear recurrence and the block norms refuse tensors that the GPU cannot reach before they
launch anything."""
import types

import pytest

from padding_free_variable_gb300 import build as pbuild

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ops():
    pbuild.build()
    from padding_free_variable_gb300 import ops as o
    return o


STREAM = types.SimpleNamespace(cuda_stream=0, device_index=0)


@pytest.mark.parametrize("stream", [None, STREAM], ids=["current", "given"])
def test_host_tensors_are_refused(ops, stream):
    n, H = 6, 16
    t = lambda *s: torch.zeros(s)  # noqa: E731
    shape = ops.glr_shape(H, 1, False)
    plan = types.SimpleNamespace(rows=n, batch=2, handle=None, scratch={shape.key: (16, 0)})
    f, z, y, st, ws = t(n, 1, H), t(n, 1, H), t(n, 1, H), t(1, 2, H), torch.zeros(16, dtype=torch.uint8)
    norm = ops.block_norm_shape(H)
    p = {"w_post": t(H), "scale": t(H), "w_pre": t(H)}
    rows = [t(n, H) for _ in range(10)]
    for call in (lambda: ops.glr_forward(plan, shape, f, z, None, st, y, st.clone(), ws, stream),
                 lambda: ops.glr_backward(plan, shape, f, z, None, ws, y, st, t(n, 1, H), t(n, 1, H), None, st.clone(), stream),
                 lambda: ops.glr_step(shape, f, z, None, t(n, H), t(n, H), y, None, stream),
                 lambda: ops.block_norm_forward(norm, *rows[:3], p, rows[3], rows[4], t(n, 4), stream),
                 lambda: ops.block_norm_backward(norm, *rows[:3], p, t(n, 4), *rows[3:8], {}, t(1 << 20), stream)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
