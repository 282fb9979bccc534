"""The 64-bit restatements of linear attention and of the norms and rotations of queries and keys against closed forms and
central differences, the frequency tables, and what the entry points refuse before they touch a device."""
import ctypes
import types

import numpy as np
import pytest

import attention_reference as ref
from padding_free_variable_gb300 import _lib, build as pbuild

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return _lib.load()


@pytest.fixture(scope="module")
def ops():
    pbuild.build()
    from padding_free_variable_gb300 import ops as o
    return o


def differences(arrays, loss):
    """Central differences of loss() in every value of the arrays."""
    for name, arr, grad in arrays:
        flat = arr.reshape(-1)
        for i in range(flat.size):
            keep = flat[i]
            flat[i] = keep + 1e-6
            up = loss()
            flat[i] = keep - 1e-6
            down = loss()
            flat[i] = keep
            assert abs((up - down) / 2e-6 - grad.reshape(-1)[i]) < 2e-7 * (1 + abs(grad.reshape(-1)[i])), (name, i)


def test_attend_closed_form():
    # every frame alike: S_t = (1 - lambda^t) / (1 - lambda) k v^T, in both directions
    L, a, b = 7, 3, 2
    q, k, v = (np.tile(x, (L, 2, 1, 1)) for x in (np.array([1.0, -2, 0.5]), np.array([0.3, 0.1, -1]), np.array([2.0, -1])))
    ld = np.log(np.array([[0.9], [0.5]]))
    o = ref.attend([L], q, k, v, ld, 0.7)
    t = np.arange(1, L + 1)
    for d, lam in ((0, 0.9), (1, 0.5)):
        s = (1 - lam ** t) / (1 - lam)
        y = o["y"][:, d, 0] if d == 0 else o["y"][::-1, d, 0]
        np.testing.assert_allclose(y, 0.7 * (q[0, 0, 0] @ k[0, 0, 0]) * s[:, None] * v[0, 0, 0], rtol=1e-13)
        np.testing.assert_allclose(o["s_n"][d, 0, 0], s[-1] * np.outer(k[0, 0, 0], v[0, 0, 0]), rtol=1e-13)
    assert (a, b) == o["s_n"].shape[3:]


def test_attend_without_decay_is_a_sum_and_without_memory_one_frame():
    rng = np.random.default_rng(3)
    lens, H = [5, 0, 3], 2
    q, k, v = (rng.normal(size=(8, 1, H, 3)) for _ in range(3))
    o = ref.attend(lens, q, k, v, np.array([[0.0, -np.inf]]), 1.0)
    rows, _ = ref.packed_rows(lens)
    r = rows[0]
    np.testing.assert_allclose(o["y"][r[-1], 0, 0], sum((q[r[-1], 0, 0] @ k[x, 0, 0]) * v[x, 0, 0] for x in r), rtol=1e-12)
    np.testing.assert_allclose(o["y"][r[-1], 0, 1], (q[r[-1], 0, 1] @ k[r[-1], 0, 1]) * v[r[-1], 0, 1], rtol=1e-12)
    assert not o["s_n"][0, 1].any()


def test_attend_gradients_match_differences():
    rng = np.random.default_rng(5)
    lens, nd, H, a, b = [3, 0, 1, 4], 2, 2, 2, 3
    n = sum(lens)
    x = {m: rng.normal(size=(n, nd, H, w)) for m, w in (("q", a), ("k", a), ("v", b), ("dy", b))}
    st = {m: rng.normal(size=(nd, len(lens), H, a, b)) for m in ("s0", "ds_n")}
    ld = np.log(rng.uniform(0.3, 1.0, size=(nd, H)))

    def loss():
        o = ref.attend(lens, x["q"], x["k"], x["v"], ld, 0.6, st["s0"])
        return (o["y"] * x["dy"]).sum() + (o["s_n"] * st["ds_n"]).sum()

    o = ref.attend(lens, x["q"], x["k"], x["v"], ld, 0.6, st["s0"], x["dy"], st["ds_n"])
    differences([("q", x["q"], o["dq"]), ("k", x["k"], o["dk"]), ("v", x["v"], o["dv"]), ("s0", st["s0"], o["ds0"])], loss)


@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
@pytest.mark.parametrize("layout,rotary", [("half", 4), ("interleaved", 4), ("half", 6), ("interleaved", 0)])
def test_qk_norm_gradients_match_differences(kind, layout, rotary):
    rng = np.random.default_rng(7)
    n, h, d = 2, 2, 7
    x, g, w, pos = rng.normal(size=(n, h, d)), rng.normal(size=(n, h, d)), rng.normal(size=d), np.array([3, 41])
    freq = 0.7 ** np.arange(rotary // 2)
    call = lambda **kw: ref.qk_norm(kind, layout, rotary, x, w, freq, pos, 1e-3, 1.3, **kw)  # noqa: E731
    o = call(dout=g)
    differences([("x", x, o["dx"]), ("w", w, o["dw"])], lambda: (call()["out"] * g).sum())


def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(9)
    x = rng.normal(size=(1, 1, 8))
    freq = np.array([1.0, 0.3, 0.05, 0.01])
    for layout in ("half", "interleaved"):
        at = lambda p, v: ref.qk_norm("none", layout, 8, v, None, freq, np.array([p]))["out"]  # noqa: E731
        assert abs(np.linalg.norm(at(17, x)) - np.linalg.norm(x)) < 1e-12
        y = rng.normal(size=(1, 1, 8))
        assert abs((at(5, x) * at(9, y)).sum() - (at(105, x) * at(109, y)).sum()) < 1e-12


def test_tables(ops):
    f = ops.rotary_frequencies(8, 10000.0)
    np.testing.assert_allclose(f, [1, 0.1, 0.01, 0.001], rtol=1e-14)
    np.testing.assert_allclose(ops.rotary_frequencies(8, 10000.0, stretch=4.0), f / 4, rtol=1e-14)
    g = ops.rotary_frequencies(8, 10000.0, stretch=4.0, trained=2 * np.pi * 100, ramp=(0.5, 9.5))
    # turns within the trained length: 100, 10 (kept), 1 (mixed: 1/18), 0.1 (slowed)
    np.testing.assert_allclose(g, [1, 0.1, 0.01 * (1 / 18 + 17 / 72), 0.001 / 4], rtol=1e-12)
    t = ops.rotary_table([0.0, np.pi, -np.pi / 2, 2 * np.pi * 5.25, 1.0], device="cpu").numpy().view(np.uint64)
    turn = t.astype(np.float64) / 2.0 ** 64
    np.testing.assert_allclose(turn, [0, 0.5, 0.75, 0.25, 1 / (2 * np.pi)], rtol=1e-15)
    # far positions keep their angle: 2^31 times a rounding of 2^-65 turn
    at = 2 ** 31 - 1
    frac = ((int(t[4]) * at) % 2 ** 64) / 2.0 ** 64
    assert abs(np.sin(2 * np.pi * frac) - np.sin(float(at))) < 1e-7
    for bad in (lambda: ops.rotary_frequencies(7), lambda: ops.rotary_frequencies(8, ramp=(2.0, 2.0)),
                lambda: ops.rotary_table([float("inf")], "cpu"), lambda: ops.rotary_table([[1.0]], "cpu"),
                lambda: ops.qk_norm_shape(1, 1, 8, kind="batch"), lambda: ops.qk_norm_shape(1, 1, 8, layout="thirds")):
        with pytest.raises(ValueError):
            bad()


def test_attend_refusals_without_a_device(lib):
    bad, S, R, IN = _lib.LSTM_ERR_INVALID_ARG, _lib.LaShape, _lib.LaRows, _lib.LaInputs
    ok = S(2, 16, 8, 1, 0, 0.25)
    rows = IN(R(256, 96, 32, 16), R(512, 96, 32, 16), R(768, 48, 16, 8))
    ref_ = lambda x: ctypes.byref(x) if x is not None else None  # noqa: E731
    assert lib.lstm_la_scratch_bytes(None, ref_(ok)) == 0
    assert lib.lstm_la_fwd(None, ref_(ok), ref_(rows), 256, None, 256, None, None, None) == bad
    assert lib.lstm_la_bwd(None, ref_(ok), ref_(rows), 256, None, 256, None, ref_(rows), None, None, None) == bad

    def step(shape=ok, rin=rows, decay=256, n=4, slots=None, count=4, sin=4096, sout=4096, y=256):
        return lib.lstm_la_step(ref_(shape), ref_(rin), decay, n, slots, count, sin, sout, y, None)

    assert step(n=0) == _lib.LSTM_OK
    for kw in (dict(shape=None), dict(rin=None), dict(decay=None), dict(decay=258), dict(n=-1), dict(count=3), dict(sin=None),
               dict(sout=None), dict(sout=4100), dict(y=None), dict(y=258), dict(slots=258), dict(sin=4098),
               dict(shape=S(0, 16, 8, 1, 0, 1.0)), dict(shape=S(2, 0, 8, 1, 0, 1.0)), dict(shape=S(2, 16, 0, 1, 0, 1.0)),
               dict(shape=S(2, 16, 8, 2, 0, 1.0)), dict(shape=S(2, 16, 8, 1, 2, 1.0)), dict(shape=S(2, 16, 8, 1, 0, float("nan"))),
               dict(shape=S(2, 16, 8, 1, 0, float("inf"))), dict(rin=IN(R(None, 96, 32, 16), rows.k, rows.v)),
               dict(rin=IN(R(258, 96, 32, 16), rows.k, rows.v)), dict(rin=IN(rows.q, R(512, -1, 32, 16), rows.v)),
               dict(rin=IN(rows.q, rows.k, R(768, 48, 16, -8))), dict(rin=IN(rows.q, rows.k, R(768, 48, (1 << 40) + 1, 8)))):
        assert step(**kw) == bad, kw
    for s in (S(2, 129, 8, 1, 0, 1.0), S(2, 16, 129, 1, 0, 1.0), S(4097, 16, 8, 1, 0, 1.0)):
        assert step(shape=s) == _lib.LSTM_ERR_UNSUPPORTED


def test_qk_norm_refusals_without_a_device(lib):
    bad, S, P, R, G = _lib.LSTM_ERR_INVALID_ARG, _lib.QkNormShape, _lib.QkNormParams, _lib.QkRows, _lib.QkNormGrads
    ok = S(2, 1, 16, 1, 8, 0, 0, 1e-6, 1.0)
    par, rows = P(256, 512, 1024, 2048, 0), R(256, 768, 48, 16, 48, 16)
    ref_ = lambda x: ctypes.byref(x) if x is not None else None  # noqa: E731

    def fwd(shape=ok, p=par, rin=rows, n=4, out=rows):
        return lib.lstm_qk_norm_fwd(None, ref_(shape), ref_(p), ref_(rin), n, ref_(out), None)

    def bwd(shape=ok, p=par, rin=rows, n=4, dout=rows, din=rows, g=G(256, 512), scratch=256):
        return lib.lstm_qk_norm_bwd(None, ref_(shape), ref_(p), ref_(rin), n, ref_(dout), ref_(din), ref_(g), scratch, None)

    assert fwd(n=0) == _lib.LSTM_OK and bwd(n=0, g=G(None, None)) == _lib.LSTM_OK
    shapes = [S(0, 1, 16, 1, 8, 0, 0, 1e-6, 1), S(2, -1, 16, 1, 8, 0, 0, 1e-6, 1), S(2, 1, 0, 1, 0, 0, 0, 1e-6, 1),
              S(2, 1, 16, 3, 8, 0, 0, 1e-6, 1), S(2, 1, 16, 1, 7, 0, 0, 1e-6, 1), S(2, 1, 16, 1, 18, 0, 0, 1e-6, 1),
              S(2, 1, 16, 1, -2, 0, 0, 1e-6, 1), S(2, 1, 16, 1, 8, 2, 0, 1e-6, 1), S(2, 1, 16, 1, 8, 0, 2, 1e-6, 1),
              S(2, 1, 16, 1, 8, 0, 0, 0.0, 1), S(2, 1, 16, 1, 8, 0, 0, float("nan"), 1), S(2, 1, 16, 1, 8, 0, 0, 1e-6, float("inf"))]
    for s in shapes:
        assert fwd(shape=s) == bad and lib.lstm_qk_norm_scratch_bytes(ref_(s), 4) == 0
    for s in (S(2, 1, 257, 1, 8, 0, 0, 1e-6, 1), S(4097, 1, 16, 1, 8, 0, 0, 1e-6, 1), S(2, 4097, 16, 1, 8, 0, 0, 1e-6, 1)):
        assert fwd(shape=s) == _lib.LSTM_ERR_UNSUPPORTED
    common = [dict(shape=None), dict(p=None), dict(rin=None), dict(n=-1), dict(n=1 << 31), dict(p=P(258, 512, 1024, 2048, 0)),
              dict(p=P(256, 512, None, 2048, 0)), dict(p=P(256, 512, 1028, 2048, 0)), dict(p=P(256, 512, 1024, None, 0)),
              dict(p=P(256, 512, 1024, 2050, 0)), dict(rin=R(None, 768, 48, 16, 48, 16)), dict(rin=R(256, None, 48, 16, 48, 16)),
              dict(rin=R(258, 768, 48, 16, 48, 16)), dict(rin=R(256, 768, -1, 16, 48, 16)),
              dict(shape=S(2, 1, 16, 0, 8, 0, 0, 1e-6, 1)), dict(shape=S(2, 0, 16, 1, 8, 0, 0, 1e-6, 1))]
    for kw in common:
        assert fwd(**kw) == bad and bwd(**kw) == bad, kw
    # written rows that share places
    for r in (R(256, 768, 31, 16, 48, 16), R(256, 768, 48, 15, 48, 16), R(256, 768, 0, 16, 48, 16), R(256, 768, 16, 32, 48, 16),
              R(256, 768, 48, 16, 15, 16), R(256, None, 48, 16, 48, 16)):
        assert fwd(out=r) == bad and bwd(din=r) == bad
    for kw in (dict(dout=None), dict(din=None), dict(g=None), dict(scratch=None), dict(scratch=264), dict(g=G(258, None)),
               dict(g=G(None, 514)), dict(dout=R(256, None, 48, 16, 48, 16))):
        assert bwd(**kw) == bad, kw
    assert fwd(out=None) == bad


STREAM = types.SimpleNamespace(cuda_stream=0, device_index=0)


@pytest.mark.parametrize("stream", [None, STREAM], ids=["current", "given"])
def test_host_tensors_are_refused(ops, stream):
    n, t = 6, lambda *s: torch.zeros(s)  # noqa: E731
    shape, norm = ops.la_shape(2, 16, 8), ops.qk_norm_shape(2, 2, 16, "rms", 8)
    plan = types.SimpleNamespace(rows=n, batch=2, handle=None, scratch={shape.key: 0})
    q, k, v, y, st, ld = t(n, 1, 2, 16), t(n, 1, 2, 16), t(n, 1, 2, 8), t(n, 1, 2, 8), t(1, 2, 2, 16, 8), t(1, 2)
    a, w, tab, pos = t(n, 2, 16), t(16), torch.zeros(4, dtype=torch.int64), torch.zeros(n, dtype=torch.int32)
    for call in (lambda: ops.la_forward(plan, shape, q, k, v, ld, st, y, st.clone(), stream),
                 lambda: ops.la_backward(plan, shape, q, k, v, ld, st, y, st, q, k, v, st.clone(), stream),
                 lambda: ops.la_step(shape, q, k, v, ld, t(n, 2, 16, 8), t(n, 2, 16, 8), y, None, stream),
                 lambda: ops.qk_norm_forward(norm, a, a, w, w, tab, pos, a, a, None, 0, stream),
                 lambda: ops.qk_norm_backward(norm, a, a, w, w, tab, pos, a, a, a, a, w, w, t(1 << 16), None, 0, stream)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
