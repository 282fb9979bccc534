"""The 64-bit restatements of the gated linear recurrence and the block norms against closed forms and central
differences, and what their entry points refuse before they touch a device."""
import ctypes

import numpy as np
import pytest

import operator_reference as ref
from padding_free_variable_gb300 import _lib, build as pbuild


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return _lib.load()


def test_glr_closed_form():
    # f constant, z constant: h_t = z (1 - a^t) for the tied cell from zero, both directions
    L, H = 9, 3
    f, z = np.full((L, 2, H), 0.7), np.full((L, 2, H), -1.3)
    o = ref.glr([L], f, z)
    a = 1 / (1 + np.exp(-0.7))
    t = np.arange(1, L + 1)
    want = -1.3 * (1 - a ** t)
    np.testing.assert_allclose(o["y"][:, 0, 1], want, rtol=1e-14)
    np.testing.assert_allclose(o["y"][::-1, 1, 1], want, rtol=1e-14)
    np.testing.assert_allclose(o["h_n"][:, 0, 0], want[-1], rtol=1e-14)


@pytest.mark.parametrize("gated", [False, True])
def test_glr_gradients_match_differences(gated):
    rng = np.random.default_rng(5)
    lens, nd, H = [4, 0, 1, 6, 6], 2, 3
    n = sum(lens)
    v = {k: rng.normal(size=(n, nd, H)) for k in ("f", "z", "i", "dy")}
    st = {k: rng.normal(size=(nd, len(lens), H)) for k in ("h0", "dh_n")}
    if not gated:
        v["i"] = None

    def loss():
        o = ref.glr(lens, v["f"], v["z"], v["i"], st["h0"])
        return (o["y"] * v["dy"]).sum() + (o["h_n"] * st["dh_n"]).sum()

    o = ref.glr(lens, v["f"], v["z"], v["i"], st["h0"], v["dy"], st["dh_n"])
    for name, arr, grad in (("f", v["f"], o["df"]), ("z", v["z"], o["dz"]), ("i", v["i"], o["di"]), ("h0", st["h0"], o["dh0"])):
        if arr is None:
            continue
        flat = arr.reshape(-1)
        for k in range(flat.size):
            keep = flat[k]
            flat[k] = keep + 1e-6
            up = loss()
            flat[k] = keep - 1e-6
            down = loss()
            flat[k] = keep
            assert abs((up - down) / 2e-6 - grad.reshape(-1)[k]) < 1e-8, (name, k)


@pytest.mark.parametrize("kind,post,gate", [("rms", None, "silu"), ("layer", None, "sigmoid"), ("rms", "none", "none"),
                                            ("none", "layer", "silu"), ("layer", "rms", "none")])
def test_block_norm_gradients_match_differences(kind, post, gate):
    rng = np.random.default_rng(6)
    n, D = 3, 5
    v = {k: rng.normal(size=(n, D)) for k in ("x", "y", "g", "dx_out", "dn")}
    names = ["scale"] + (["w_post", "b_post"] if (post or kind) != "none" else []) + (["w_pre", "b_pre"] if kind != "none" else [])
    p = {k: rng.normal(size=D) for k in names}
    if gate == "none":
        v["g"] = None

    def call(**kw):
        return ref.block_norm(kind, gate, v["x"], v["y"], v["g"], p, 1e-6, post_kind=post, **kw)

    def loss():
        o = call()
        return (o["x_out"] * v["dx_out"]).sum() + ((o["n"] * v["dn"]).sum() if kind != "none" else 0.0)

    o = call(dx_out=v["dx_out"], dn=v["dn"] if kind != "none" else None, backward=True)
    pairs = [(v["x"], o["dx"]), (v["y"], o["dy"])] + ([(v["g"], o["dgate"])] if gate != "none" else []) + \
        [(p[k], o["d" + k]) for k in names]
    for arr, grad in pairs:
        flat = arr.reshape(-1)
        for k in range(flat.size):
            keep = flat[k]
            flat[k] = keep + 1e-6
            up = loss()
            flat[k] = keep - 1e-6
            down = loss()
            flat[k] = keep
            assert abs((up - down) / 2e-6 - grad.reshape(-1)[k]) < 1e-7 * (1 + abs(grad.reshape(-1)[k]))


def test_glr_refusals_without_a_device(lib):
    ok = _lib.GlrShape(32, 1, 0, 0)
    g = _lib.GlrGates(256, 512, None, 32, 32)
    assert lib.lstm_glr_workspace_bytes(None, ctypes.byref(ok)) == 0
    bad = _lib.LSTM_ERR_INVALID_ARG
    assert lib.lstm_glr_fwd(None, ctypes.byref(ok), ctypes.byref(g), None, 256, None, None, None, None) == bad
    assert lib.lstm_glr_bwd(None, ctypes.byref(ok), ctypes.byref(g), 256, 256, None, ctypes.byref(g), None, None, None) == bad

    def step(shape=ok, gates=g, rows=4, slots=None, n=4, state=256, y=256):
        return lib.lstm_glr_step(ctypes.byref(shape) if shape else None, ctypes.byref(gates) if gates else None, rows,
                                 slots, n, state, state, y, None)

    assert step(rows=0) == _lib.LSTM_OK
    for kw in (dict(shape=None), dict(gates=None), dict(rows=-1), dict(n=3), dict(state=None), dict(y=None), dict(y=258),
               dict(state=258), dict(shape=_lib.GlrShape(0, 1, 0, 0)), dict(shape=_lib.GlrShape(32, 2, 0, 0)),
               dict(shape=_lib.GlrShape(32, 1, 2, 0)), dict(shape=_lib.GlrShape(32, 1, 0, 2)),
               dict(shape=_lib.GlrShape(32, 1, 0, 1)), dict(slots=258), dict(gates=_lib.GlrGates(256, 512, 768, 32, 32)),
               dict(gates=_lib.GlrGates(257, 512, None, 32, 32)), dict(gates=_lib.GlrGates(256, 512, None, 31, 32)),
               dict(gates=_lib.GlrGates(None, 512, None, 32, 32))):
        assert step(**kw) == bad, kw
    assert step(shape=_lib.GlrShape(65537, 1, 0, 0)) == _lib.LSTM_ERR_UNSUPPORTED


def test_block_norm_refusals_without_a_device(lib):
    S, P, IN = _lib.BlockNormShape, _lib.BlockNormParams, _lib.BlockNormInputs
    bad = _lib.LSTM_ERR_INVALID_ARG

    def fwd(shape=S(32, 1, 1, 2, 0, 0, 0, 1e-6), p=P(), rin=IN(256, 512, 768, 32, 32), rows=4, x_out=256, n=256, stats=None):
        return lib.lstm_block_norm_fwd(ctypes.byref(shape) if shape else None, ctypes.byref(p) if p else None,
                                       ctypes.byref(rin) if rin else None, rows, x_out, n, stats, None)

    def bwd(shape=S(32, 1, 1, 2, 0, 0, 0, 1e-6), p=P(), rin=IN(256, 512, 768, 32, 32), rows=4, stats=256, dn=256,
            din=IN(256, 512, 768, 32, 32), scratch=256, grads=P()):
        return lib.lstm_block_norm_bwd(ctypes.byref(shape), ctypes.byref(p), ctypes.byref(rin), rows, stats, 256, dn,
                                       ctypes.byref(din) if din else None, ctypes.byref(grads) if grads else None, scratch, None)

    assert fwd(rows=0) == _lib.LSTM_OK
    shapes = [S(0, 1, 1, 2, 0, 0, 0, 1e-6), S(32, 3, 1, 2, 0, 0, 0, 1e-6), S(32, 1, -1, 2, 0, 0, 0, 1e-6),
              S(32, 1, 1, 3, 0, 0, 0, 1e-6), S(32, 1, 1, 2, 2, 0, 0, 1e-6), S(32, 1, 1, 2, 0, 2, 0, 1e-6),
              S(32, 1, 1, 2, 0, 0, 2, 1e-6), S(32, 1, 1, 2, 0, 0, 0, 0.0), S(32, 1, 1, 2, 0, 0, 0, float("nan"))]
    for s in shapes:
        assert fwd(shape=s) == bad
        assert lib.lstm_block_norm_scratch_bytes(ctypes.byref(s), 4) == 0
    assert fwd(shape=S(16385, 1, 1, 2, 0, 0, 0, 1e-6)) == _lib.LSTM_ERR_UNSUPPORTED
    for kw in (dict(shape=None), dict(p=None), dict(rin=None), dict(rows=-1), dict(rows=1 << 31), dict(x_out=None), dict(n=None),
               dict(x_out=258), dict(n=257), dict(stats=264), dict(p=P(258)), dict(rin=IN(None, 512, 768, 32, 32)),
               dict(rin=IN(256, 512, None, 32, 32)), dict(rin=IN(256, 512, 768, 31, 32)), dict(rin=IN(256, 512, 768, 32, 31)),
               dict(rin=IN(256, None, None, 32, 32)), dict(rin=IN(258, 512, 768, 32, 32)),
               dict(shape=S(32, 0, 1, 2, 0, 0, 0, 1e-6), p=P(256)), dict(shape=S(32, 1, 0, 2, 0, 0, 0, 1e-6), p=P(None, None, None, 256)),
               dict(shape=S(32, 1, 0, 2, 0, 0, 0, 1e-6)), dict(shape=S(32, 1, 1, 0, 0, 0, 0, 1e-6))):
        assert fwd(**kw) == bad, kw
    for kw in (dict(din=None), dict(grads=None), dict(stats=None), dict(stats=264), dict(scratch=None), dict(scratch=264),
               dict(din=IN(None, 512, 768, 32, 32)), dict(din=IN(256, None, 768, 32, 32)), dict(din=IN(256, 512, None, 32, 32)),
               dict(din=IN(256, 512, 768, 31, 32)), dict(din=IN(256, 512, 768, 32, 31)), dict(grads=P(258)), dict(dn=258),
               dict(shape=S(32, 1, 0, 2, 0, 0, 0, 1e-6))):
        assert bwd(**kw) == bad, kw
