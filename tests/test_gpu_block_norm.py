"""The norms around a block on the GPU against their 64-bit restatement, value by value within derived bounds
(operator_reference)."""
import numpy as np
import pytest

import operator_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
VECS = ("w_post", "b_post", "scale", "w_pre", "b_pre")


@pytest.fixture(scope="module", autouse=True)
def _needs_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from padding_free_variable_gb300 import build
    build.build()


def ops():
    from padding_free_variable_gb300 import ops as o
    return o


def near(got, want, bound, dtype, what):
    got, want, bound = got.double().cpu().numpy(), np.asarray(want), np.asarray(bound)
    if dtype == "bf16":
        bound = bound + 2.0 ** -8 * np.abs(want)
    bad = ~(np.abs(got - want) <= bound + 1e-36)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], bound[bad][:4])


class Case:
    def __init__(self, n, D, kind="rms", gate="silu", branch="f32", stream="f32", norm=None, post=None, names=None, pad=0,
                 block=True, errors=("dx_out", "dn"), seed=0, mean=0.1):
        o = ops()
        self.n, self.D, self.kind, self.gate, self.post = n, D, kind, gate if block else "none", post if block else "none"
        self.branch, self.stream, self.norm = branch, stream, norm or branch
        self.shape = o.block_norm_shape(D, kind, self.gate, branch == "bf16", stream == "bf16", self.norm == "bf16", 1e-6,
                                        post_kind=self.post)
        rng = np.random.default_rng(seed + D * 31 + n)

        def rows(dt, mean=0.0, std=1.0, pad=0):
            t = torch.full((n, D + pad), float("nan"), dtype=DT[dt], device="cuda")
            t[:, :D] = torch.from_numpy(rng.normal(mean, std, (n, D))).to("cuda", DT[dt])
            return t[:, :D] if pad else t

        self.x = rows(stream, std=1.4)
        self.y = rows(branch, mean, 0.6, pad) if block else None
        self.g = rows(branch, std=1.3, pad=2 * pad) if self.gate != "none" else None
        pk = kind if post is None else post
        if names is None:
            names = [k for k in VECS if (block or k in ("w_pre", "b_pre")) and not (k.endswith("post") and pk == "none")
                     and not (k.endswith("pre") and kind == "none")]
        self.p = {k: torch.from_numpy(rng.normal(0 if k[0] == "b" else 1, 0.3, D)).float().cuda() for k in names}
        self.dx_out = rows(stream, std=0.7) if "dx_out" in errors else None
        self.dn = rows(self.norm) if "dn" in errors and kind != "none" else None
        nan = lambda like, pad: None if like is None else torch.full((n, D + pad), float("nan"), dtype=like.dtype, device="cuda")[:, :D]  # noqa: E731
        self.x_out = nan(self.x, 0).contiguous() if block else None
        self.nn = torch.full((n, D), float("nan"), dtype=DT[self.norm], device="cuda") if kind != "none" else None
        self.stats = torch.full((n, 4), float("nan"), device="cuda")
        self.dx, self.dy, self.dg = nan(self.x, 0).contiguous(), nan(self.y, pad), nan(self.g, 3 * pad)
        self.dp = {k: torch.full((D,), float("nan"), device="cuda") for k in names}
        self.scratch = torch.full((o.block_norm_scratch_bytes(self.shape, n),), 255, dtype=torch.uint8, device="cuda")

    def forward(self, stream=None):
        ops().block_norm_forward(self.shape, self.x, self.y, self.g, self.p, self.x_out, self.nn, self.stats, stream)

    def backward(self, stream=None):
        ops().block_norm_backward(self.shape, self.x, self.y, self.g, self.p, self.stats, self.dx_out, self.dn, self.dx, self.dy,
                                  self.dg, self.dp, self.scratch, stream)

    def want(self):
        num = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        return ref.block_norm(self.kind, self.gate, num(self.x), num(self.y), num(self.g), {k: num(v) for k, v in self.p.items()},
                              1e-6, num(self.dx_out), num(self.dn), self.post, True)

    def check(self):
        self.forward()
        self.backward()
        torch.cuda.synchronize()
        w = self.want()
        for got, name, dt in ((self.x_out, "x_out", self.stream), (self.nn, "n", self.norm), (self.dx, "dx", self.stream),
                              (self.dy, "dy", self.branch), (self.dg, "dgate", self.branch)):
            if got is not None:
                near(got, w[name], w["~" + name], dt, name)
        for k, v in self.dp.items():
            near(v, w["d" + k], w["~d" + k], "f32", "d" + k)


CASES = [
    # rows, D, kind, gate, branch, stream, norm dtype, kind after the block, padding of strided rows
    (1, 1, "rms", "silu", "f32", "f32", None, None, 0),
    (3, 2, "layer", "sigmoid", "bf16", "bf16", None, None, 0),
    (1, 8, "rms", "none", "bf16", "f32", None, None, 0),
    (5, 33, "layer", "silu", "f32", "f32", None, None, 0),
    (7, 64, "rms", "silu", "f32", "bf16", "bf16", None, 8),
    (9, 256, "layer", "sigmoid", "bf16", "f32", "f32", None, 16),
    (700, 264, "rms", "silu", "bf16", "bf16", None, None, 0),
    (311, 517, "layer", "sigmoid", "f32", "f32", None, None, 3),
    (64, 511, "rms", "silu", "bf16", "bf16", None, None, 1),
    (1300, 1024, "rms", "silu", "bf16", "bf16", None, None, 0),
    (400, 1024, "layer", "silu", "f32", "f32", "bf16", None, 4),
    (50, 1032, "layer", "sigmoid", "bf16", "bf16", None, None, 0),
    (40, 2048, "rms", "sigmoid", "f32", "f32", None, None, 0),
    (33, 4104, "layer", "silu", "bf16", "f32", None, None, 0),
    (17, 5001, "rms", "none", "f32", "f32", None, None, 0),
    (9, 8192, "layer", "silu", "bf16", "bf16", None, None, 0),
    (5, 16384, "layer", "sigmoid", "f32", "bf16", None, None, 0),
    (3, 16383, "rms", "silu", "bf16", "f32", None, None, 0),
    (30, 128, "rms", "silu", "f32", "f32", None, "none", 0),
    (30, 128, "none", "silu", "bf16", "bf16", None, "layer", 0),
    (30, 136, "layer", "none", "f32", "f32", None, "rms", 0),
    (20, 96, "none", "sigmoid", "f32", "f32", None, "none", 0),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}x{c[1]}-{c[2]}-{c[3]}-{c[4]}-{c[5]}" for c in CASES])
def test_matches_definition(case):
    n, D, kind, gate, branch, stream, norm, post, pad = case
    Case(n, D, kind, gate, branch, stream, norm, post, pad=pad).check()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("D,dtype", [(40, "f32"), (1024, "bf16"), (77, "bf16")])
def test_first_pre_norm_alone(kind, D, dtype):
    Case(37, D, kind, branch=dtype, stream=dtype, block=False).check()


@pytest.mark.parametrize("names", [(), ("scale",), ("w_pre", "b_post")])
def test_absent_parameters(names):
    Case(21, 72, "layer", "silu", names=names).check()


@pytest.mark.parametrize("errors", [("dx_out",), ("dn",), ()])
def test_absent_errors(errors):
    Case(21, 72, "rms", "silu", errors=errors).check()


def test_a_large_mean_keeps_its_deviation():
    # deviations far below the mean: the variance is taken around the mean, not as a difference of squares
    Case(11, 520, "layer", "none", mean=300.0).check()


def test_constant_and_zero_rows():
    c = Case(6, 96, "layer", "silu")
    c.y[1] = 0
    c.y[2] = 2.5
    c.x[1] = 0
    c.g[1] = -80.0
    c.check()


def test_nan_and_infinities_stay_in_their_row():
    c, d = Case(9, 264, "rms", "silu"), Case(9, 264, "rms", "silu")
    d.y[4, 7] = float("nan")
    d.x[6, 1] = float("inf")
    for k in (c, d):
        k.forward()
        k.backward()
    rest = [0, 1, 2, 3, 5, 7, 8]
    for a, b in ((c.x_out, d.x_out), (c.nn, d.nn), (c.dx, d.dx), (c.dy, d.dy), (c.dg, d.dg)):
        assert torch.equal(a[rest], b[rest])
    assert torch.isnan(d.nn[4]).all() and torch.isnan(d.dp["w_post"]).any()


def test_in_place_stream_and_errors():
    c = Case(50, 256, "rms", "silu", "bf16", "bf16")
    c.forward()
    c.backward()
    want = c.x_out.clone(), c.nn.clone(), c.dx.clone()
    c.dx.copy_(c.dx_out)
    ops().block_norm_backward(c.shape, c.x, c.y, c.g, c.p, c.stats, c.dx, c.dn, c.dx, c.dy, c.dg, c.dp, c.scratch)
    assert torch.equal(c.dx, want[2])
    ops().block_norm_forward(c.shape, c.x, c.y, c.g, c.p, c.x, c.nn, None)
    assert torch.equal(c.x, want[0]) and torch.equal(c.nn, want[1])


def test_repeats_agree_bitwise_also_on_another_stream_and_in_a_graph():
    c = Case(5000, 136, "layer", "silu", "bf16", "f32", pad=8)
    c.forward()
    c.backward()
    outs = [c.x_out, c.nn, c.dx, c.dy, c.dg] + list(c.dp.values())
    want = [t.clone() for t in outs]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for t in outs:
        t.fill_(3)
    torch.cuda.synchronize()
    c.forward(s)
    c.backward(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.forward()
        c.backward()
    for t in outs:
        t.fill_(3)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_rows_past_32_bits():
    # gate rows 2^26 elements apart
    n, D, ld = 36, 32, 1 << 26
    c = Case(n, D, "rms", "silu", "bf16", "bf16")
    buf = torch.empty(n * ld, dtype=torch.bfloat16, device="cuda").view(n, ld)
    g, dg = buf[:, :D], buf[:, D:2 * D]
    g.copy_(c.g)
    c.g, c.dg = g, dg
    c.check()


def test_no_rows():
    c = Case(0, 48, "rms", "silu")
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    assert all(not v.any() for v in c.dp.values())


def test_gradient_against_differences():
    c = Case(12, 40, "layer", "silu")
    c.forward()
    c.backward()
    num = lambda t: t.double().cpu().numpy()  # noqa: E731
    rng = np.random.default_rng(3)
    x, y, g, dx_out, dn = (num(t) for t in (c.x, c.y, c.g, c.dx_out, c.dn))
    p = {k: num(v) for k, v in c.p.items()}
    way = {k: rng.normal(size=x.shape) for k in "xyg"}
    wp = {k: rng.normal(size=40) for k in p}

    def loss(e):
        o = ref.block_norm("layer", "silu", x + e * way["x"], y + e * way["y"], g + e * way["g"], {k: v + e * wp[k] for k, v in p.items()})
        return (o["x_out"] * dx_out).sum() + (o["n"] * dn).sum()

    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    parts = [num(a) * way[k] for a, k in ((c.dx, "x"), (c.dy, "y"), (c.dg, "g"))] + [num(c.dp[k]) * wp[k] for k in p]
    assert abs(slope - sum(v.sum() for v in parts)) < 256 * ref.U * sum(np.abs(v).sum() for v in parts) + 1e-8 * abs(slope)


def test_refusals():
    from padding_free_variable_gb300._lib import LSTMError
    o, c = ops(), Case(6, 32, "rms", "silu")
    args = dict(shape=c.shape, x=c.x, y=c.y, gate=c.g, params=c.p, x_out=c.x_out, n=c.nn, stats=c.stats)
    for kw in (dict(x=c.x.double()), dict(x=c.x[:, :16]), dict(y=c.y[:5]), dict(gate=c.g.t()), dict(params={"scale": c.p["scale"][:9]}),
               dict(n=c.nn.bfloat16()), dict(stats=c.stats[:, :2]), dict(x_out=c.x_out[:, ::2])):
        with pytest.raises(ValueError):
            o.block_norm_forward(**{**args, **kw})
    for kw in (dict(gate=None), dict(n=None), dict(y=None)):
        with pytest.raises(LSTMError):
            o.block_norm_forward(**{**args, **kw})
    with pytest.raises(ValueError):
        o.block_norm_shape(32, "mean")
    with pytest.raises(ValueError):
        o.block_norm_shape(32, gate="tanh")
