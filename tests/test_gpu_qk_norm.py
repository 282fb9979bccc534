"""Norms and rotations of queries and keys on the GPU against their 64-bit restatement, value by value within derived bounds
(attention_reference), over head sizes, layouts, strides, positions and plans where they can go wrong."""
import numpy as np
import pytest

import attention_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


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
        bound = bound + ref.BF16 * (np.abs(want) + bound)
    bad = ~(np.abs(got - want) <= bound + 1e-36)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], bound[bad][:4])


class Case:
    def __init__(self, n, qh, kh, d, kind="rms", rotary=0, layout="half", dtype="f32", gap=0, shift=0, plan=None, positions=None,
                 first=0, weights=True, seed=0, turn_scale=1.0, head_major=False):
        o, rng = ops(), np.random.default_rng(seed + 17 * d + qh)
        self.plan, self.first, self.dtype, self.kind, self.layout, self.rotary = plan, first, dtype, kind, layout, rotary
        self.turn_scale = turn_scale
        n = plan.rows if plan is not None else n
        self.n, self.heads, self.d = n, (qh, kh), d
        dt = DT[dtype]
        self.shape = o.qk_norm_shape(qh, kh, d, kind, rotary, layout, dtype == "bf16", 1e-5, turn_scale)
        width = (qh + kh) * d + gap

        def rows(fill=None):
            b = torch.full((n * width + shift + 16,), float("nan"), dtype=dt, device="cuda")
            t = b[shift:shift + n * width].view(n, width)
            q, k = t[:, :qh * d].unflatten(1, (qh, d)), t[:, qh * d:(qh + kh) * d].unflatten(1, (kh, d))
            if head_major:
                t = b[shift:shift + n * (qh + kh) * d].view(qh + kh, n, d)
                q, k = t[:qh].transpose(0, 1), t[qh:].transpose(0, 1)
            if fill is not None:
                q.copy_(torch.from_numpy(fill(size=(n, qh, d))))
                k.copy_(torch.from_numpy(fill(size=(n, kh, d))))
            return b, q, k if kh else None

        _, *self.x = rows(lambda size: rng.normal(0.2, 1.5, size=size))
        _, *self.dout = rows(rng.normal)
        self.obuf, *self.out = rows()
        self.dbuf, *self.dx = rows()
        on = weights and kind != "none"
        self.w = [torch.from_numpy(rng.normal(1, 0.3, size=d)).float().cuda() if on and h else None for h in (qh, kh)]
        self.dw = [torch.full((d,), float("nan"), device="cuda") if on and h else None for h in (qh, kh)]
        self.freq = o.rotary_frequencies(rotary) if rotary else None
        self.table = o.rotary_table(self.freq) if rotary else None
        self.pos = positions
        self.positions = None if positions is None else torch.tensor(positions, dtype=torch.int32, device="cuda")
        self.scratch = torch.full((o.qk_norm_scratch_bytes(self.shape, n),), 255, dtype=torch.uint8, device="cuda")

    def forward(self, out=None, **kw):
        ops().qk_norm_forward(self.shape, *self.x, *self.w, self.table, self.positions, *(out or self.out), plan=self.plan,
                              first_position=self.first, **kw)

    def backward(self, **kw):
        ops().qk_norm_backward(self.shape, *self.x, *self.w, self.table, self.positions, *self.dout, *self.dx, *self.dw, self.scratch,
                               plan=self.plan, first_position=self.first, **kw)

    def where(self):
        """positions of the rows, and which are live"""
        live = np.ones(self.n, bool)
        step = np.zeros(self.n, np.int64)
        if self.plan is not None:
            bs, off, _, length = self.plan.tables()
            step = np.repeat(np.arange(len(bs)), np.diff(off))
            slot = np.arange(self.n) - off[step]
            live = step < length[slot]
        return (step + self.first if self.pos is None else np.array(self.pos, dtype=np.int64)), live

    def check(self, backward=True):
        self.forward()
        if backward:
            self.backward()
        torch.cuda.synchronize()
        pos, live = self.where()
        num = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        for m in range(2):
            if self.heads[m] == 0:
                continue
            w = ref.qk_norm(self.kind, self.layout, self.rotary, num(self.x[m]), num(self.w[m]), self.freq, pos, 1e-5, self.turn_scale,
                            num(self.dout[m]) if backward else None, live)
            near(self.out[m], w["out"], w["~out"], self.dtype, "out")
            if backward:
                near(self.dx[m], w["dx"], w["~dx"], self.dtype, "dx")
                if self.dw[m] is not None:
                    near(self.dw[m], w["dw"], w["~dw"], "f32", "dw")


CASES = [
    # rows, q heads, k heads, size, kind, rotary, layout, dtype, gap, shift
    (1, 1, 0, 1, "rms", 0, "half", "f32", 0, 0),
    (1, 1, 1, 2, "none", 2, "half", "f32", 0, 0),
    (5, 2, 1, 3, "layer", 2, "interleaved", "f32", 1, 1),
    (33, 8, 8, 64, "rms", 64, "half", "bf16", 512, 0),
    (33, 8, 8, 64, "rms", 64, "interleaved", "bf16", 512, 0),
    (33, 8, 2, 64, "rms", 32, "half", "f32", 0, 0),
    (33, 8, 2, 64, "layer", 32, "interleaved", "f32", 4, 4),
    (100, 3, 5, 128, "layer", 128, "half", "bf16", 0, 0),
    (100, 3, 5, 128, "none", 96, "half", "bf16", 8, 8),
    (57, 5, 2, 74, "layer", 38, "interleaved", "f32", 3, 0),
    (57, 5, 2, 74, "rms", 38, "half", "bf16", 3, 0),
    (57, 5, 2, 77, "rms", 6, "half", "bf16", 3, 1),
    (20, 1, 1, 256, "rms", 256, "half", "f32", 0, 0),
    (20, 1, 1, 255, "layer", 254, "interleaved", "f32", 0, 0),
    (20, 7, 3, 200, "rms", 40, "half", "bf16", 0, 0),
    (20, 7, 3, 200, "rms", 36, "half", "bf16", 0, 0),
    (20, 40, 40, 8, "rms", 8, "half", "bf16", 0, 0),
    (20, 40, 40, 8, "rms", 4, "half", "bf16", 0, 2),
    (20, 33, 1, 16, "layer", 0, "half", "f32", 0, 2),
    (9000, 4, 4, 32, "rms", 32, "half", "bf16", 0, 0),
    (9000, 2, 1, 33, "layer", 12, "interleaved", "f32", 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{i}-{c[1]}+{c[2]}x{c[3]}-{c[4]}-{c[5]}{c[6][0]}-{c[7]}" for i, c in enumerate(CASES)])
def test_matches_definition(case):
    n, qh, kh, d, kind, rotary, layout, dtype, gap, shift = case
    pos = np.random.default_rng(n).integers(0, 100000, n).tolist()
    Case(n, qh, kh, d, kind, rotary, layout, dtype, gap, shift, positions=pos).check()


def test_far_and_negative_positions():
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 12345678, 2 ** 24 + 1, -7]
    for layout in ("half", "interleaved"):
        Case(8, 2, 2, 64, "rms", 64, layout, positions=pos).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_positions_of_plans(dtype):
    o = ops()
    lens = [70, 0, 1, 33, 70, 2]
    for plan, first in ((o.Plan(lens), 0), (o.Plan(lens, window=(20, 30)), 20), (o.Plan(lens, segments=(16, 8)), 0),
                        (o.Plan(lens, padded=True), 0), (o.Plan(lens), 10 ** 12)):
        Case(0, 3, 2, 64, "rms", 48, "half", dtype, plan=plan, first=first).check()
    Case(0, 1, 1, 32, "rms", 32, "interleaved", dtype, plan=o.Plan([5000, 3])).check()
    # positions given beside a padded plan: its masked rows give zeros all the same
    plan = o.Plan([5, 2, 0], padded=True)
    c = Case(0, 2, 2, 16, "layer", 16, "half", dtype, plan=plan, positions=list(range(100, 100 + plan.rows)))
    c.x[0][~torch.from_numpy(c.where()[1]).cuda()] = float("nan")
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    assert torch.isfinite(c.out[0]).all() and torch.isfinite(c.dx[0]).all() and torch.isfinite(c.dw[0]).all()


@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
def test_without_weights_and_with_a_scale(kind):
    Case(40, 2, 3, 48, kind, 32, "half", positions=list(range(40)), weights=False, turn_scale=1.3).check()


def test_in_place_head_major_and_streams():
    for dtype in ("f32", "bf16"):
        c = Case(50, 4, 2, 64, "rms", 64, "half", dtype, positions=list(range(50)), head_major=True)
        c.check()
        want = [t.clone() for t in c.out]
        x = [t.clone(memory_format=torch.preserve_format) for t in c.x]
        c.x = [t.clone(memory_format=torch.preserve_format) for t in x]
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        c.forward(out=c.x, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(c.x, want))
        # gradients over the errors that came in
        c.x, keep, c.dx = x, [t.clone() for t in c.dx], c.dout
        c.backward()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(c.dx, keep))


def test_repeats_bitwise_captures_and_leaves_neighbours():
    c = Case(3000, 3, 2, 40, "rms", 40, "half", "bf16", gap=5, shift=3, positions=[i * 7 for i in range(3000)])
    c.check()
    want = [t.clone() for t in (c.obuf, c.dbuf, *c.dw)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.forward()
        c.backward()
    for t in (*c.out, *c.dx, *c.dw):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (c.obuf, c.dbuf, *c.dw)):
        assert torch.equal(a.nan_to_num(9.0), b.nan_to_num(9.0))
    gap = c.obuf[3:3 + 3000 * 205].view(3000, 205)[:, 200:]
    assert gap.isnan().all() and c.obuf[:3].isnan().all()


def test_wanted_gradients_and_no_rows():
    o = ops()
    c = Case(700, 2, 2, 64, "rms", 64, "half", positions=list(range(700)))
    c.check()
    full, dx = [t.clone() for t in c.dw], [t.clone() for t in c.dx]
    c.dw = [None, c.dw[1].fill_(0)]
    c.backward()
    torch.cuda.synchronize()
    assert torch.equal(c.dw[1], full[1]) and torch.equal(c.dx[0], dx[0])
    c.dw, c.scratch = [None, None], None
    c.backward()
    torch.cuda.synchronize()
    assert torch.equal(c.dx[1], dx[1])
    e = torch.empty(0, 2, 64, device="cuda")
    o.qk_norm_forward(c.shape, e, e, *c.w, c.table, None, e, e, plan=o.Plan([0, 0]))
    o.qk_norm_backward(c.shape, e, e, *c.w, c.table, None, e, e, e, e, *full, torch.empty(16, dtype=torch.uint8, device="cuda"),
                       plan=o.Plan([0]))
    torch.cuda.synchronize()
    assert not full[0].any() and not full[1].any()


def test_bad_arguments():
    o = ops()
    from padding_free_variable_gb300._lib import LSTMError
    c = Case(12, 2, 2, 16, "rms", 8, "half", positions=list(range(12)))
    q, k = c.x
    call = lambda **kw: o.qk_norm_forward(**{**dict(shape=c.shape, q=q, k=k, wq=c.w[0], wk=c.w[1], table=c.table,  # noqa: E731
                                                    positions=c.positions, q_out=c.out[0], k_out=c.out[1]), **kw})
    call()
    for kw in (dict(k=None), dict(k=k[:5]), dict(k=k.double()), dict(wq=c.w[0].double()), dict(table=c.table[:2]), dict(table=c.table.int()),
               dict(positions=c.positions.long()), dict(positions=c.positions[:3]), dict(q_out=None),
               dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(table=None), dict(positions=None), dict(plan=o.Plan([5, 5])), dict(q_out=c.out[0][:, :1].expand(-1, 2, -1)),
               dict(q_out=c.out[0][:1].expand(12, -1, -1))):
        with pytest.raises(LSTMError):
            call(**kw)
    torch.cuda.synchronize()
