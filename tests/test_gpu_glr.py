"""The gated linear recurrence on the GPU against its 64-bit restatement, value by value within derived bounds
(operator_reference): forward, backward, single frames, over lengths, widths, strides, plans and gates where it can go
wrong."""
import numpy as np
import pytest

import operator_reference as ref

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
    """|got - want| within the bound (and a rounding to bf16)."""
    got, want, bound = got.double().cpu().numpy(), np.asarray(want), np.asarray(bound)
    if dtype == "bf16":
        bound = bound + 2.0 ** -8 * np.abs(want)
    bad = ~(np.abs(got - want) <= bound + 1e-36)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], bound[bad][:4])


class Case:
    def __init__(self, lens, nd, H, dtype="f32", cell="tied", padded=False, states=True, seed=0, window=None, bias=1.5,
                 layout="blocks", shift=0):
        o = ops()
        self.lens, self.nd, self.H, self.dtype, self.gated, self.padded = list(lens), nd, H, dtype, cell == "gated", padded
        self.plan = o.Plan(lens, padded=padded)
        self.shape = o.glr_shape(H, nd, dtype == "bf16", cell)
        rng = np.random.default_rng(seed + 977 * H + len(self.lens))
        n, nb = self.plan.rows, 3 if self.gated else 2
        v = rng.normal(size=(4, n, nd, H)) * np.array([1.5, 1, 1.2, 1]).reshape(4, 1, 1, 1)
        v[0] += bias
        self.v = {k: torch.from_numpy(v[k_]).to("cuda", DT[dtype]) for k_, k in enumerate(("f", "z", "i", "dy"))}
        st = rng.normal(size=(2, nd, len(self.lens), H)) * 0.8
        self.h0, self.dh_n = [torch.from_numpy(s).float().cuda() if states else None for s in st]
        # the gates as a user's projection holds them: blocks of a row, direction by direction, or planes of their own
        e = n * nb * nd * H + shift + 64
        self.buf, self.gbuf = [torch.full((e,), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2)]

        def view(b):
            b = b[shift:]
            if layout == "blocks":
                t = b[:n * nb * nd * H].view(n, nb, nd, H)
                return [t[:, k] for k in range(nb)]
            if layout == "dirs":
                t = b[:n * nb * nd * H].view(n, nd, nb, H)
                return [t[:, :, k] for k in range(nb)]
            t = b[:n * nb * nd * H].view(nb, nd, n, H)
            return [t[k].transpose(0, 1) for k in range(nb)]

        self.gates, self.grads = view(self.buf), view(self.gbuf)
        for k, name in enumerate(("f", "z", "i")[:nb]):
            self.gates[k].copy_(self.v[name])
        if not self.gated:
            self.gates.append(None)
            self.grads.append(None)
        f32 = lambda: torch.full((nd, len(self.lens), H), float("nan"), device="cuda")  # noqa: E731
        self.y = torch.full((n, nd, H), float("nan"), dtype=DT[dtype], device="cuda")
        self.h_n, self.dh0 = f32(), f32()
        self.ws = torch.full((o.glr_workspace_bytes(self.plan, self.shape),), 255, dtype=torch.uint8, device="cuda")

    def forward(self, stream=None, ws=True):
        ops().glr_forward(self.plan, self.shape, *self.gates, self.h0, self.y, self.h_n, self.ws if ws else None, stream)

    def backward(self, stream=None):
        ops().glr_backward(self.plan, self.shape, *self.gates, self.ws, self.v["dy"], self.dh_n, *self.grads, self.dh0, stream)

    def want(self):
        num = {k: t.double().cpu().numpy() for k, t in self.v.items()}
        st = [None if t is None else t.double().cpu().numpy() for t in (self.h0, self.dh_n)]
        return ref.glr(self.lens, num["f"], num["z"], num["i"] if self.gated else None, st[0], num["dy"], st[1], self.padded)

    def check(self):
        self.forward()
        self.backward()
        torch.cuda.synchronize()
        w = self.want()
        near(self.y, w["y"], w["~y"], self.dtype, "y")
        near(self.h_n, w["h_n"], w["~h_n"], "f32", "h_n")
        for k, name in enumerate(("df", "dz", "di")[:3 if self.gated else 2]):
            near(self.grads[k], w[name], w["~" + name], self.dtype, name)
        near(self.dh0, w["dh0"], w["~dh0"], "f32", "dh0")
        assert self.plan.poll() == 0
        return w


MANY = [int(v) for v in np.random.default_rng(8).integers(0, 151, 1000)]
CASES = [
    # lengths, directions, H, dtype, cell, padded, layout, shift (elements off the buffer's start)
    ([1], 1, 1, "f32", "tied", False, "blocks", 0),
    ([1], 2, 8, "bf16", "gated", False, "blocks", 0),
    ([0, 0, 0], 2, 16, "f32", "tied", False, "blocks", 0),
    ([2, 0, 1], 1, 7, "f32", "gated", False, "dirs", 1),
    ([5, 40, 39, 1, 2, 3, 4, 30], 1, 32, "f32", "tied", False, "blocks", 0),
    ([64], 2, 64, "f32", "gated", False, "blocks", 0),
    ([63, 64, 65, 0, 1, 127, 128, 129], 2, 40, "f32", "tied", False, "planes", 0),
    ([63, 64, 65, 0, 1, 127, 128, 129], 2, 40, "bf16", "gated", False, "dirs", 0),
    ([300, 7, 191, 192, 193], 2, 203, "f32", "gated", False, "blocks", 0),
    ([300, 7, 191, 192, 193], 1, 203, "bf16", "tied", False, "blocks", 3),
    ([300, 7, 191, 192, 193], 2, 130, "bf16", "tied", False, "blocks", 2),
    ([257, 8], 2, 132, "f32", "tied", False, "planes", 1),
    ([1500], 1, 256, "bf16", "tied", False, "blocks", 0),
    ([1033, 1], 2, 128, "f32", "gated", False, "blocks", 0),
    ([4100], 2, 33, "f32", "tied", False, "blocks", 0),
    ([2500, 2499], 1, 512, "f32", "tied", False, "blocks", 0),
    ([9000], 1, 64, "bf16", "gated", False, "blocks", 0),
    ([30] * 300, 2, 24, "f32", "tied", False, "blocks", 0),
    # sequences of a tile or two, and many sequences: a warp each
    ([16, 3, 0, 9, 1, 8], 2, 7, "bf16", "gated", False, "blocks", 1),
    ([16, 3, 0, 9, 1, 8], 1, 33, "f32", "tied", False, "dirs", 0),
    ([13, 0, 16, 2], 2, 40, "bf16", "tied", True, "blocks", 0),
    (MANY, 2, 36, "f32", "gated", False, "blocks", 0),
    (MANY, 2, 8, "bf16", "tied", False, "blocks", 0),
    (MANY, 2, 5, "f32", "tied", False, "planes", 0),
    ([5, 0, 17, 70, 3], 2, 16, "f32", "gated", True, "blocks", 0),
    ([5, 0, 17, 170, 3], 2, 96, "bf16", "tied", True, "dirs", 0),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{i}-nd{c[1]}-H{c[2]}-{c[3]}-{c[4]}{'-padded' if c[5] else ''}"
                                             for i, c in enumerate(CASES)])
def test_matches_definition(case):
    lens, nd, H, dtype, cell, padded, layout, shift = case
    Case(lens, nd, H, dtype, cell, padded, layout=layout, shift=shift).check()


LONG, SHORT = [5000, 257, 256, 255, 129, 33, 0, 8], [700, 255, 130, 1]


@pytest.mark.parametrize("lens,nd,H,dtype,cell,padded,layout", [
    (LONG, 2, 8, "bf16", "gated", False, "blocks"), (LONG, 1, 16, "bf16", "tied", False, "planes"),
    (LONG, 2, 24, "bf16", "gated", False, "dirs"), (LONG, 1, 32, "bf16", "tied", False, "blocks"),
    (LONG, 1, 4, "f32", "tied", False, "blocks"), (LONG, 2, 16, "f32", "gated", False, "dirs"),
    (LONG, 2, 20, "f32", "tied", False, "blocks"), (LONG, 1, 32, "f32", "gated", False, "planes"),
    (SHORT, 2, 8, "f32", "gated", False, "blocks"), (SHORT, 1, 24, "f32", "tied", True, "blocks"),
    (SHORT, 2, 16, "bf16", "tied", True, "dirs"), (SHORT, 1, 32, "bf16", "gated", False, "blocks"),
    ([70] * 40 + [300] * 3, 2, 12, "f32", "gated", False, "blocks")])
def test_narrow_layers(lens, nd, H, dtype, cell, padded, layout):
    # at most 32 units: the lanes of a warp divide among steps, cut into pieces and not
    Case(lens, nd, H, dtype, cell, padded, layout=layout).check()


@pytest.mark.parametrize("bias", [-9.0, 0.0, 6.0, 12.0])
def test_gates_near_their_ends(bias):
    # forget gates close to 0 (nothing kept) and to 1 (a memory of thousands of frames): 1 - a keeps its digits
    Case([700, 333], 1, 64, "f32", "tied", bias=bias, seed=3).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinite_gates(dtype):
    c = Case([90, 31], 2, 32, dtype, "gated", seed=4)
    for k, name in enumerate(("f", "i")):
        t = c.v[name]
        t[::7] = float("inf")
        t[3::11] = -float("inf")
        t[5::13] = 100.0
        t[6::17] = -100.0
        c.gates[0 if name == "f" else 2].copy_(t)
    c.check()


def test_nan_stays_in_its_unit_and_sequence():
    c, d = Case([70, 69, 200], 2, 40, seed=9), Case([70, 69, 200], 2, 40, seed=9)
    rows, _ = ref.packed_rows(c.lens)
    d.gates[1][int(rows[1][40]), 0, 5] = float("nan")
    for k in (c, d):
        k.forward()
        k.backward()
    hit = torch.zeros_like(c.y, dtype=torch.bool)
    hit[torch.from_numpy(rows[1]).cuda(), 0, 5] = True
    assert torch.equal(c.y[~hit], d.y[~hit])
    assert torch.isnan(d.y[torch.from_numpy(rows[1][40:]).cuda(), 0, 5]).all()
    assert torch.equal(c.y[torch.from_numpy(rows[1][:40]).cuda(), 0, 5], d.y[torch.from_numpy(rows[1][:40]).cuda(), 0, 5])
    for a, b in zip(c.grads[:2], d.grads[:2]):
        assert torch.equal(a[~hit], b[~hit])


def test_masked_rows_are_not_read():
    lens = [5, 0, 70, 3]
    c, d = Case(lens, 2, 24, padded=True, seed=2), Case(lens, 2, 24, padded=True, seed=2)
    rows, n = ref.packed_rows(lens, True)
    off = torch.ones(n, dtype=torch.bool, device="cuda")
    off[torch.from_numpy(np.concatenate(rows)).cuda()] = False
    for t, bad in ((d.gates[0], float("nan")), (d.gates[1], float("inf")), (d.v["dy"], float("nan"))):
        t[off] = bad
    for k in (c, d):
        k.forward()
        k.backward()
    for a, b in [(c.y, d.y), (c.h_n, d.h_n), (c.dh0, d.dh0)] + list(zip(c.grads[:2], d.grads[:2])):
        assert torch.equal(a, b)
    assert not c.y[off].any() and not c.grads[0][off].any() and not c.grads[1][off].any()


def test_without_states_and_workspace():
    c = Case([40, 129, 0], 2, 48, states=False)
    w = c.check()
    y = c.y.clone()
    c.y.zero_()
    c.forward(ws=False)
    assert torch.equal(y, c.y)
    assert not c.h_n[:, 2].any() and not w["h_n"][:, 2].any()


def test_repeats_agree_bitwise_and_leave_the_rest_alone():
    c = Case([500, 3, 77, 1300], 2, 72, "bf16", "gated", shift=5)
    c.check()
    first = [t.clone() for t in (c.y, c.h_n, c.dh0, c.gbuf)]
    assert torch.isnan(c.gbuf[:5].float()).all() and torch.isnan(c.gbuf[-40:].float()).all()
    for t in (c.y, c.h_n, c.dh0):
        t.fill_(3)
    c.forward()
    c.backward()
    for a, b in zip(first, (c.y, c.h_n, c.dh0, c.gbuf)):
        assert torch.equal(a.nan_to_num(7), b.nan_to_num(7))


def test_on_another_stream_and_in_a_graph():
    c = Case([200, 90], 1, 64)
    c.check()
    want = [t.clone() for t in (c.y, c.grads[0], c.dh0)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for t in (c.y, c.gbuf, c.dh0):
        t.fill_(3)
    torch.cuda.synchronize()
    c.forward(s)
    c.backward(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (c.y, c.grads[0], c.dh0)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.forward()
        c.backward()
    for _ in range(2):
        for t in (c.y, c.gbuf, c.dh0):
            t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (c.y, c.grads[0], c.dh0)))


def test_one_plan_on_two_streams_at_once():
    # sequences that are cut: their pieces' maps must not be shared between the streams
    a, b = Case([6000, 5000], 2, 64, "f32", "gated", seed=1), Case([6000, 5000], 2, 64, "f32", "gated", seed=2)
    b.plan = a.plan
    want = []
    for c in (a, b):
        c.check()
        want.append([t.clone() for t in (c.y, c.gbuf, c.h_n, c.dh0)])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip((a, b), streams):
            c.forward(s)
            c.backward(s)
    torch.cuda.synchronize()
    for c, w in zip((a, b), want):
        for got, t in zip((c.y, c.gbuf, c.h_n, c.dh0), w):
            assert torch.equal(got.nan_to_num(7), t.nan_to_num(7))


def test_windows_continue_the_recurrence():
    # forward direction: window after window, each from the last one's state, is the whole scan
    lens, H = [150, 20, 333, 0], 56
    c = Case(lens, 1, H, states=True)
    c.forward()
    w = c.want()
    cat = c.plan.unpack(c.v["f"].view(-1, H)), c.plan.unpack(c.v["z"].view(-1, H))
    y = torch.zeros_like(cat[0])
    h = c.h0
    for k in range(0, 333, 100):
        p = ops().Plan(lens, window=(k, 100))
        f, z = (p.pack(t).view(p.rows, 1, H) for t in cat)
        out, h_n = torch.empty_like(f), torch.empty_like(h)
        ops().glr_forward(p, c.shape, f, z, None, h, out, h_n, None)
        p.unpack(out.view(p.rows, H), y)
        h = h_n
    near(c.plan.pack(y).view(-1, 1, H), w["y"], w["~y"], "f32", "windows")
    near(h, w["h_n"], w["~h_n"], "f32", "final state")


@pytest.mark.parametrize("dtype,cell,H", [("f32", "tied", 64), ("bf16", "gated", 40), ("f32", "gated", 33), ("bf16", "tied", 1)])
def test_single_frames_are_the_scan(dtype, cell, H):
    L, rows = 12, 5
    c = Case([L] * rows, 1, H, dtype, cell)
    w = c.want()
    slots = torch.tensor([6, 2, 0, 7, 3], dtype=torch.int32, device="cuda")
    cache = torch.full((9, H), 5.0, device="cuda")
    cache[slots.long()] = c.h0[0]
    y = torch.empty((rows, 1, H), dtype=DT[dtype], device="cuda")
    for t in range(L):      # equal lengths: rows t * rows .. are frame t in caller order
        g = [None if v is None else v[t * rows:(t + 1) * rows] for v in c.gates]
        ops().glr_step(c.shape, *g, cache, cache, y, slots)
        at = slice(t * rows, (t + 1) * rows)
        near(y, w["y"][at], w["~y"][at], dtype, t)
    near(cache[slots.long()][None], w["h_n"], w["~h_n"], "f32", "state")
    assert (cache[torch.tensor([1, 4, 5, 8]).cuda()] == 5).all()


def test_step_idle_rows_and_separate_states():
    H, rows = 40, 6
    c = Case([rows], 1, H)
    g = [None if v is None else v for v in c.gates]
    slots = torch.tensor([-1, 3, 99, 0, 4, -7], dtype=torch.int32, device="cuda")
    before = torch.randn(5, H, device="cuda")
    after = torch.full((5, H), 9.0, device="cuda")
    y = torch.full((rows, 1, H), 9.0, device="cuda")
    ops().glr_step(c.shape, *g, before, after, y, slots)
    torch.cuda.synchronize()
    assert not y[[0, 2, 5]].any() and (after[[1, 2]] == 9).all()
    for r, s in ((1, 3), (3, 0), (4, 4)):
        a = torch.sigmoid(c.v["f"][r, 0].double())
        want = a * before[s].double() + torch.sigmoid(-c.v["f"][r, 0].double()) * c.v["z"][r, 0].double()
        assert (y[r, 0] - want).abs().max() < 1e-5 and torch.equal(y[r, 0], after[s])
    ops().glr_step(c.shape, *[None if v is None else v[:0] for v in g], before, after, y[:0], slots[:0])


def test_offsets_beyond_32_bits():
    # row stride 2^26 elements: the last rows of gates and gradients lie past 2^31 elements
    o, H, rows, ld = ops(), 16, 36, 1 << 26
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    c = Case([rows], 1, H, "bf16", "tied")
    g = buf.view(rows, 1, ld)
    f, z, df, dz = (g[:, :, k * H:(k + 1) * H] for k in range(4))
    f.copy_(c.v["f"])
    z.copy_(c.v["z"])
    o.glr_forward(c.plan, c.shape, f, z, None, c.h0, c.y, c.h_n, c.ws)
    o.glr_backward(c.plan, c.shape, f, z, None, c.ws, c.v["dy"], c.dh_n, df, dz, None, c.dh0)
    w = c.want()
    near(c.y, w["y"], w["~y"], "bf16", "y")
    near(df, w["df"], w["~df"], "bf16", "df")
    near(dz, w["dz"], w["~dz"], "bf16", "dz")
    near(c.dh0, w["dh0"], w["~dh0"], "f32", "dh0")


def test_gradient_against_differences():
    # the 64-bit loss along a random direction, against the kernel's gradients
    c = Case([40, 9, 100], 2, 12, "f32", "gated")
    c.forward()
    c.backward()
    rng = np.random.default_rng(1)
    num = {k: t.double().cpu().numpy() for k, t in c.v.items()}
    h0, dh_n = (t.double().cpu().numpy() for t in (c.h0, c.dh_n))
    way = {k: rng.normal(size=num[k].shape) for k in ("f", "z", "i")}
    wh = rng.normal(size=h0.shape)

    def loss(e):
        o = ref.glr(c.lens, *(num[k] + e * way[k] for k in ("f", "z", "i")), h0 + e * wh)
        return (o["y"] * num["dy"]).sum() + (o["h_n"] * dh_n).sum()

    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    got = sum((g.double().cpu().numpy() * way[k]).sum() for g, k in zip(c.grads, ("f", "z", "i")))
    got += (c.dh0.double().cpu().numpy() * wh).sum()
    size = sum(np.abs(g.double().cpu().numpy() * way[k]).sum() for g, k in zip(c.grads, ("f", "z", "i")))
    assert abs(slope - got) < 64 * ref.U * size + 1e-8 * abs(slope)


def test_refusals():
    o, c = ops(), Case([6, 3], 2, 16)
    f, z, _ = c.gates
    args = dict(plan=c.plan, shape=c.shape, f=f, z=z, i=None, h0=c.h0, y=c.y, h_n=c.h_n, workspace=c.ws)
    for kw in (dict(i=z), dict(f=f.float().double()), dict(z=z[:-1]), dict(f=f.contiguous()), dict(y=c.y[:, :1]), dict(h0=c.h0[:1]),
               dict(h_n=c.h_n.half()), dict(workspace=c.ws[:-1]), dict(shape=o.glr_shape(16, 2, True)),
               dict(shape=o.glr_shape(16, 2, False, "gated"))):
        with pytest.raises(ValueError):
            o.glr_forward(**{**args, **kw})
    from padding_free_variable_gb300._lib import LSTMError
    with pytest.raises(LSTMError):
        o.glr_backward(c.plan, c.shape, f, z, None, None, c.v["dy"], None, *c.grads, None)
    with pytest.raises(ValueError):
        o.glr_shape(16, 1, False, "other")
    with pytest.raises(LSTMError):        # the state cache is shorter than the rows
        o.glr_step(o.glr_shape(16, 1, False), f[:, :1], z[:, :1], None, c.h0[0], c.h0[0], c.y[:, :1].contiguous())
