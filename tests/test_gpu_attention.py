"""Linear attention with a decay for each head on the GPU against its 64-bit restatement, value by value within derived
bounds (attention_reference): forward, backward, single frames, over lengths, head sizes, strides, plans and decays where it
can go wrong."""
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
    """|got - want| within the bound (and a rounding to bf16)."""
    got, want, bound = got.double().cpu().numpy(), np.asarray(want), np.asarray(bound)
    if dtype == "bf16":
        bound = bound + ref.BF16 * (np.abs(want) + bound)
    bad = ~(np.abs(got - want) <= bound + 1e-36)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], bound[bad][:4])


class Case:
    def __init__(self, lens, nd, H, dk, dv, dtype="f32", padded=False, states=True, seed=0, layout="blocks", shift=0, decays=None,
                 plan=None):
        o = ops()
        self.lens, self.nd, self.H, self.dk, self.dv, self.dtype, self.padded = list(lens), nd, H, dk, dv, dtype, padded
        self.plan = plan or o.Plan(lens, padded=padded)
        self.scale = 0.3
        self.shape = o.la_shape(H, dk, dv, nd, dtype == "bf16", self.scale)
        rng = np.random.default_rng(seed + 977 * dk + 31 * dv + len(self.lens))
        n, B, dt = self.plan.rows, self.plan.batch, DT[dtype]
        self.v = {m: torch.from_numpy(rng.normal(size=(n, nd, H, w)) * s).to("cuda", dt)
                  for m, w, s in (("q", dk, 1.0), ("k", dk, dk ** -0.5), ("v", dv, 1.0), ("dy", dv, 1.0))}
        st = rng.normal(size=(2, nd, B, H, dk, dv)) * 0.8
        self.s0, self.ds_n = [torch.from_numpy(s).float().cuda() if states else None for s in st]
        ld = np.log(rng.uniform(0.2, 1.0, size=(nd, H)) ** 0.3) if decays is None else np.resize(np.array(decays), (nd, H))
        self.ld = torch.from_numpy(ld).float().cuda()
        # q, k, v as a user's projection holds them: blocks of a row, head by head, or planes of their own
        w = 2 * dk + dv
        e = n * nd * H * w + shift + 64
        self.buf, self.gbuf = [torch.full((e,), float("nan"), dtype=dt, device="cuda") for _ in range(2)]

        def views(b):
            b = b[shift:shift + n * nd * H * w]
            if layout == "blocks":
                t, c = b.view(n, nd * H * w), nd * H * dk
                return [t[:, :c].unflatten(1, (nd, H, dk)), t[:, c:2 * c].unflatten(1, (nd, H, dk)), t[:, 2 * c:].unflatten(1, (nd, H, dv))]
            if layout == "heads":
                t = b.view(n, nd, H, w)
                return [t[..., :dk], t[..., dk:2 * dk], t[..., 2 * dk:]]
            t = b.view(nd, H, n, w)
            return [x.permute(2, 0, 1, 3) for x in (t[..., dv:dv + dk], t[..., dv + dk:], t[..., :dv])]

        self.x, self.g = views(self.buf), views(self.gbuf)
        for t, m in zip(self.x, "qkv"):
            t.copy_(self.v[m])
        f32 = lambda: torch.full((nd, B, H, dk, dv), float("nan"), device="cuda")  # noqa: E731
        self.y = torch.full((n, nd, H, dv), float("nan"), dtype=dt, device="cuda")
        self.s_n, self.ds0 = f32(), f32()

    def forward(self, **kw):
        ops().la_forward(self.plan, self.shape, *self.x, self.ld, self.s0, self.y, self.s_n, **kw)

    def backward(self, **kw):
        ops().la_backward(self.plan, self.shape, *self.x, self.ld, self.s0, self.v["dy"], self.ds_n, *self.g, self.ds0, **kw)

    def want(self):
        num = {m: t.double().cpu().numpy() for m, t in self.v.items()}
        st = [None if t is None else t.double().cpu().numpy() for t in (self.s0, self.ds_n)]
        return ref.attend(self.lens, num["q"], num["k"], num["v"], self.ld.double().cpu().numpy(), np.float32(self.scale), st[0],
                          num["dy"], st[1], self.padded, self.dtype == "bf16")

    def compare(self, w):
        near(self.y, w["y"], w["~y"], self.dtype, "y")
        near(self.s_n, w["s_n"], w["~s_n"], "f32", "s_n")
        for t, m in zip(self.g, ("dq", "dk", "dv")):
            near(t, w[m], w["~" + m], self.dtype, m)
        near(self.ds0, w["ds0"], w["~ds0"], "f32", "ds0")

    def check(self, **kw):
        self.forward(**kw)
        self.backward(**kw)
        torch.cuda.synchronize()
        w = self.want()
        self.compare(w)
        assert self.plan.poll() == 0
        return w


MANY = [int(v) for v in np.random.default_rng(8).integers(0, 90, 300)]
CASES = [
    # lengths, directions, heads, key, value, dtype, padded, layout, shift (elements off the buffer's start)
    ([1], 1, 1, 1, 1, "f32", False, "blocks", 0),
    ([1], 2, 2, 8, 8, "bf16", False, "blocks", 0),
    ([0, 0, 0], 2, 2, 16, 8, "f32", False, "blocks", 0),
    ([2, 0, 1], 1, 3, 7, 5, "f32", False, "heads", 1),
    ([5, 40, 39, 1, 2, 3, 4, 30], 1, 2, 16, 16, "f32", False, "blocks", 0),
    ([63, 64, 65, 0, 1, 127, 128, 129], 2, 2, 32, 64, "f32", False, "planes", 0),
    ([63, 64, 65, 0, 1, 127, 128, 129], 2, 2, 64, 64, "bf16", False, "blocks", 0),
    ([63, 64, 65, 0, 1, 127, 128, 129], 1, 2, 64, 64, "bf16", False, "heads", 8),
    ([255, 256, 257, 3], 1, 3, 128, 128, "bf16", False, "blocks", 0),
    ([200, 130], 2, 1, 128, 64, "bf16", False, "planes", 0),
    ([200, 130], 2, 1, 64, 128, "bf16", False, "blocks", 0),
    ([200, 130, 0], 1, 2, 24, 104, "bf16", False, "blocks", 0),
    ([200, 130, 0], 1, 2, 72, 8, "bf16", False, "heads", 16),
    ([200, 130], 1, 2, 64, 64, "bf16", False, "blocks", 3),
    ([200, 13], 2, 2, 20, 12, "bf16", False, "blocks", 0),
    ([200, 13], 2, 2, 37, 53, "bf16", False, "blocks", 0),
    ([300, 7, 191, 192, 193], 2, 3, 37, 53, "f32", False, "blocks", 0),
    ([257, 8], 1, 2, 128, 128, "f32", False, "planes", 1),
    ([1500], 1, 2, 64, 64, "bf16", False, "blocks", 0),
    ([2500, 2499, 1], 1, 1, 128, 128, "bf16", False, "blocks", 0),
    ([1033, 1], 2, 2, 32, 32, "f32", False, "blocks", 0),
    ([4100], 2, 1, 16, 24, "f32", False, "blocks", 0),
    (MANY, 2, 2, 8, 12, "f32", False, "blocks", 0),
    (MANY, 1, 2, 32, 16, "bf16", False, "blocks", 0),
    ([5, 0, 17, 70, 3], 2, 2, 16, 16, "f32", True, "blocks", 0),
    ([5, 0, 17, 170, 3], 2, 2, 64, 32, "bf16", True, "heads", 0),
    ([5, 0, 17, 170, 3], 1, 2, 9, 11, "bf16", True, "planes", 0),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{i}-nd{c[1]}-{c[2]}x{c[3]}x{c[4]}-{c[5]}{'-padded' if c[6] else ''}" for i, c in enumerate(CASES)])
def test_matches_definition(case):
    lens, nd, H, dk, dv, dtype, padded, layout, shift = case
    Case(lens, nd, H, dk, dv, dtype, padded, layout=layout, shift=shift).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [24, 64, 128])
def test_without_states(dtype, size):
    c = Case([70, 300, 0, 129], 2, 2, size, size, dtype, states=False)
    w = c.check()
    y, s_n = c.y.clone(), c.s_n.clone()
    c.s_n = None
    c.forward()
    keep, c.ds0 = c.ds0, None
    c.backward()
    torch.cuda.synchronize()
    assert torch.equal(c.y, y)
    c.s_n, c.ds0 = s_n, keep
    c.compare(w)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays_from_none_to_all(dtype):
    # no decay at all, one that is read as none, none of the past left, subnormal and far powers
    decays = [0.0, 0.5, float("-inf"), -300.0, -90.0, -1e-7, -0.7, -12.0]
    Case([190, 64, 1, 700], 2, 8, 64, 64, dtype, decays=decays, seed=3).check()


@pytest.mark.parametrize("dtype,size", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_cut_sequences_agree_with_uncut(dtype, size):
    # few long sequences are cut into pieces; without a scratch they are not: the C call with no scratch
    from padding_free_variable_gb300 import _lib
    c = Case([5000, 1, 3333], 2, 1, size, size, dtype, seed=1, decays=[-0.002, -0.05])
    o = ops()
    assert o.la_scratch_bytes(c.plan, c.shape) > 0
    w = c.check()
    for t in (c.y, c.s_n, c.ds0, c.gbuf):
        t.fill_(float("nan"))
    key, dev = c.shape.key, 0
    three = o._la_three(key, *c.x, c.plan.rows, o._LA_IN, dev)
    grads = o._la_three(key, *c.g, c.plan.rows, o._LA_GRADS, dev)
    lib, s = _lib.load(), torch.cuda.current_stream().cuda_stream
    p = lambda t: t.data_ptr()  # noqa: E731
    assert lib.lstm_la_fwd(c.plan.handle, c.shape.ref, three, p(c.ld), p(c.s0), p(c.y), p(c.s_n), None, s) == 0
    assert lib.lstm_la_bwd(c.plan.handle, c.shape.ref, three, p(c.ld), p(c.s0), p(c.v["dy"]), p(c.ds_n), grads, p(c.ds0), None, s) == 0
    torch.cuda.synchronize()
    c.compare(w)


@pytest.mark.parametrize("lens", [[300, 40], [6000]], ids=["whole", "cut"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_states_carried_in_place(lens, dtype):
    c = Case(lens, 1, 2, 64, 64, dtype, seed=2)
    w = c.check()
    c.s_n, c.ds0 = c.s0.clone(), c.ds_n.clone()
    s0, ds_n = c.s0, c.ds_n
    c.s0, keep = c.s_n, c.s_n
    c.forward()
    c.s0, c.ds_n = s0, c.ds0
    c.backward()
    torch.cuda.synchronize()
    assert c.s_n is keep
    c.ds_n = ds_n
    c.compare(w)


def test_two_halves_carry_their_state():
    # frames 0..99 and 100..249 of one sequence as two calls
    a = Case([250], 1, 2, 64, 64, "f32", seed=4)
    a.forward()
    o, mid = ops(), torch.empty_like(a.s0)
    y, end = torch.empty_like(a.y), torch.empty_like(a.s0)
    for lo, hi, s, t in ((0, 100, a.s0, mid), (100, 250, mid, end)):
        o.la_forward(o.Plan([hi - lo]), a.shape, *[x[lo:hi] for x in a.x], a.ld, s, y[lo:hi], t)
    torch.cuda.synchronize()
    w = a.want()
    near(y, w["y"], w["~y"], "f32", "y")
    near(end, w["s_n"], w["~s_n"], "f32", "s_n")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_segments_and_windows(dtype):
    o = ops()
    lens = [300, 130, 1, 0]
    seg = [m for n in lens for m in ([min(128, n - s) for s in range(0, max(n - 64, 1), 64)] if n else [0])]
    plan = o.Plan(lens, segments=(128, 64))
    assert sorted(plan.lengths.tolist()) == sorted(lens) and plan.rows == sum(seg)
    Case(seg, 2, 2, 64, 32, dtype, plan=plan).check()
    plan = o.Plan(lens, window=(100, 150))
    Case([max(0, min(n - 100, 150)) for n in lens], 1, 2, 32, 64, dtype, plan=plan).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_inputs_shared_by_heads(dtype):
    # one key and value for all heads: read through a stride of zero, a gradient for each head
    c = Case([150, 20], 1, 4, 64, 64, dtype)
    for m in (1, 2):
        c.x[m] = c.x[m][:, :, :1].contiguous().expand(-1, -1, 4, -1)
        c.v["qkv"[m]] = c.x[m].contiguous()
    c.check()
    c.g[1] = c.g[1][:, :, :1].expand(-1, -1, 4, -1)
    from padding_free_variable_gb300._lib import LSTMError
    with pytest.raises(LSTMError):
        c.backward()


@pytest.mark.parametrize("dtype,size", [("f32", 40), ("bf16", 64), ("bf16", 128)])
def test_repeats_bitwise_and_leaves_neighbours(dtype, size):
    c = Case([400, 70, 1], 2, 2, size, size, dtype, layout="heads", shift=8)
    first = None
    for _ in range(3):
        for t in (c.y, c.s_n, c.ds0, c.gbuf):
            t.fill_(7.0)
        c.forward()
        c.backward()
        torch.cuda.synchronize()
        now = [t.clone() for t in (c.y, c.s_n, c.ds0, c.gbuf)]
        if first:
            assert all(torch.equal(x, y) for x, y in zip(first, now))
        first = now
    assert (c.gbuf[:8] == 7).all() and (c.gbuf[-56:] == 7).all()


@pytest.mark.parametrize("dtype,size", [("f32", 24), ("bf16", 64), ("bf16", 128)])
def test_infinities_stay_in_their_head_and_sequence(dtype, size):
    c = Case([300, 200, 129], 1, 3, size, size, dtype, seed=6)
    rows = ref.packed_rows(c.lens)[0]
    for m, bad in ((0, float("nan")), (1, float("inf")), (2, float("-inf"))):
        c.x[m][int(rows[1][77]), 0, 1, 3] = bad
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    w = c.want()
    mine = np.zeros((c.plan.rows, 1, c.H), bool)
    mine[rows[1], 0, 1] = True
    keep = torch.from_numpy(~mine).cuda()
    near(c.y[keep], w["y"][~mine], w["~y"][~mine], dtype, "y")
    for t, m in zip(c.g, ("dq", "dk", "dv")):
        near(t[keep], w[m][~mine], w["~" + m][~mine], dtype, m)
    assert not torch.isfinite(c.y[int(rows[1][77]), 0, 1]).all()


@pytest.mark.parametrize("dtype,size,lens", [("f32", 32, [200, 3]), ("bf16", 64, [200, 3]), ("bf16", 64, [5000])])
def test_streams_and_graphs(dtype, size, lens):
    c = Case(lens, 2, 1, size, size, dtype)
    w = c.check()
    side = torch.cuda.Stream()
    for t in (c.y, c.s_n, c.ds0, c.gbuf):
        t.fill_(float("nan"))
    torch.cuda.synchronize()
    c.forward(stream=side)
    c.backward(stream=side)
    side.synchronize()
    c.compare(w)
    # captured, replayed on new inputs; two graphs on two streams at once
    d = Case(lens, 2, 1, size, size, dtype, seed=9, plan=c.plan)
    graphs = []
    for x in (c, d):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.forward()
            x.backward()
        graphs.append(g)
    for x in (c, d):
        for t in (x.y, x.s_n, x.ds0, x.gbuf):
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    c.compare(w)
    d.compare(d.want())


def test_a_wait_that_runs_out_leaves_the_device_usable():
    # a limit that a product may or may not meet: either way the call ends, and the next one is right
    c = Case([400, 70, 1], 2, 2, 64, 64, "bf16", seed=8)
    c.plan.set_wait_limit(1)
    c.forward()
    c.backward()
    assert c.plan.poll() in (0, 4)
    c.plan.set_wait_limit(2000000000)
    c.check()


# ------------------------------------------------------------------ single frames

STEPS = [(1, 1, 1, 1, "f32"), (3, 2, 16, 8, "f32"), (9, 3, 37, 53, "f32"), (9, 3, 37, 53, "bf16"), (40, 8, 64, 64, "bf16"),
         (40, 2, 128, 128, "f32"), (5, 2, 128, 20, "bf16"), (7, 1, 3, 128, "f32"), (300, 4, 8, 8, "bf16")]


@pytest.mark.parametrize("rows,H,dk,dv,dtype", STEPS)
@pytest.mark.parametrize("in_place", [False, True])
def test_single_frames(rows, H, dk, dv, dtype, in_place):
    o, rng = ops(), np.random.default_rng(rows + dk)
    slots = rows + 5
    new = lambda *s: torch.from_numpy(rng.normal(size=s))  # noqa: E731
    pre = new(rows, 1, H, 2 * dk + dv).to("cuda", DT[dtype])
    q, k, v = pre[..., :dk], pre[..., dk:2 * dk], pre[..., 2 * dk:]
    ld = torch.from_numpy(np.log(rng.uniform(0.1, 1, size=(1, H)))).float().cuda()
    state = new(slots, H, dk, dv).float().cuda()
    at = torch.from_numpy(rng.permutation(slots)[:rows].astype(np.int32)).cuda()
    idle = np.arange(rows) % 4 == 3
    at[torch.from_numpy(idle).cuda()] = torch.tensor([-1, slots, 2 ** 31 - 1], dtype=torch.int32).repeat(rows)[:int(idle.sum())].cuda()
    shape = o.la_shape(H, dk, dv, 1, dtype == "bf16", 0.4)
    out = state.clone() if in_place else torch.full_like(state, 5.0)
    y = torch.full((rows, 1, H, dv), float("nan"), dtype=DT[dtype], device="cuda")
    o.la_step(shape, q, k, v, ld, out if in_place else state, out, y, at)
    torch.cuda.synchronize()
    num = lambda t: t.double().cpu().numpy()  # noqa: E731
    live, where = ~idle, at.cpu().numpy()[~idle]
    w = ref.attend([1] * int(live.sum()), num(q)[live], num(k)[live], num(v)[live], num(ld), np.float32(0.4), num(state)[where][None])
    near(y[torch.from_numpy(live).cuda()], w["y"], w["~y"], dtype, "y")
    assert not y[torch.from_numpy(idle).cuda()].any()
    near(out[torch.from_numpy(where).long().cuda()], w["s_n"][0], w["~s_n"][0], "f32", "state")
    rest = np.setdiff1d(np.arange(slots), where)
    assert torch.equal(out[rest], state[rest] if in_place else torch.full_like(state[rest], 5.0))


def test_single_frames_follow_the_scan():
    c = Case([70, 33, 70], 1, 2, 64, 64, "f32", seed=12)
    c.forward()
    rows = ref.packed_rows(c.lens)[0]
    o, cache = ops(), c.s0[0].clone()
    y = torch.empty_like(c.y)
    for t in range(70):
        on = [b for b in range(3) if t < c.lens[b]]
        r = torch.tensor([int(rows[b][t]) for b in on], device="cuda")
        out = torch.empty(len(on), 1, 2, 64, device="cuda")
        o.la_step(c.shape, *[x[r] for x in c.x], c.ld, cache, cache, out, torch.tensor(on, dtype=torch.int32, device="cuda"))
        y[r] = out
    torch.cuda.synchronize()
    w = c.want()
    near(y, w["y"], w["~y"], "f32", "y")
    near(cache, w["s_n"][0], w["~s_n"][0], "f32", "state")


def test_single_frames_captured():
    o = ops()
    shape = o.la_shape(2, 64, 64)
    q, k, v = (torch.randn(6, 1, 2, 64, device="cuda") for _ in range(3))
    ld = torch.full((1, 2), -0.1, device="cuda")
    cache, y = torch.randn(6, 2, 64, 64, device="cuda"), torch.empty(6, 1, 2, 64, device="cuda")
    want = cache.double()
    o.la_step(shape, q, k, v, ld, cache.clone(), cache.clone(), y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o.la_step(shape, q, k, v, ld, cache, cache, y)
    for _ in range(5):
        g.replay()
        want = np.exp(float(ld[0, 0])) * want + k[:, 0, :, :, None].double() * v[:, 0, :, None].double()
    torch.cuda.synchronize()
    assert (cache.double() - want).abs().max() < 40 * 2.0 ** -24 * want.abs().max()


def test_states_past_32_bits():
    # a cache of 2.4e9 values: its last slots lie beyond what 32 bits count
    o, slots = ops(), 73000
    shape = o.la_shape(2, 128, 128, scale=0.5)
    q, k, v = (torch.randn(3, 1, 2, 128, device="cuda") for _ in range(3))
    ld = torch.full((1, 2), -0.3, device="cuda")
    cache = torch.empty(slots, 2, 128, 128, device="cuda")
    at = torch.tensor([slots - 1, 65537, 0], dtype=torch.int32, device="cuda")
    state = torch.randn(3, 2, 128, 128, device="cuda")
    cache[at.long()] = state
    y = torch.empty(3, 1, 2, 128, device="cuda")
    o.la_step(shape, q, k, v, ld, cache, cache, y, at)
    num = lambda t: t.double().cpu().numpy()  # noqa: E731
    w = ref.attend([1] * 3, num(q), num(k), num(v), num(ld), np.float32(0.5), num(state)[None])
    near(y, w["y"], w["~y"], "f32", "y")
    near(cache[at.long()], w["s_n"][0], w["~s_n"][0], "f32", "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_past_32_bits(dtype):
    # rows 2^28 + 64 values apart: the last one starts beyond 2^31 values
    c = Case([6, 3, 1], 1, 1, 64, 64, dtype, seed=5)
    step = 2 ** 28 + 64
    buf = torch.empty(9 * step + 512, dtype=DT[dtype], device="cuda")
    wide = [buf.as_strided((10, 1, 1, 64), (step, 64, 64, 1), 64 * m) for m in range(6)]
    for m in range(3):
        wide[m].copy_(c.x[m])
    c.x, c.g = wide[:3], wide[3:]
    c.check()


def test_no_frames_and_bad_arguments():
    o = ops()
    from padding_free_variable_gb300._lib import LSTMError
    c = Case([0, 0], 1, 2, 16, 16)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    assert torch.equal(c.s_n, c.s0) and torch.equal(c.ds0, c.ds_n)
    c.s0 = c.ds_n = None
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    assert not c.s_n.any() and not c.ds0.any()
    c = Case([9, 4], 1, 2, 16, 16)
    q, k, v = c.x
    for args in ((q[:5], k, v), (q, k.double(), v), (q, k, v[..., :8]), (q.transpose(2, 3).contiguous().transpose(2, 3), k, v)):
        with pytest.raises(ValueError):
            o.la_forward(c.plan, c.shape, *args, c.ld, c.s0, c.y, c.s_n)
    with pytest.raises(ValueError):
        o.la_forward(c.plan, c.shape, q, k, v, c.ld[0], c.s0, c.y, c.s_n)
    with pytest.raises(ValueError):
        o.la_forward(c.plan, c.shape, q, k, v, c.ld, c.s0, c.y[:, :, :1], c.s_n)
    flat = torch.zeros(c.s0.numel() + 4, device="cuda")
    a, b = flat[:c.s0.numel()].view_as(c.s0), flat[4:].view_as(c.s0)
    with pytest.raises(LSTMError):
        o.la_forward(c.plan, c.shape, q, k, v, c.ld, a, c.y, b)
    with pytest.raises(LSTMError):
        o.la_forward(c.plan, c.shape, q, k, v, None, c.s0, c.y, c.s_n)
    for bad in (o.la_shape(2, 129, 16), o.la_shape(2, 16, 0), o.la_shape(2, 16, 16, 3), o.la_shape(2, 16, 16, scale=float("nan"))):
        assert o.la_scratch_bytes(c.plan, bad) == 0
        x, w = [torch.zeros(13, bad.num_directions, 2, m, device="cuda") for m in (bad.key_size, bad.value_size)], bad.num_directions
        with pytest.raises(LSTMError):
            o.la_forward(c.plan, bad, x[0], x[0], x[1], torch.zeros(w, 2, device="cuda"), None, x[1], None)
    assert c.plan.poll() == 0
