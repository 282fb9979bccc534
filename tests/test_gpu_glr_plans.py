"""The gated linear recurrence on the plans of RETURNN-style segments and of truncated windows, whose units are pieces of the
caller's sequences, against the 64-bit restatement of each piece alone; and gates that stay near 1 for long."""
import numpy as np
import pytest

import operator_reference as ref
from test_gpu_glr import DT, Case, near, ops

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from padding_free_variable_gb300 import build
    build.build()


def pieces(lens, chunk, step):
    """(sequence, first frame, frames) of every segment."""
    out = []
    for b, L in enumerate(lens):
        s = 0
        while True:
            out.append((b, s, max(0, min(chunk, L - s))))
            if s + chunk >= L:
                break
            s += step
    return out


@pytest.mark.parametrize("lens,chunk,step,nd,H,dtype,cell", [
    ([150, 20, 333, 0], 100, 50, 2, 40, "f32", "gated"), ([150, 20, 333, 0], 64, 64, 1, 24, "bf16", "tied"),
    ([5000, 300], 2000, 1500, 2, 64, "f32", "tied"), ([70, 3], 16, 8, 2, 33, "f32", "gated")])
def test_segments(lens, chunk, step, nd, H, dtype, cell):
    o = ops()
    plan = o.Plan(lens, segments=(chunk, step))
    units = pieces(lens, chunk, step)
    assert plan.batch == len(units) and plan.rows == sum(u[2] for u in units)
    shape = o.glr_shape(H, nd, dtype == "bf16", cell)
    rng = np.random.default_rng(H)
    gated = cell == "gated"
    # the caller's frame of every packed row, from the plan; the restatement packs the same pieces itself
    frame = plan.pack(torch.arange(sum(lens), dtype=torch.float32, device="cuda")[:, None].repeat(1, 4))[:, 0].long()
    rows_of, _ = ref.packed_rows([u[2] for u in units])
    starts = np.concatenate([[0], np.cumsum(lens)])
    for (b, s, n), rows in zip(units, rows_of):
        assert np.array_equal(frame.cpu().numpy()[rows], starts[b] + s + np.arange(n))
    v = {k: torch.from_numpy(rng.normal(1.0 if k == "f" else 0.0, 1, (sum(lens), nd, H))).to("cuda", DT[dtype])[frame] for k in "fzid"}
    st = lambda: torch.from_numpy(rng.normal(size=(nd, len(units), H))).float().cuda()  # noqa: E731
    h0, dh_n = st(), st()
    h_n, dh0, y = torch.empty_like(h0), torch.empty_like(h0), torch.empty_like(v["f"])
    df, dz, di = torch.empty_like(y), torch.empty_like(y), torch.empty_like(y) if gated else None
    ws = torch.empty(o.glr_workspace_bytes(plan, shape), dtype=torch.uint8, device="cuda")
    i = v["i"] if gated else None
    o.glr_forward(plan, shape, v["f"], v["z"], i, h0, y, h_n, ws)
    o.glr_backward(plan, shape, v["f"], v["z"], i, ws, v["d"], dh_n, df, dz, di, dh0)
    num = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    w = ref.glr([u[2] for u in units], num(v["f"]), num(v["z"]), num(i), num(h0), num(v["d"]), num(dh_n))
    for got, name, dt in ((y, "y", dtype), (h_n, "h_n", "f32"), (df, "df", dtype), (dz, "dz", dtype), (di, "di", dtype), (dh0, "dh0", "f32")):
        if got is not None:
            near(got, w[name], w["~" + name], dt, name)


def test_window_gradients():
    # a window's plan, both directions: its pieces alone
    lens, nd, H, start, width = [150, 20, 333, 120], 2, 40, 100, 100
    o = ops()
    plan = o.Plan(lens, window=(start, width))
    n = [max(0, min(width, L - start)) for L in lens]
    assert plan.rows == sum(n) and plan.batch == len(lens)
    c = Case(n, nd, H, "f32", "gated")
    c.plan = plan
    c.check()


def test_long_memories():
    # 20 000 frames of gates near 1: roundings do not drift beyond their bounds
    for bias in (6.0, 9.0, 12.0):
        Case([20000, 257], 1, 8, "f32", "tied", bias=bias, seed=7).check()


@pytest.mark.parametrize("cell", ["tied", "gated"])
def test_gates_errors_average_out(cell):
    # h = a h0 with h0 = 1: the gate itself.  A product of n gates drifts by n times their mean error; held to half a rounding
    # (2^-25 of the value) over every range of gates above 1/2, a million of each
    o, H, B = ops(), 65536, 16
    plan, shape = o.Plan([1] * B), o.glr_shape(H, 1, False, cell)
    h0, zero = torch.ones(1, B, H, device="cuda"), torch.zeros(B, 1, H, device="cuda")
    y = torch.empty_like(zero)
    for lo, hi in ((0, 1), (1, 2), (2, 4), (4, 8), (8, 12), (12, 16)):
        f = torch.rand(B, 1, H, generator=torch.Generator(device="cuda").manual_seed(lo), device="cuda") * (hi - lo) + lo
        o.glr_forward(plan, shape, f, zero, zero if cell == "gated" else None, h0, y, None, None)
        off = y.double() / torch.sigmoid(f.double()) - 1
        assert abs(float(off.mean())) < 2.0 ** -25 and float(off.abs().max()) < 16 * ref.U
