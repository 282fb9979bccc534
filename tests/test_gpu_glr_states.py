"""A state carried in place through the gated linear recurrence (h_n over h0, dh0 over dh_n): the same bits as with arrays of
their own, whether sequences are cut into pieces or not; arrays that overlap otherwise are refused."""
import pytest

from test_gpu_glr import Case, ops

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from padding_free_variable_gb300 import build
    build.build()


CASES = [
    # cut: 16-byte rows, rows of 4 and of 2 bytes' alignment, narrow layers
    ([6000, 5000], 2, 64, "f32", "gated", 0), ([9000, 0, 3], 1, 64, "bf16", "tied", 0), ([4100, 300], 2, 33, "f32", "tied", 0),
    ([5000, 40], 1, 130, "bf16", "gated", 1), ([7000, 255], 2, 16, "f32", "gated", 0),
    # uncut, and a warp a sequence
    ([63, 64, 65, 0, 1, 129], 2, 40, "f32", "tied", 0), ([70, 0, 300], 1, 24, "bf16", "gated", 0),
    ([16, 3, 0, 9, 1, 8], 2, 7, "bf16", "gated", 1), ([0, 0], 1, 8, "f32", "tied", 0),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{i}-H{c[2]}-{c[3]}" for i, c in enumerate(CASES)])
def test_states_in_place(case):
    lens, nd, H, dtype, cell, shift = case
    c = Case(lens, nd, H, dtype, cell, shift=shift)
    c.forward()
    c.backward()
    want = [t.clone() for t in (c.y, c.gbuf, c.h_n, c.dh0)]
    c.y.fill_(3)
    c.gbuf.fill_(float("nan"))
    c.h_n, c.dh0 = c.h0, c.dh_n
    c.forward()
    c.backward()
    for got, t in zip((c.y, c.gbuf, c.h0, c.dh_n), want):
        assert torch.equal(got.nan_to_num(7), t.nan_to_num(7))


def test_more_pieces_than_run_at_once():
    o, L, H = ops(), 60000, 512
    plan, shape = o.Plan([L]), o.glr_shape(H, 1, False)
    g = torch.Generator(device="cuda").manual_seed(5)
    t = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    f, z, dy, h0, dh_n = t(L, 1, H) + 2, t(L, 1, H), t(L, 1, H), t(1, 1, H), t(1, 1, H)
    ws = torch.empty(o.glr_workspace_bytes(plan, shape), dtype=torch.uint8, device="cuda")

    def both(h_in, h_out, e_in, e_out):
        y, df, dz = torch.empty_like(f), torch.empty_like(f), torch.empty_like(f)
        o.glr_forward(plan, shape, f, z, None, h_in, y, h_out, ws)
        o.glr_backward(plan, shape, f, z, None, ws, dy, e_in, df, dz, None, e_out)
        return y, df, dz, h_out, e_out

    want = both(h0, torch.empty_like(h0), dh_n, torch.empty_like(h0))
    for _ in range(5):
        h, e = h0.clone(), dh_n.clone()
        assert all(torch.equal(a, b) for a, b in zip(both(h, h, e, e), want))


def test_overlapping_states_are_refused():
    from padding_free_variable_gb300._lib import LSTMError
    for lens in ([600, 20], [0, 0]):
        c = Case(lens, 1, 16)
        n = c.h0.numel()
        buf = torch.zeros(2 * n, device="cuda")
        low, near, apart = (buf[k:k + n].view(c.h0.shape) for k in (0, 4, n))
        for a, b in ((low, near), (near, low)):
            c.h0, c.h_n = a, b
            with pytest.raises(LSTMError):
                c.forward()
            c.dh_n, c.dh0 = a, b
            with pytest.raises(LSTMError):
                c.backward()
        c.h0, c.h_n, c.dh_n, c.dh0 = low, apart, low, apart
        c.forward()
        c.backward()
    c = Case([5], 1, 16)
    cache = torch.zeros(7, 16, device="cuda")
    f, z, _ = c.gates
    with pytest.raises(LSTMError):
        ops().glr_step(c.shape, f, z, None, cache[:5], cache[1:6], c.y)
    ops().glr_step(c.shape, f, z, None, cache[:5], cache[:5], c.y)
