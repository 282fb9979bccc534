"""Scratch of the gated linear recurrence's calls on sequences that are cut into pieces: a caller's own, one for each stream,
and one for each call that a graph captures."""
import pytest

from test_gpu_glr import Case, ops

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
LENS = [6000, 5000]


@pytest.fixture(scope="module", autouse=True)
def _needs_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from padding_free_variable_gb300 import build
    build.build()


def kept(plan):
    return [v for v in plan.scratch.values() if isinstance(v, torch.Tensor)]


def outs(c):
    return c.y, c.gbuf, c.h_n, c.dh0


def capture(c):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.forward()
        c.backward()
    return g


def test_two_graphs_of_one_plan_replayed_at_once():
    a, b = Case(LENS, 2, 64, "f32", "gated", seed=1), Case(LENS, 2, 64, "f32", "gated", seed=2)
    b.plan = a.plan
    graphs = [capture(c) for c in (a, b)]
    assert not kept(a.plan)         # else a later capture would be given the same one
    want = []
    for c in (a, b):
        c.check()
        want.append([t.clone() for t in outs(c)])
        for t in outs(c):
            t.fill_(float("nan"))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, w in zip((a, b), want):
        for got, t in zip(outs(c), w):
            assert torch.equal(got.nan_to_num(7), t.nan_to_num(7))


def test_a_captured_call_on_a_stream_beside_the_current_one():
    c = Case(LENS, 1, 64)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.wait_stream(torch.cuda.current_stream())
        c.forward(s)
        c.backward(s)
        torch.cuda.current_stream().wait_stream(s)
    assert not kept(c.plan)
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in outs(c)]
    c.check()
    assert all(torch.equal(x.nan_to_num(7), y.nan_to_num(7)) for x, y in zip(got, outs(c)))


def test_a_scratch_of_the_callers():
    o, c = ops(), Case(LENS, 1, 64, "bf16")
    need = o.glr_scratch_bytes(c.plan, c.shape)
    assert need > 0 and o.glr_scratch_bytes(Case([200, 90], 1, 64).plan, c.shape) == 0
    mine = torch.full((need + 64,), 85, dtype=torch.uint8, device="cuda")
    f, z, _ = c.gates

    def forward(scratch):
        o.glr_forward(c.plan, c.shape, f, z, None, c.h0, c.y, c.h_n, c.ws, scratch=scratch)

    def backward(scratch):
        o.glr_backward(c.plan, c.shape, f, z, None, c.ws, c.v["dy"], c.dh_n, c.grads[0], c.grads[1], None, c.dh0, scratch=scratch)

    for call in (forward, backward):
        mine.fill_(85)
        call(mine[:need])
        assert (mine[:need] != 85).any() and (mine[need:] == 85).all()
        for bad in (mine[:need - 1], mine[:need].cpu()):
            with pytest.raises(ValueError):
                call(bad)
    assert not kept(c.plan)
    got = [t.clone() for t in outs(c)]
    c.check()
    assert len(kept(c.plan)) == 1       # the plan's own, for both calls of this stream
    assert all(torch.equal(x.nan_to_num(7), y.nan_to_num(7)) for x, y in zip(got, outs(c)))
