"""The block norms at widths that no multiple of 8 divides, in rows that start equally far from a multiple of 8 values (the
kernels that read groups of 8 from there), and at the aligned widths of the larger CTAs, against the 64-bit restatement:
every size of a CTA, types, rows enough for several trips of CTAs that stay, in place, neighbours that are not finite."""
import numpy as np
import pytest

from test_gpu_block_norm import Case, ops

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from padding_free_variable_gb300 import build
    build.build()


CASES = [
    # rows, D, kind, gate, branch, stream, padding of strided rows (a multiple of 8)
    # CTAs of several rows (4, 8, 16, 32 threads a row), of 64 to 512 threads, one or two rows at a time
    (20000, 7, "rms", "silu", "f32", "f32", 0), (30000, 17, "layer", "sigmoid", "bf16", "f32", 8),
    (20000, 33, "rms", "none", "bf16", "bf16", 0), (12000, 77, "layer", "silu", "f32", "f32", 0),
    (9000, 131, "layer", "silu", "bf16", "bf16", 0), (9000, 249, "rms", "sigmoid", "f32", "f32", 16),
    (4000, 511, "rms", "silu", "bf16", "bf16", 0), (3000, 517, "layer", "sigmoid", "f32", "f32", 0),
    (3000, 517, "layer", "sigmoid", "f32", "f32", 8), (3000, 1001, "rms", "silu", "bf16", "f32", 0),
    (3000, 1001, "layer", "none", "bf16", "bf16", 24), (2500, 1023, "rms", "sigmoid", "f32", "f32", 0),
    (1500, 1533, "layer", "silu", "bf16", "f32", 0), (1200, 2045, "rms", "none", "f32", "f32", 0),
    (1000, 2501, "rms", "silu", "bf16", "bf16", 0), (1000, 2501, "layer", "sigmoid", "f32", "f32", 8),
    (900, 2999, "layer", "silu", "bf16", "f32", 0), (1000, 3501, "rms", "silu", "bf16", "bf16", 0),
    (1000, 3501, "layer", "silu", "bf16", "f32", 8), (700, 3501, "layer", "none", "f32", "f32", 0),
    (700, 4089, "rms", "sigmoid", "bf16", "f32", 0), (310, 4091, "layer", "silu", "f32", "f32", 0),
    (400, 7001, "layer", "silu", "bf16", "bf16", 0), (400, 8185, "rms", "none", "f32", "f32", 0),
    # aligned: one group a thread in CTAs of 320 to 512 threads
    (1400, 2560, "rms", "silu", "bf16", "bf16", 0), (1400, 2560, "layer", "sigmoid", "f32", "f32", 8),
    (1400, 3584, "layer", "silu", "bf16", "f32", 0), (1400, 4096, "rms", "none", "bf16", "bf16", 0),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}x{c[1]}-{c[2]}-{c[3]}-{c[4]}-{c[5]}-{c[6]}" for c in CASES])
def test_matches_definition(case):
    n, D, kind, gate, branch, stream, pad = case
    Case(n, D, kind, gate, branch, stream, pad=pad).check()


def test_few_rows_of_every_small_width():
    # the last rows, whose groups must not be read past the end
    for D in list(range(1, 26)) + [39, 63, 121]:
        for n in (1, 2, 3, 9):
            Case(n, D, "layer" if D % 2 else "rms", "silu", "bf16", "f32" if D % 3 else "bf16").check()


def run(c):
    c.forward()
    c.backward()
    torch.cuda.synchronize()


PLACES = [(3000, 517, "layer", "f32", "f32"), (4000, 511, "rms", "bf16", "bf16"), (2000, 1001, "layer", "bf16", "f32"),
          (900, 3501, "rms", "bf16", "bf16"), (9000, 33, "rms", "f32", "f32")]


@pytest.mark.parametrize("n,D,kind,branch,stream", PLACES)
def test_in_place(n, D, kind, branch, stream):
    c = Case(n, D, kind, "silu", branch, stream)
    run(c)
    want = [t.clone() for t in (c.x_out, c.nn, c.stats, c.dx, c.dy, c.dg)]
    dp = {k: v.clone() for k, v in c.dp.items()}
    c.dx.copy_(c.dx_out)
    ops().block_norm_backward(c.shape, c.x, c.y, c.g, c.p, c.stats, c.dx, c.dn, c.dx, c.dy, c.dg, c.dp, c.scratch)
    ops().block_norm_forward(c.shape, c.x, c.y, c.g, c.p, c.x, c.nn, c.stats)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((c.x, c.nn, c.stats, c.dx, c.dy, c.dg), want))
    assert all(torch.equal(c.dp[k], v) for k, v in dp.items())


@pytest.mark.parametrize("n,D,kind,branch,stream", PLACES)
def test_what_is_not_finite_stays_in_its_row(n, D, kind, branch, stream):
    c, d = Case(n, D, kind, "silu", branch, stream), Case(n, D, kind, "silu", branch, stream)
    hit = [1, 4, 11, n - 2]
    nan, inf = float("nan"), float("inf")
    for t, r, at, bad in ((d.y, 1, 0, nan), (d.y, 1, D - 1, nan), (d.x, 4, 0, inf), (d.x, 4, D - 1, -inf), (d.g, 11, D - 1, nan),
                          (d.dn, 11, 0, inf), (d.dx_out, n - 2, D - 1, nan), (d.x, n - 2, 0, nan)):
        t[r, at] = bad
    run(c)
    run(d)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[hit] = False
    for a, b in ((c.x_out, d.x_out), (c.nn, d.nn), (c.dx, d.dx), (c.dy, d.dy), (c.dg, d.dg)):
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(d.nn[1]).all() and torch.isnan(d.dx[n - 2]).any()


def test_repeats_agree_bitwise():
    for n, D, kind, branch, stream in PLACES:
        c = Case(n, D, kind, "silu", branch, stream)
        run(c)
        outs = [c.x_out, c.nn, c.dx, c.dy, c.dg] + list(c.dp.values())
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(3)
        c.scratch.fill_(255)
        run(c)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_nothing_is_written_beside_the_rows():
    for D, pad in ((517, 8), (33, 16), (3501, 8)):
        c = Case(40, D, "layer", "silu", pad=pad)
        guard = torch.full((40 * D + 64,), 7.0, device="cuda")
        c.x_out = guard[32:32 + 40 * D].view(40, D)
        run(c)
        assert (guard[:32] == 7).all() and (guard[-32:] == 7).all()
        for t, extra in ((c.dy, pad), (c.dg, 3 * pad)):
            beside = torch.as_strided(t, (39, extra), (D + extra, 1), t.storage_offset() + D)
            assert torch.isnan(beside).all()
