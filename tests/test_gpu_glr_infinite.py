"""Infinite states and errors in the gated linear recurrence: what stays infinite frame by frame stays so in the scan, however
its steps are grouped and however small the products of their gates become."""
import numpy as np
import pytest

import operator_reference as ref
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
    # a CTA a sequence (rows in 16 bytes, of 4 and of 2 bytes' alignment, narrow layers), cut, a warp a sequence
    ([300, 7, 129], 2, 64, "f32", "tied", 0), ([300, 7, 129], 1, 96, "bf16", "gated", 0), ([200, 65], 2, 33, "f32", "gated", 0),
    ([200, 65], 1, 130, "bf16", "tied", 1), ([300, 200], 1, 16, "f32", "gated", 0), ([300, 200], 2, 24, "bf16", "tied", 0),
    ([5000, 900], 1, 64, "f32", "gated", 0), ([5000, 900], 1, 33, "f32", "tied", 0), ([5000, 900], 2, 16, "bf16", "gated", 0),
    ([100] * 700, 1, 40, "f32", "gated", 0), ([16, 9, 3], 2, 40, "f32", "tied", 0),
]


def same(got, want, what):
    """Infinite where the definition is, with its sign, and finite elsewhere (values: the other tests)."""
    got, want = got.double().cpu().numpy(), np.asarray(want)
    assert not np.isnan(want).any(), what
    assert not np.isnan(got).any(), (what, int(np.isnan(got).sum()))
    at = np.isinf(got) | np.isinf(want)
    assert np.array_equal(got[at], want[at]), what


@pytest.mark.parametrize("case", CASES, ids=[f"{i}-H{c[2]}-{c[3]}-{c[4]}" for i, c in enumerate(CASES)])
@pytest.mark.parametrize("bias", [-9.0, -2.0, 3.0])
def test_infinite_states_and_errors(case, bias):
    lens, nd, H, dtype, cell, shift = case
    c = Case(lens, nd, H, dtype, cell, shift=shift, bias=bias, seed=11)
    inf = float("inf")
    c.h0[:, 0, ::5] = inf                   # a state that comes in, then one that an input makes
    c.h0[:, 1, 1::5] = -inf
    rows, _ = ref.packed_rows(lens)
    mid = torch.from_numpy(np.concatenate([r[len(r) // 2:len(r) // 2 + 1] for r in rows])).cuda()
    c.v["z"][mid, :, 2::5] = inf
    c.gates[1].copy_(c.v["z"])
    c.forward()
    w = c.want()
    same(c.y, w["y"], "y")
    same(c.h_n, w["h_n"], "h_n")
    # the error: infinite from outside for some units whose states are finite
    c.dh_n[:, 0, 3::5] = -inf
    c.v["dy"][mid, :, 4::5] = inf
    c.backward()
    w = c.want()
    same(c.grads[1], w["dz"], "dz")
    same(c.dh0, w["dh0"], "dh0")


@pytest.mark.parametrize("cell", ["tied", "gated"])
def test_the_smallest_gates(cell):
    # sig(-100) is below the smallest normal number and above 0
    L, H = 200, 40
    c = Case([L, L], 1, H, "f32", cell)
    c.v["f"].fill_(-100.0)
    c.gates[0].copy_(c.v["f"])
    c.h0[0, 0] = float("inf")
    c.forward()
    w = c.want()
    same(c.y, w["y"], "y")
    cache, y = c.h0[0].clone(), torch.empty(2, 1, H, device="cuda")
    for t in range(L):
        ops().glr_step(c.shape, *[None if v is None else v[2 * t:2 * t + 2] for v in c.gates], cache, cache, y)
        same(y, w["y"][2 * t:2 * t + 2], t)
    same(cache[None], w["h_n"], "state")
