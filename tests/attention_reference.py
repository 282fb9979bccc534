"""64-bit restatements (numpy) of linear attention with a decay for each head and of the norms and rotations of its queries
and keys, frame by frame from their definitions, with bounds on what the arithmetic may be off.

The bounds are derived, not fitted.  u = 2^-24 is half an ulp of fp32.

Linear attention.  Every term of a state is a product that is added up in fp32, decayed by powers of lambda that are
exponentials of a rounded logarithm (4 |ln lambda| u a step: the logarithm in base 2, its product with the number of steps and
the exponential's own argument), at most one rounding of the sum a step (2 u: tensor cores may cut off where others round), and
a handful more when a chunk of steps begins or ends (32 u in all, which also holds the weight's and the scale's products).  So
with |S| the state of absolute values, its error e follows the same recurrence: e' = lambda e + (2 + 4 |ln lambda|) u |S|, and 32 u |S|
at the end.  An output adds `a` products of the query with it and up to 128 of one chunk: (a + 128) 2 u of the absolute sum.
bf16: products between two frames of a chunk are rounded to bf16 (2^-8) before they weigh the values, and the state enters
its product in two bf16 pieces (2^-16): together less than 1.02 2^-8 of the absolute sum.  The result's own rounding to bf16 is at
most 2^-8 of it.

Norms.  As in the norms around a block: sums over a head add four pairs a lane and then a tree: 64 u of the absolute sum.  An
angle is exact up to its fp32 rounding in half turns (pi 2^-24) and the sine's and cosine's 2 ulp: 8 u absolute each.
"""
import numpy as np

from operator_reference import U, packed_rows

BF16 = 2.0 ** -8            # half an ulp of bf16, relative to the value at most


def attend(lengths, q, k, v, log_decay, scale, s0=None, dy=None, ds_n=None, padded=False, bf16=False):
    """q, k [rows, nd, heads, a], v, dy [rows, nd, heads, b], s0, ds_n [nd, B, heads, a, b], log_decay [nd, heads].  Values under
    a name, their error bounds under "~name"."""
    q, k, v = (x.astype(np.float64) for x in (q, k, v))
    rows_of, n = packed_rows(lengths, padded)
    nd, H, a = q.shape[1:]
    b, B = v.shape[3], len(rows_of)
    shape = (nd, B, H, a, b)
    s0 = np.zeros(shape) if s0 is None else s0.astype(np.float64)
    ds_n = np.zeros(shape) if ds_n is None else ds_n.astype(np.float64)
    ld = np.minimum(np.maximum(log_decay.astype(np.float64), -138.0), 0.0)
    piece = 1.02 * BF16 if bf16 else 0.0
    o = {x: np.zeros((n, nd, H, b if x.strip("~") in ("y", "dv") else a)) for x in ("y", "~y", "dq", "~dq", "dk", "~dk", "dv", "~dv")}
    o.update({x: np.zeros(shape) for x in ("s_n", "~s_n", "ds0", "~ds0")})
    mul = lambda m, x: np.einsum("hab,hb->ha", m, x)       # noqa: E731
    tmul = lambda m, x: np.einsum("hab,ha->hb", m, x)      # noqa: E731
    outer = lambda x, y: np.einsum("ha,hb->hab", x, y)     # noqa: E731
    c = abs(scale)
    for bi, rows in enumerate(rows_of):
        for d in range(nd):
            r = rows if d == 0 else rows[::-1]
            lam = np.exp(ld[d])[:, None, None]
            step = ((2 + 4 * np.abs(ld[d])) * U)[:, None, None]
            S, big, err = s0[d, bi], np.abs(s0[d, bi]), np.zeros((H, a, b))
            for x in r:
                S = lam * S + outer(k[x, d], v[x, d])
                big = lam * big + np.abs(outer(k[x, d], v[x, d]))
                err = lam * err + step * big
                e = err + (32 + 2 * (a + 128)) * U * big + piece * big
                o["y"][x, d], o["~y"][x, d] = scale * tmul(S, q[x, d]), c * tmul(e, np.abs(q[x, d]))
                if dy is not None:
                    e = err + (32 + 2 * (b + 128)) * U * big + piece * big
                    o["dq"][x, d], o["~dq"][x, d] = scale * mul(S, dy[x, d]), c * mul(e, np.abs(dy[x, d]))
            o["s_n"][d, bi], o["~s_n"][d, bi] = S, err + 32 * U * big
            if dy is None:
                continue
            D, big, err = ds_n[d, bi], np.abs(ds_n[d, bi]), np.zeros((H, a, b))
            for x in r[::-1]:
                g = outer(q[x, d], dy[x, d])
                D, big = D + scale * g, big + c * np.abs(g)
                err = err + step * big
                e = err + (32 + 2 * (b + 128)) * U * big + piece * big
                o["dk"][x, d], o["~dk"][x, d] = mul(D, v[x, d]), mul(e, np.abs(v[x, d]))
                e = err + (32 + 2 * (a + 128)) * U * big + piece * big
                o["dv"][x, d], o["~dv"][x, d] = tmul(D, k[x, d]), tmul(e, np.abs(k[x, d]))
                D, big, err = lam * D, lam * big, lam * err
            o["ds0"][d, bi], o["~ds0"][d, bi] = D, err + 32 * U * big
    return o


def qk_norm(kind, layout, rotary, x, w, freq, pos, eps=1e-6, turn_scale=1.0, dout=None, live=None):
    """x, dout [rows, heads, d]; w [d] or None; freq [rotary / 2] radians a position; pos [rows]; live [rows] of bool.  Values
    under a name, bounds under "~name"."""
    x = x.astype(np.float64)
    n, h, d = x.shape
    S = 64 * U
    w = np.ones(d) if w is None else w.astype(np.float64)
    left = np.arange(rotary // 2) * (1 if layout == "half" else 2)
    right = left + (rotary // 2 if layout == "half" else 1)
    # position 10^12 times a frequency is off by 10^12 2^-53 = 10^-4 in 64 bits: the angle, modulo a turn, in long doubles (2^-64)
    turn_ = 2 * np.arccos(np.longdouble(-1))
    ang = pos.astype(np.longdouble)[:, None] * (np.asarray(freq, dtype=np.longdouble) if rotary else np.zeros(0))
    ang = (ang - turn_ * np.floor(ang / turn_)).astype(np.float64)
    co, si = turn_scale * np.cos(ang)[:, None], turn_scale * np.sin(ang)[:, None]
    ec = abs(turn_scale) * 10 * U

    def turn(v, ev, way):
        out, eo = v.copy(), ev + 2 * U * np.abs(v)
        a, b, ea, eb = v[..., left], v[..., right], ev[..., left], ev[..., right]
        size = np.abs(a) + np.abs(b)
        out[..., left], out[..., right] = a * co - way * b * si, way * a * si + b * co
        eo[..., left] = ea * np.abs(co) + eb * np.abs(si) + ec * size + 4 * U * abs(turn_scale) * size
        eo[..., right] = ea * np.abs(si) + eb * np.abs(co) + ec * size + 4 * U * abs(turn_scale) * size
        return out, eo

    m = x.mean(-1, keepdims=True) if kind == "layer" else np.zeros((n, h, 1))
    t = x - m
    et = U * np.abs(x) + (np.abs(x).mean(-1, keepdims=True) * S if kind == "layer" else 0.0)
    if kind == "none":
        hat, eh, r, er = t, np.zeros_like(t), np.ones((n, h, 1)), 0.0
    else:
        var = (t * t).mean(-1, keepdims=True) + eps
        r = 1 / np.sqrt(var)
        er = (2 * (np.abs(t) * et + et * et).mean(-1, keepdims=True) + S * var) / (2 * var) * 1.01 + 8 * U
        hat = t * r
        eh = et * r + np.abs(hat) * (er + 4 * U)
    o = {}
    o["out"], o["~out"] = turn(hat * w, eh * np.abs(w) + 2 * U * np.abs(hat * w), 1.0)
    on = np.ones((n, 1, 1)) if live is None else live.astype(np.float64)[:, None, None]
    o["out"], o["~out"] = o["out"] * on, o["~out"] * on
    if dout is None:
        return o
    g, eg = turn(dout.astype(np.float64) * on, np.zeros_like(x), -1.0)
    terms = np.abs(g * hat)
    # rows are added in at most 608 * 8 warps, each in order, then those: every addition rounds
    o["dw"] = (g * hat).sum((0, 1))
    o["~dw"] = (eg * np.abs(hat) + (np.abs(g) + eg) * eh).sum((0, 1)) + (n * h / 608.0 + 608 + 64) * U * terms.sum((0, 1))
    g, eg = g * w, eg * np.abs(w) + 2 * U * np.abs(g * w)
    if kind != "none":
        along = (g * hat).mean(-1, keepdims=True)
        ea = (eg * np.abs(hat) + np.abs(g) * eh + eg * eh).mean(-1, keepdims=True) + S * np.abs(g * hat).mean(-1, keepdims=True)
        mean, em = 0.0, 0.0
        if kind == "layer":
            mean = g.mean(-1, keepdims=True)
            em = eg.mean(-1, keepdims=True) + S * np.abs(g).mean(-1, keepdims=True)
        size = np.abs(g) + np.abs(mean) + np.abs(hat * along)
        eg = r * (eg + em + eh * np.abs(along) + (np.abs(hat) + eh) * ea + (er + 8 * U) * size)
        g = r * (g - mean - hat * along)
    o["dx"], o["~dx"] = g * on, eg * on
    return o
