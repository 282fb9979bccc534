"""64-bit restatements (numpy) of the gated linear recurrence and of the norms around a block, frame by frame and row by
row from their definitions, with bounds on what 32-bit arithmetic may be off.

The bounds are derived, not fitted.  u = 2^-24 is half an ulp of fp32.  A gate's smaller side e/(1+e), e = exp(-|x|), has
the argument's rounding (|x| u), the hardware exponential (2 ulp = 4 u), 1 + e (u), the hardware reciprocal (2 u) and the
product (u): (8 + |x|) u relative.  A step multiplies by the gate and adds, in any grouping of the steps, with a few
roundings more, so every factor and term of h_t = sum_s (prod a) b_s carries at most EPS_t = (16 + |f| + |i|) u relative,
and errors travel along the same recurrence in absolute values.  Rounding to bf16 adds 2^-8 of the value (its half ulp is
2^-9).  Sums over a row of D values add groups of at most 32 values before a tree: 64 u of the sum of the absolute values.
"""
import numpy as np

U = 2.0 ** -24


def sig(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def packed_rows(lengths, padded=False):
    """row[b][t]: packed row of frame t of the caller's sequence b, and the number of rows."""
    lengths = list(lengths)
    B, T = len(lengths), max(lengths) if len(lengths) else 0
    if padded:
        return [np.arange(L) * B + b for b, L in enumerate(lengths)], B * T
    order = sorted(range(B), key=lambda b: (-lengths[b], b))
    rows = [np.zeros(L, np.int64) for L in lengths]
    r = 0
    for t in range(T):
        for b in order:
            if lengths[b] > t:
                rows[b][t] = r
                r += 1
    return rows, r


def glr(lengths, f, z, i=None, h0=None, dy=None, dh_n=None, padded=False):
    """f, z, i, dy [rows, ndir, H]; h0, dh_n [ndir, B, H].  Values under a name, their error bounds under "~name"."""
    f, z = f.astype(np.float64), z.astype(np.float64)
    i = None if i is None else i.astype(np.float64)
    rows_of, n = packed_rows(lengths, padded)
    nd, H = f.shape[1:]
    B = len(rows_of)
    h0 = np.zeros((nd, B, H)) if h0 is None else h0.astype(np.float64)
    dh_n = np.zeros((nd, B, H)) if dh_n is None else dh_n.astype(np.float64)
    a, c = sig(f), sig(-f)
    g, gc = (c, a) if i is None else (sig(i), sig(-i))
    eps = (16 + np.minimum(np.abs(f), 90) + (0 if i is None else np.minimum(np.abs(i), 90))) * U
    o = {k: np.zeros((n, nd, H)) for k in ("y", "~y", "df", "~df", "dz", "~dz", "di", "~di")}
    o.update({k: np.zeros((nd, B, H)) for k in ("h_n", "~h_n", "dh0", "~dh0")})
    for b, rows in enumerate(rows_of):
        for d in range(nd):
            r = rows if d == 0 else rows[::-1]
            h, big, err = h0[d, b], np.abs(h0[d, b]), np.zeros(H)
            prev = np.zeros((len(r), H))
            perr = np.zeros((len(r), H))
            for k, x in enumerate(r):
                prev[k], perr[k] = h, err
                b_ = g[x, d] * z[x, d]
                h = a[x, d] * h + b_
                big = a[x, d] * big + np.abs(b_)
                err = a[x, d] * err + eps[x, d] * big
                o["y"][x, d], o["~y"][x, d] = h, err
            o["h_n"][d, b], o["~h_n"][d, b] = h, err
            if dy is None:
                continue
            e, big, err = dh_n[d, b], np.abs(dh_n[d, b]), np.zeros(H)
            for k in range(len(r) - 1, -1, -1):
                x = r[k]
                G, big, err = dy[x, d] + e, np.abs(dy[x, d]) + big, err + 2 * U * (np.abs(dy[x, d]) + big)
                s = prev[k] if i is not None else prev[k] - z[x, d]
                sabs = np.abs(prev[k]) + (0 if i is not None else np.abs(z[x, d]))
                slope, ep = a[x, d] * c[x, d], 3 * eps[x, d]
                o["df"][x, d] = G * s * slope
                o["~df"][x, d] = slope * (err * sabs + big * (perr[k] + ep * sabs))
                o["dz"][x, d], o["~dz"][x, d] = G * g[x, d], g[x, d] * (err + ep * big)
                if i is not None:
                    o["di"][x, d] = G * z[x, d] * g[x, d] * gc[x, d]
                    o["~di"][x, d] = np.abs(z[x, d]) * g[x, d] * gc[x, d] * (err + ep * big)
                e, big, err = a[x, d] * G, a[x, d] * big, a[x, d] * (err + eps[x, d] * big)
            o["dh0"][d, b], o["~dh0"][d, b] = e, err
    return o


def block_norm(kind, gate, x, y, g, p, eps=1e-6, dx_out=None, dn=None, post_kind=None, backward=False):
    """Rows [n, D]; p: dict of w_post, b_post, scale, w_pre, b_pre (any absent).  y None: pre-norm only.  kind / post_kind
    "none": that norm absent.  Values under a name, their error bounds under "~name"."""
    post = kind if post_kind is None else post_kind
    x = x.astype(np.float64)
    D = x.shape[1]
    S = 64 * U                      # a row sum, relative to the sum of absolute values
    one, zero = np.ones(D), np.zeros(D)
    P = {k: p[k].astype(np.float64) if p.get(k) is not None else (zero if k[0] == "b" else one)
         for k in ("w_post", "b_post", "scale", "w_pre", "b_pre")}
    o = {}

    def norm(kd, v, ev):
        """normalised rows, 1/deviation, and the bounds of the former (absolute) and of the latter (relative)"""
        if kd == "none":
            return v, np.ones((len(v), 1)), ev, 0.0
        m = v.mean(1, keepdims=True) if kd == "layer" else np.zeros((len(v), 1))
        em = (np.abs(v).mean(1, keepdims=True) * S + ev.mean(1, keepdims=True)) if kd == "layer" else 0.0
        w = v - m
        ew = ev + em + U * (np.abs(v) + np.abs(m))
        var = (w * w).mean(1, keepdims=True) + eps
        evar = 2 * (np.abs(w) * ew + ew * ew).mean(1, keepdims=True) + S * var
        r = 1 / np.sqrt(var)
        er = evar / (2 * var) * 1.01 + 8 * U
        return w * r, r, ew * r + np.abs(w) * r * (er + 4 * U), er

    def through(kd, hat, eh, r, er, t, et):
        """a norm's backward pass r (t - mean t - hat mean(t hat)) and its bound"""
        if kd == "none":
            return t, et
        q = (t * hat).mean(1, keepdims=True)
        eq = (et * np.abs(hat) + np.abs(t) * eh + et * eh).mean(1, keepdims=True) + S * np.abs(t * hat).mean(1, keepdims=True)
        m, em = 0.0, 0.0
        if kd == "layer":
            m = t.mean(1, keepdims=True)
            em = et.mean(1, keepdims=True) + S * np.abs(t).mean(1, keepdims=True)
        v = r * (t - m - hat * q)
        size = np.abs(t) + np.abs(m) + np.abs(hat * q)
        return v, r * (et + em + eh * np.abs(q) + (np.abs(hat) + eh) * eq + (er + 8 * U) * size)

    if y is None:
        x1, e1 = x, np.zeros_like(x)
    else:
        y = y.astype(np.float64)
        yh, ry, eyh, ery = norm(post, y, np.zeros_like(y))
        v = yh * P["w_post"] + P["b_post"]
        ev = eyh * np.abs(P["w_post"]) + 4 * U * (np.abs(yh * P["w_post"]) + np.abs(P["b_post"]))
        act, slope, ea = np.ones_like(y), np.zeros_like(y), np.zeros_like(y)
        if gate != "none":
            g = g.astype(np.float64)
            s, c = sig(g), sig(-g)
            eg = (12 + np.minimum(np.abs(g), 90)) * U
            act, slope = (s, s * c) if gate == "sigmoid" else (g * s, s * (1 + g * c))
            ea = np.abs(act) * eg
            eslope = (2 * s * c if gate == "sigmoid" else s * (1 + 2 * np.abs(g) * c)) * eg
        x1 = x + P["scale"] * v * act
        e1 = np.abs(P["scale"]) * (ev * np.abs(act) + np.abs(v) * ea) + 6 * U * (np.abs(x) + np.abs(P["scale"] * v * act))
        o["x_out"], o["~x_out"] = x1, e1
    xh, rx, exh, erx = norm(kind, x1, e1)
    if kind != "none":
        o["n"] = xh * P["w_pre"] + P["b_pre"]
        o["~n"] = exh * np.abs(P["w_pre"]) + 4 * U * (np.abs(xh * P["w_pre"]) + np.abs(P["b_pre"]))
    if not backward:
        return o
    dx = np.zeros_like(x) if dx_out is None else dx_out.astype(np.float64)
    edx = np.zeros_like(x)
    if dn is not None:
        dn = dn.astype(np.float64)
        t, et = through(kind, xh, exh, rx, erx, dn * P["w_pre"], U * np.abs(dn * P["w_pre"]))
        edx = et + 2 * U * (np.abs(dx) + np.abs(t))
        dx = dx + t
    o["dx"], o["~dx"] = dx, edx
    sums = {"w_pre": (dn * xh, np.abs(dn) * exh), "b_pre": (dn, 0 * dn)} if dn is not None else \
        {"w_pre": (0 * x, 0 * x), "b_pre": (0 * x, 0 * x)}
    if y is not None:
        du, edu = P["scale"] * dx, np.abs(P["scale"]) * edx + U * np.abs(P["scale"] * dx)
        dv, edv = du * act, edu * np.abs(act) + (np.abs(du) + edu) * ea + U * np.abs(du * act)
        t, et = dv * P["w_post"], (edv + U * np.abs(dv)) * np.abs(P["w_post"])
        o["dy"], o["~dy"] = through(post, yh, eyh, ry, ery, t, et)
        if gate != "none":
            o["dgate"] = du * v * slope
            o["~dgate"] = (edu * np.abs(v) + (np.abs(du) + edu) * ev) * np.abs(slope) + \
                (np.abs(du * v)) * eslope + 4 * U * np.abs(du * v) * (np.abs(slope) + eslope)
        sums["w_post"] = (dv * yh, edv * np.abs(yh) + (np.abs(dv) + edv) * eyh)
        sums["b_post"] = (dv, edv)
        sums["scale"] = (dx * v * act, edx * np.abs(v * act) + (np.abs(dx) + edx) * (ev * np.abs(act) + np.abs(v) * ea))
    n = len(x)
    for k, (v, e) in sums.items():
        # rows are added in at most 304 ranges, each in order: n/304 + 304 additions, and a few roundings a term
        o["d" + k] = v.sum(0)
        o["~d" + k] = e.sum(0) + (n / 304 + 304 + 16) * U * np.abs(v).sum(0)
    return o
