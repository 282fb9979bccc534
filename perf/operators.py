"""The packed sequence operators as a user's program calls them, with their plain forms, for timing and comparison.

Two operators over the packed rows of a plan (row ``off[t] + j`` is frame t of the j-th longest sequence), and one for a
single new frame:

scan / train   the gated linear recurrence h_t = a_t h_{t-1} + b_t with a = sigmoid(f), per unit and direction; cell "tied"
               has b = (1 - a) z, cell "gated" has b = sigmoid(i) z.  "scan" is the forward pass (h of every frame and the
               final states), "train" the forward pass and the gradients of f, z, i and h_0.
step           the same recurrence for one new frame of each of many streams, whose states lie in a cache of slots.
norm /         the norms around a block: x' = x + s * (norm(y) w_post [+ b_post]) * act(gate), n = norm(x') w_pre [+ b_pre];
norm_train     "norm" is the forward pass, "norm_train" the forward pass and every gradient.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a few short words: the smallest call, where the launch is the cost
        {"name": "scan-words-f32", "op": "scan", "cell": "tied", "dtype": "f32", "ndir": 1, "hidden": 32, "batch": 8,
         "dist": "uniform", "lo": 5, "hi": 40, "empty": 0, "h0": False, "lens_seed": 1001},
        # the library's headline batch (64 utterances, 40 k frames, both directions) in bf16
        {"name": "scan-utterances-bf16", "op": "scan", "cell": "gated", "dtype": "bf16", "ndir": 2, "hidden": 512,
         "batch": 64, "dist": "lognormal", "lo": 100, "hi": 2000, "empty": 0, "h0": False, "lens_seed": 1003},
        # one recording of 65 536 frames, not cut into segments
        {"name": "scan-recording-bf16", "op": "scan", "cell": "tied", "dtype": "bf16", "ndir": 1, "hidden": 1024,
         "batch": 1, "dist": "uniform", "lo": 65536, "hi": 65536, "empty": 0, "h0": True, "lens_seed": 7},
        # odd width (no vector access lines up), sequences of no frame and of one, a carried state
        {"name": "scan-odd-f32", "op": "scan", "cell": "gated", "dtype": "f32", "ndir": 2, "hidden": 203, "batch": 37,
         "dist": "uniform", "lo": 1, "hi": 700, "empty": 3, "h0": True, "lens_seed": 11},
        # a training step's pass on the headline batch
        {"name": "train-utterances-bf16", "op": "train", "cell": "tied", "dtype": "bf16", "ndir": 2, "hidden": 512,
         "batch": 64, "dist": "lognormal", "lo": 100, "hi": 2000, "empty": 0, "h0": False, "lens_seed": 1003},
        # many sequences of an fp32 layer, three gates
        {"name": "train-batch-f32", "op": "train", "cell": "gated", "dtype": "f32", "ndir": 2, "hidden": 256,
         "batch": 128, "dist": "uniform", "lo": 100, "hi": 1000, "empty": 0, "h0": False, "lens_seed": 1004},
        # two long sequences: little to do side by side, much one after another; states in, their gradients out
        {"name": "train-long-f32", "op": "train", "cell": "tied", "dtype": "f32", "ndir": 1, "hidden": 512, "batch": 2,
         "dist": "uniform", "lo": 20001, "hi": 30001, "empty": 0, "h0": True, "lens_seed": 13},
        # streaming recognition: one new frame of eight streams
        {"name": "step-streams-bf16", "op": "step", "cell": "tied", "dtype": "bf16", "ndir": 1, "hidden": 512, "batch": 8,
         "slots": 16, "idle": 1, "h0": True},
        # a server's tick over thousands of streams
        {"name": "step-server-f32", "op": "step", "cell": "gated", "dtype": "f32", "ndir": 1, "hidden": 1024,
         "batch": 4096, "slots": 5000, "idle": 97, "h0": True},
        # the same tick's norms: few rows, latency counts
        {"name": "norm-streams-bf16", "op": "norm", "kind": "rms", "gate": "silu", "branch": "bf16", "stream": "bf16",
         "rows": 8, "width": 1024},
        # the headline batch's block, both directions side by side in a row
        {"name": "norm-train-utterances-bf16", "op": "norm_train", "kind": "rms", "gate": "silu", "branch": "bf16",
         "stream": "bf16", "rows": 40555, "width": 1024},
        # an fp32 layer of odd width, centred norms with biases
        {"name": "norm-train-odd-f32", "op": "norm_train", "kind": "layer", "gate": "sigmoid", "branch": "f32",
         "stream": "f32", "rows": 9564, "width": 517},
    ]


def draw(rng):
    """One more case: widths, batches and lengths spread over their logarithms, odd ones among them."""
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))

    op = rng.choice(["scan", "scan", "train", "train", "step", "norm", "norm_train"])
    work = math.exp(rng.uniform(math.log(2e4), math.log(3.2e7)))      # units of one pass
    dtype = rng.choice(["f32", "bf16"])
    if op in ("norm", "norm_train"):
        work = min(work, 2.6e7)
        width = log(16, 8192)
        width = width // 8 * 8 if rng.random() < 0.7 else width
        stream = rng.choice(["f32", dtype])
        return {"op": op, "kind": rng.choice(["rms", "layer"]), "gate": rng.choice(["none", "sigmoid", "silu"]),
                "branch": dtype, "stream": stream, "rows": max(1, min(200000, int(work / width))), "width": width}
    hidden = log(8, 2048)
    hidden = hidden // 8 * 8 if rng.random() < 0.7 else hidden
    case = {"op": op, "cell": rng.choice(["tied", "gated"]), "dtype": dtype, "hidden": hidden}
    if op == "step":
        batch = max(1, min(16384, int(min(work, 1.6e7) / hidden)))
        return dict(case, ndir=1, batch=batch, slots=batch + rng.randrange(0, batch + 8),
                    idle=rng.randrange(0, batch // 8 + 1), h0=True)
    ndir = rng.choice([1, 2])
    batch = log(1, 256)
    mean = max(1, min(65536, int(work / (hidden * ndir * batch))))
    if batch == 1 or rng.random() < 0.2:
        lo = hi = mean
        dist = "uniform"
    else:
        dist = rng.choice(["uniform", "lognormal"])
        lo, hi = max(1, mean // 6), max(1, mean * 2 - mean // 6)
    case.update(ndir=ndir, batch=batch, dist=dist, lo=lo, hi=min(hi, 65536), h0=rng.random() < 0.5,
                empty=rng.choice([0, 0, 0, 2]) if batch > 4 else 0, lens_seed=rng.randrange(1 << 30))
    while int(lengths_of(case).sum()) * ndir * hidden > 3.3e7:
        case["hi"] = max(case["hi"] * 3 // 4, 1)
        case["lo"] = min(case["lo"], case["hi"])
    return case


def lengths_of(case):
    """The sequences' lengths: a function of the case alone."""
    rng = random.Random(case["lens_seed"])
    lo, hi, n = case["lo"], case["hi"], case["batch"]
    if case["dist"] == "lognormal":
        median = math.sqrt(lo * hi) * 1.3
        lens = [int(min(hi, max(lo, round(median * math.exp(0.5 * rng.gauss(0, 1)))))) for _ in range(n)]
    else:
        lens = [rng.randint(lo, hi) for _ in range(n)]
    if case["empty"]:                     # sequences of no frame, and one of a single frame
        lens[1:1 + case["empty"]] = [0] * case["empty"]
        lens[0] = 1
    return np.array(lens, dtype=np.int64)


def packing(lens):
    """Sorted order, batch sizes and offsets of the packed rows."""
    order = np.argsort(-lens, kind="stable")
    top = lens[order]
    steps = int(top[0]) if len(top) else 0
    bs = (len(top) - np.searchsorted(top[::-1], np.arange(steps), side="right")).astype(np.int64)
    off = np.concatenate([[0], np.cumsum(bs)]).astype(np.int64)
    return order, top, bs, off


# ------------------------------------------------------------------ inputs

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(case, seed):
    """The tensors of a call, on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)

    def normal(*shape, mean=0.0, std=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(dtype)

    s = {}
    if case["op"] in ("norm", "norm_train"):
        n, d, br, st = case["rows"], case["width"], DT[case["branch"]], DT[case["stream"]]
        s["x"] = normal(n, d, std=1.5, dtype=st)                       # the residual stream
        s["y"] = normal(n, d, mean=0.1, std=0.6, dtype=br)             # the block's output
        s["gate"] = normal(n, d, std=1.2, dtype=br) if case["gate"] != "none" else None
        s["p"] = {"w_post": normal(d, mean=1.0, std=0.2), "scale": normal(d, mean=0.5, std=0.2),
                  "w_pre": normal(d, mean=1.0, std=0.2)}
        if case["kind"] == "layer":
            s["p"].update(b_post=normal(d, std=0.1), b_pre=normal(d, std=0.1))
        if case["op"] == "norm_train":
            s["dx_out"] = normal(n, d, std=0.7, dtype=st)
            s["dn"] = normal(n, d, std=0.9, dtype=br)
        return s
    h, nd, dt = case["hidden"], case["ndir"], DT[case["dtype"]]
    blocks = 2 if case["cell"] == "tied" else 3
    rows = case["batch"] if case["op"] == "step" else int(lengths_of(case).sum())
    # one projection's rows [f | z | i], the forget gates biased towards keeping
    pre = torch.empty((rows, blocks, nd, h), dtype=dt, device="cuda")
    pre[:, 0] = normal(rows, nd, h, mean=2.0, std=1.5, dtype=dt)
    pre[:, 1] = normal(rows, nd, h, dtype=dt)
    if blocks == 3:
        pre[:, 2] = normal(rows, nd, h, dtype=dt)
    s["pre"] = pre
    if case["op"] == "step":
        s["state"] = normal(case["slots"], h, std=0.7)
        r = random.Random(int(seed) * 31 + 5)
        slots = r.sample(range(case["slots"]), rows)
        slots = [-1 if k >= rows - case["idle"] else v for k, v in enumerate(slots)]
        s["slots"] = torch.tensor(slots, dtype=torch.int32, device="cuda")
        return s
    s["h0"] = normal(nd, case["batch"], h, std=0.7) if case["h0"] else None
    if case["op"] == "train":
        s["dy"] = normal(rows, nd, h, dtype=dt)
        s["dh_n"] = normal(nd, case["batch"], h) if case["h0"] else None
    return s


def prepare(case, seed):
    s = inputs(case, seed)
    s["case"] = case
    if case["op"] in ("norm", "norm_train"):
        s["x_out"], s["n"] = torch.empty_like(s["x"]), torch.empty_like(s["y"])
        if case["op"] == "norm_train":
            s["dx"], s["dy"] = torch.empty_like(s["x"]), torch.empty_like(s["y"])
            s["dgate"] = torch.empty_like(s["y"]) if s["gate"] is not None else None
            s["dp"] = {k: torch.empty_like(v) for k, v in s["p"].items()}
    else:
        s["y"] = torch.empty((s["pre"].shape[0], case["ndir"], case["hidden"]), dtype=s["pre"].dtype, device="cuda")
        if case["op"] == "step":
            s["new_state"] = torch.zeros((case["slots"] + 1, case["hidden"]), device="cuda")
        else:
            s["h_n"] = torch.empty((case["ndir"], case["batch"], case["hidden"]), device="cuda")
        if case["op"] == "train":
            s["dpre"] = torch.empty_like(s["pre"])
            s["dh0"] = torch.empty_like(s["h_n"]) if case["h0"] else None
    if own:     # the program's plan, operator descriptions and workspaces
        from padding_free_variable_gb300 import ops
        s["ops"] = ops
        if case["op"] in ("norm", "norm_train"):
            s["shape"] = ops.block_norm_shape(case["width"], case["kind"], case["gate"], case["branch"] == "bf16",
                                              case["stream"] == "bf16", case["branch"] == "bf16", EPS)
            s["stats"] = torch.empty((case["rows"], 4), device="cuda") if case["op"] == "norm_train" else None
            if case["op"] == "norm_train":
                s["scratch"] = torch.empty(ops.block_norm_scratch_bytes(s["shape"], case["rows"]), dtype=torch.uint8,
                                           device="cuda")
        else:
            s["shape"] = ops.glr_shape(case["hidden"], case["ndir"], case["dtype"] == "bf16", case["cell"])
            if case["op"] != "step":
                s["plan"] = ops.Plan(lengths_of(case))
            if case["op"] == "train":
                s["workspace"] = torch.empty(ops.glr_workspace_bytes(s["plan"], s["shape"]), dtype=torch.uint8, device="cuda")
    elif case["op"] in ("scan", "train"):
        lens = lengths_of(case)
        order, top, bs, off = packing(lens)
        t = np.repeat(np.arange(len(bs)), bs)
        j = np.arange(len(t)) - off[t]
        s["rows"] = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in
                     {"t": t, "j": j, "len": top[j], "off": off, "seq": order[j]}.items()}
        s["steps"], s["order"], s["top"] = len(bs), torch.from_numpy(order).cuda(), torch.from_numpy(top).cuda()
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if op in ("scan", "train"):
        return own_scan(s) if own else plain_scan(s)
    if op == "step":
        return own_step(s) if own else plain_step(s)
    return own_norm(s) if own else plain_norm(s)


def gates(pre):
    return pre[:, 0], pre[:, 1], pre[:, 2] if pre.shape[1] == 3 else None


def own_scan(s):
    ops, (f, z, i) = s["ops"], gates(s["pre"])
    ops.glr_forward(s["plan"], s["shape"], f, z, i, s["h0"], s["y"], s["h_n"], s.get("workspace"))
    if s["case"]["op"] == "scan":
        return {"y": s["y"], "h_n": s["h_n"]}
    ops.glr_backward(s["plan"], s["shape"], f, z, i, s["workspace"], s["dy"], s["dh_n"], *gates(s["dpre"]), s["dh0"])
    return {"y": s["y"], "h_n": s["h_n"], "dpre": s["dpre"], "dh0": s["dh0"]}


def own_step(s):
    f, z, i = gates(s["pre"])
    new = s["new_state"][:s["case"]["slots"]]
    s["ops"].glr_step(s["shape"], f, z, i, s["state"], new, s["y"], s["slots"])
    return {"y": s["y"], "state": new}


def own_norm(s):
    ops = s["ops"]
    ops.block_norm_forward(s["shape"], s["x"], s["y"], s["gate"], s["p"], s["x_out"], s["n"], s["stats"])
    if s["case"]["op"] == "norm":
        return {"x_out": s["x_out"], "n": s["n"]}
    ops.block_norm_backward(s["shape"], s["x"], s["y"], s["gate"], s["p"], s["stats"], s["dx_out"], s["dn"], s["dx"],
                            s["dy"], s["dgate"], s["dp"], s["scratch"])
    return {"x_out": s["x_out"], "n": s["n"], "dx": s["dx"], "dy": s["dy"], "dgate": s["dgate"], "dp": s["dp"]}


# The plain forms: elementary operations in 32 bits.  The recurrence is composed by doubling: after k rounds every row
# holds the affine map of its last 2^k frames, so ceil(log2 T) rounds over all rows replace T steps.

def gate_values(f, z, i):
    a, keep = torch.sigmoid(f), torch.sigmoid(-f)
    return a, keep, (keep if i is None else torch.sigmoid(i)) * z


def earlier(s, k, back=False):
    """[ndir * rows] index of the row k steps before each row in its direction's order (after, with `back`); -1 if none."""
    r, rows = s["rows"], s["rows"]["t"].numel()
    down = torch.where(r["t"] >= k, r["off"][(r["t"] - k).clamp_min(0)] + r["j"], -1)
    up = torch.where(r["t"] + k < r["len"], r["off"][(r["t"] + k).clamp_max(s["steps"] - 1)] + r["j"], -1)
    if s["case"]["ndir"] == 1:
        return up if back else down
    at = torch.cat([up, down] if back else [down, up])
    at[rows:] += rows * (at[rows:] >= 0)
    return at


def compose(s, a, b, back=False):
    k = 1
    while k < s["steps"]:
        p = earlier(s, k, back)
        ok = (p >= 0)[:, None]
        p = p.clamp_min(0)
        b = b + torch.where(ok, a * b[p], 0.0)
        a = torch.where(ok, a * a[p], a)
        k *= 2
    return b


def plain_scan(s):
    case, r = s["case"], s["rows"]
    nd, h, rows = case["ndir"], case["hidden"], s["pre"].shape[0]

    def flat(v):        # [rows, ndir, H] -> [ndir * rows, H] in 32 bits
        return None if v is None else v.float().transpose(0, 1).reshape(nd * rows, h)

    def packed(v):
        return v.view(nd, rows, h).transpose(0, 1)

    f, z, i = (flat(v) for v in gates(s["pre"]))
    a, keep, b = gate_values(f, z, i)
    dirs = torch.arange(nd, device="cuda").repeat_interleave(rows)
    seq = r["seq"].repeat(nd)
    before = earlier(s, 1)
    first = (before < 0)[:, None]
    start = s["h0"][dirs, seq] if s["h0"] is not None else torch.zeros((), device="cuda")
    hs = compose(s, a, b + torch.where(first, a * start, 0.0))
    # the states after each sequence's last frame (the initial ones, if it has none)
    live = s["top"] > 0
    ends = r["off"][(s["top"] - 1).clamp_min(0)] + torch.arange(len(s["top"]), device="cuda")
    ends = ends if nd == 1 else torch.stack([ends, torch.arange(len(s["top"]), device="cuda") + rows])
    ends = torch.where(live, ends, 0)
    h_n = torch.empty_like(s["h_n"])
    h_n[:, s["order"]] = torch.where(live[:, None], hs[ends].view(nd, -1, h),
                                     s["h0"][:, s["order"]] if s["h0"] is not None else 0.0)
    out = {"y": packed(hs).to(s["y"].dtype), "h_n": h_n}
    if case["op"] == "scan":
        return out
    after = earlier(s, 1, True)
    last = (after < 0)[:, None]
    g = flat(s["dy"]) + (torch.where(last, s["dh_n"][dirs, seq], 0.0) if s["dh_n"] is not None else 0.0)
    g = compose(s, torch.where(last, 0.0, a[after.clamp_min(0)]), g, True)
    h_prev = torch.where(first, start, hs[before.clamp_min(0)])
    if i is None:
        parts = [g * (h_prev - z) * a * keep, g * keep]
    else:
        si = torch.sigmoid(i)
        parts = [g * h_prev * a * keep, g * si, g * z * si * torch.sigmoid(-i)]
    out["dpre"] = torch.stack([packed(v) for v in parts], 1).to(s["dpre"].dtype)
    out["dh0"] = None
    if s["dh0"] is not None:
        begins = torch.arange(len(s["top"]), device="cuda")
        tail = torch.where(live, r["off"][(s["top"] - 1).clamp_min(0)] + begins, 0)
        begins = torch.where(live, begins, 0) if nd == 1 else torch.stack([torch.where(live, begins, 0), tail + rows])
        out["dh0"] = torch.empty_like(s["dh0"])
        out["dh0"][:, s["order"]] = torch.where(live[:, None], (a * g)[begins].view(nd, -1, h), s["dh_n"][:, s["order"]])
    return out


def plain_step(s):
    f, z, i = (None if v is None else v[:, 0].float() for v in gates(s["pre"]))
    a, _, b = gate_values(f, z, i)
    on = (s["slots"] >= 0)[:, None]
    at = torch.where(s["slots"] >= 0, s["slots"], s["case"]["slots"]).long()
    h = a * s["state"][at.clamp_max(s["case"]["slots"] - 1)] + b
    s["new_state"][at] = h
    return {"y": torch.where(on, h, 0.0).to(s["y"].dtype)[:, None], "state": s["new_state"][:s["case"]["slots"]]}


def plain_norm(s):
    case, p = s["case"], s["p"]
    layer = case["kind"] == "layer"

    def norm(v):
        v = v - v.mean(1, keepdim=True) if layer else v
        r = 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
        return v * r, r

    def through(hat, r, d):         # the norm's backward pass
        d = d - hat * (d * hat).mean(1, keepdim=True) - (d.mean(1, keepdim=True) if layer else 0.0)
        return r * d

    x, y = s["x"].float(), s["y"].float()
    yh, ry = norm(y)
    v = yh * p["w_post"] + (p["b_post"] if layer else 0.0)
    q = s["gate"].float() if s["gate"] is not None else None
    sg = torch.sigmoid(q) if q is not None else None
    act = 1.0 if q is None else sg if case["gate"] == "sigmoid" else q * sg
    x1 = x + p["scale"] * v * act
    xh, rx = norm(x1)
    out = {"x_out": x1.to(s["x"].dtype), "n": (xh * p["w_pre"] + (p["b_pre"] if layer else 0.0)).to(s["y"].dtype)}
    if case["op"] == "norm":
        return out
    dn = s["dn"].float()
    dx = s["dx_out"].float() + through(xh, rx, dn * p["w_pre"])
    du = p["scale"] * dx
    dv = du * act
    out["dx"], out["dy"] = dx.to(s["x"].dtype), through(yh, ry, dv * p["w_post"]).to(s["y"].dtype)
    out["dgate"] = None
    if q is not None:
        slope = sg * (1.0 - sg) if case["gate"] == "sigmoid" else sg * (1.0 + q * (1.0 - sg))
        out["dgate"] = (du * v * slope).to(s["y"].dtype)
    out["dp"] = {"w_post": (dv * yh).sum(0), "scale": (dx * v * act).sum(0), "w_pre": (dn * xh).sum(0)}
    if layer:
        out["dp"].update(b_post=dv.sum(0), b_pre=dn.sum(0))
    return out


# ------------------------------------------------------------------ what a pass has to move

def work(case):
    def size(dtype):
        return 2 if dtype == "bf16" else 4

    op = case["op"]
    if op in ("norm", "norm_train"):
        n, d, br, st = case["rows"], case["width"], size(case["branch"]), size(case["stream"])
        gate = 0 if case["gate"] == "none" else 1
        vecs = (5 if case["kind"] == "layer" else 3) * d * 4
        if op == "norm":        # x, y, gate in; x', n out
            return {"bytes": n * d * (2 * st + (2 + gate) * br) + vecs, "flops": 14.0 * n * d}
        # x, y, gate, dx', dn in; x', n, dx, dy, dgate out
        return {"bytes": n * d * (4 * st + (4 + 2 * gate) * br) + 2 * vecs, "flops": 44.0 * n * d}
    e, h = size(case["dtype"]), case["hidden"]
    blocks = 2 if case["cell"] == "tied" else 3
    if op == "step":
        live = case["batch"] - case["idle"]
        return {"bytes": live * h * (blocks * e + 8) + case["batch"] * (h * e + 4), "flops": 10.0 * live * h}
    n = int(lengths_of(case).sum()) * case["ndir"] * h
    state = case["ndir"] * case["batch"] * h * 4
    if op == "scan":            # the gates (and h_0) in; h and h_n out
        return {"bytes": n * (blocks + 1) * e + state * (2 if case["h0"] else 1), "flops": 10.0 * n}
    # the gates, dy (and h_0, dh_n) in; h, h_n and the gates' gradients (and dh_0) out
    return {"bytes": n * (2 * blocks + 2) * e + state * (4 if case["h0"] else 1), "flops": 30.0 * n}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    """Frame by frame from the definition, in 64 bits; gradients by the chain rule, frame by frame backwards."""
    s = inputs(case, seed)
    sig = lambda v: 1.0 / (1.0 + torch.exp(-v))  # noqa: E731
    if case["op"] in ("norm", "norm_train"):
        n = s["x"].shape[0]
        d = case["width"]
        x, y = s["x"].double(), s["y"].double()
        p = {k: v.double() for k, v in s["p"].items()}
        zero = torch.zeros(d, dtype=torch.float64, device="cuda")
        q = s["gate"].double() if s["gate"] is not None else None
        act, slope = torch.ones_like(y), torch.zeros_like(y)
        if case["gate"] == "sigmoid":
            act = sig(q)
            slope = act * sig(-q)
        elif case["gate"] == "silu":
            act = q * sig(q)
            slope = sig(q) + q * sig(q) * sig(-q)
        centre = 1.0 if case["kind"] == "layer" else 0.0
        my = centre * y.sum(1, keepdim=True) / d
        sy = torch.sqrt(((y - my) ** 2).sum(1, keepdim=True) / d + EPS)
        v = (y - my) / sy * p["w_post"] + p.get("b_post", zero)
        x1 = x + p["scale"] * v * act
        mx = centre * x1.sum(1, keepdim=True) / d
        sx = torch.sqrt(((x1 - mx) ** 2).sum(1, keepdim=True) / d + EPS)
        out = {"x_out": x1, "n": (x1 - mx) / sx * p["w_pre"] + p.get("b_pre", zero)}
        if case["op"] == "norm":
            return out
        dn = s["dn"].double()
        t = dn * p["w_pre"]
        t = t - centre * t.sum(1, keepdim=True) / d
        dx = s["dx_out"].double() + t / sx - (x1 - mx) * (t * (x1 - mx)).sum(1, keepdim=True) / (d * sx ** 3)
        t = dx * p["scale"] * act * p["w_post"]
        t = t - centre * t.sum(1, keepdim=True) / d
        out["dx"] = dx
        out["dy"] = t / sy - (y - my) * (t * (y - my)).sum(1, keepdim=True) / (d * sy ** 3)
        out["dgate"] = dx * p["scale"] * v * slope if q is not None else None
        out["dp"] = {"w_post": (dx * p["scale"] * act * (y - my) / sy).sum(0), "scale": (dx * v * act).sum(0),
                     "w_pre": (dn * (x1 - mx) / sx).sum(0)}
        if case["kind"] == "layer":
            out["dp"].update(b_post=(dx * p["scale"] * act).sum(0), b_pre=dn.sum(0))
        assert out["dx"].shape[0] == n
        return out
    pre = s["pre"].double()
    f, z = pre[:, 0], pre[:, 1]
    a = sig(f)
    u = sig(-f) if case["cell"] == "tied" else sig(pre[:, 2])
    if case["op"] == "step":
        y = torch.zeros_like(z)
        new = torch.zeros((case["slots"], case["hidden"]), dtype=torch.float64, device="cuda")
        on = torch.nonzero(s["slots"] >= 0)[:, 0]
        at = s["slots"][on].long()
        y[on, 0] = a[on, 0] * s["state"].double()[at] + u[on, 0] * z[on, 0]
        new[at] = y[on, 0]
        return {"y": y, "state": new}
    nd, nb, h = case["ndir"], case["batch"], case["hidden"]
    order, top, bs, off = packing(lengths_of(case))
    steps = len(bs)
    order = torch.from_numpy(order).cuda()
    b = u * z
    hs, prev = torch.empty_like(z), torch.empty_like(z)
    zero = torch.zeros((nd, nb, h), dtype=torch.float64, device="cuda")
    state = s["h0"].double()[:, order] if s["h0"] is not None else zero.clone()
    for d in range(nd):
        for t in (range(steps) if d == 0 else range(steps - 1, -1, -1)):
            m, r = int(bs[t]), slice(int(off[t]), int(off[t + 1]))
            prev[r, d] = state[d, :m]
            state[d, :m] = torch.addcmul(b[r, d], a[r, d], state[d, :m])
            hs[r, d] = state[d, :m]
    h_n = torch.empty_like(state)
    h_n[:, order] = state
    if case["op"] == "scan":
        return {"y": hs, "h_n": h_n}
    g = torch.empty_like(z)
    dy = s["dy"].double()
    err = s["dh_n"].double()[:, order] if s["dh_n"] is not None else zero.clone()
    for d in range(nd):
        for t in (range(steps - 1, -1, -1) if d == 0 else range(steps)):
            m, r = int(bs[t]), slice(int(off[t]), int(off[t + 1]))
            g[r, d] = dy[r, d] + err[d, :m]
            err[d, :m] = a[r, d] * g[r, d]
    if case["cell"] == "tied":
        parts = [g * (prev - z) * a * sig(-f), g * u]
    else:
        parts = [g * prev * a * sig(-f), g * u, g * z * u * sig(-pre[:, 2])]
    dh0 = torch.empty_like(err)
    dh0[:, order] = err
    return {"y": hs, "h_n": h_n, "dpre": torch.stack(parts, 1), "dh0": dh0 if s["h0"] is not None else None}
