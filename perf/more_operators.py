"""Linear attention over packed rows and the norms and rotations of its queries and keys, as a user's program calls them,
with their plain forms, for timing and comparison.

Row ``off[t] + j`` of a packed batch is frame t of the j-th longest sequence; a second direction runs from the last frame
to the first.

attend / attend_train   per head, with a decay 0 < e^l <= 1 of its own and S_0 = 0 unless given:
                        S_t = e^l S_{t-1} + k_t v_t^T,  o_t = scale * S_t^T q_t.  "attend" is the forward pass (o of every
                        frame and the final states), "attend_train" the forward pass and the gradients of q, k, v and S_0.
attend_step             the same for one new frame of each of many streams, whose states lie in a cache of slots.
turn / turn_train       what stands before it: each head's query and key is normalised over the head, weighted, and its first
                        ``rotary`` values are rotated pairwise by position times the pair's frequency.  "turn" is the forward
                        pass, "turn_train" the forward pass and every gradient.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
CHUNK = 64


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a few short words: the smallest call, where the launch is the cost
        {"name": "attend-words-f32", "op": "attend", "dtype": "f32", "ndir": 1, "heads": 2, "dk": 16, "dv": 16, "batch": 8,
         "dist": "uniform", "lo": 5, "hi": 40, "empty": 0, "s0": False, "lens_seed": 1001},
        # the library's headline batch (64 utterances, 40 k frames, 512 channels in both directions) in bf16
        {"name": "attend-utterances-bf16", "op": "attend", "dtype": "bf16", "ndir": 2, "heads": 8, "dk": 64, "dv": 64,
         "batch": 64, "dist": "lognormal", "lo": 100, "hi": 2000, "empty": 0, "s0": False, "lens_seed": 1003},
        # one recording of 65 536 frames of 1 024 channels, not cut into segments, its state carried in
        {"name": "attend-recording-bf16", "op": "attend", "dtype": "bf16", "ndir": 1, "heads": 8, "dk": 128, "dv": 128,
         "batch": 1, "dist": "uniform", "lo": 65536, "hi": 65536, "empty": 0, "s0": True, "lens_seed": 7},
        # odd head sizes (no vector access lines up), sequences of no frame and of one, a carried state
        {"name": "attend-odd-f32", "op": "attend", "dtype": "f32", "ndir": 2, "heads": 3, "dk": 37, "dv": 53, "batch": 37,
         "dist": "uniform", "lo": 1, "hi": 700, "empty": 3, "s0": True, "lens_seed": 11},
        # a training step's pass on the headline batch
        {"name": "attend-train-utterances-bf16", "op": "attend_train", "dtype": "bf16", "ndir": 2, "heads": 8, "dk": 64,
         "dv": 64, "batch": 64, "dist": "lognormal", "lo": 100, "hi": 2000, "empty": 0, "s0": False, "lens_seed": 1003},
        # a batch of 256 utterances of a 1 024 wide layer, wide heads
        {"name": "attend-train-wide-bf16", "op": "attend_train", "dtype": "bf16", "ndir": 1, "heads": 8, "dk": 128, "dv": 128,
         "batch": 256, "dist": "lognormal", "lo": 20, "hi": 200, "empty": 0, "s0": False, "lens_seed": 1005},
        # two long fp32 sequences: few heads to do side by side; states in, their gradients out
        {"name": "attend-train-long-f32", "op": "attend_train", "dtype": "f32", "ndir": 1, "heads": 8, "dk": 32, "dv": 64,
         "batch": 2, "dist": "uniform", "lo": 10001, "hi": 20001, "empty": 0, "s0": True, "lens_seed": 13},
        # streaming recognition: one new frame of eight streams
        {"name": "attend-step-streams-bf16", "op": "attend_step", "dtype": "bf16", "ndir": 1, "heads": 8, "dk": 64, "dv": 64,
         "batch": 8, "slots": 16, "idle": 1, "s0": True},
        # a server's tick over a thousand streams of wide heads
        {"name": "attend-step-server-f32", "op": "attend_step", "dtype": "f32", "ndir": 1, "heads": 8, "dk": 128, "dv": 128,
         "batch": 1024, "slots": 1200, "idle": 27, "s0": True},
        # the same tick's queries and keys: few rows at far positions, latency counts
        {"name": "turn-streams-bf16", "op": "turn", "kind": "rms", "dtype": "bf16", "qh": 8, "kh": 8, "d": 64, "rotary": 64,
         "layout": "half", "gap": 512, "rows": 8, "reach": 65536},
        # the headline batch's queries and keys, positions from the packing, part of each head rotated
        {"name": "turn-train-utterances-bf16", "op": "turn_train", "kind": "rms", "dtype": "bf16", "qh": 16, "kh": 16, "d": 64,
         "rotary": 32, "layout": "half", "gap": 1024, "batch": 64, "dist": "lognormal", "lo": 100, "hi": 2000, "empty": 0,
         "lens_seed": 1003},
        # odd heads, fewer of them for the keys, interleaved pairs, centred norms, positions of a long stream
        {"name": "turn-train-odd-f32", "op": "turn_train", "kind": "layer", "dtype": "f32", "qh": 5, "kh": 2, "d": 74,
         "rotary": 38, "layout": "interleaved", "gap": 3, "rows": 9564, "reach": 4000000},
    ]


def draw(rng):
    """One more case: sizes of heads, batches and lengths spread over their logarithms, odd ones among them."""
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))

    op = rng.choice(["attend", "attend", "attend_train", "attend_train", "attend_step", "turn", "turn_train"])
    dtype = rng.choice(["f32", "bf16"])
    values = math.exp(rng.uniform(math.log(2e4), math.log(4e7 if dtype == "bf16" else 1.5e7)))     # of one operand
    if op in ("turn", "turn_train"):
        d = log(4, 256)
        d = max(8, d // 8 * 8) if rng.random() < 0.7 else d
        kh = log(1, 16)
        qh = kh * rng.choice([1, 1, 1, 2, 4])
        rotary = rng.choice([0, d // 2 * 2, d // 2 * 2, d // 4 * 2])
        case = {"op": op, "kind": rng.choice(["none", "rms", "rms", "layer"]), "dtype": dtype, "qh": qh, "kh": kh, "d": d,
                "rotary": rotary, "layout": rng.choice(["half", "interleaved"]), "gap": rng.choice([0, kh * d, kh * d, 5])}
        rows = max(1, min(150000, int(values / ((qh + kh) * d))))
        if rng.random() < 0.5:
            return dict(case, rows=rows, reach=log(16, 10000000))
        batch = min(rows, log(1, 200))
        mean = max(1, rows // batch)
        return dict(case, batch=batch, dist="uniform", lo=max(1, mean // 4), hi=max(1, mean * 2 - mean // 4), empty=0,
                    lens_seed=rng.randrange(1 << 30))
    dk, dv = log(8, 128), log(8, 128)
    if rng.random() < 0.7:
        dk, dv = dk // 8 * 8, dv // 8 * 8
    if rng.random() < 0.5:
        dv = dk
    case = {"op": op, "dtype": dtype, "heads": log(1, 16), "dk": dk, "dv": dv}
    if op == "attend_step":
        batch = max(1, min(4096, int(values * 3 / (case["heads"] * dk * dv))))
        return dict(case, ndir=1, batch=batch, slots=batch + rng.randrange(0, batch // 4 + 8), idle=rng.randrange(0, batch // 8 + 1),
                    s0=True)
    case["ndir"] = rng.choice([1, 2])
    width = case["heads"] * case["ndir"] * max(dk, dv)
    batch = log(1, max(1, min(256, int(1.5e7 / (width * min(dk, dv))))))
    mean = max(1, min(65536, int(values / (width * batch))))
    if batch == 1 or rng.random() < 0.2:
        lo = hi = mean
        dist = "uniform"
    else:
        dist = rng.choice(["uniform", "lognormal"])
        lo, hi = max(1, mean // 6), max(1, mean * 2 - mean // 6)
    case.update(batch=batch, dist=dist, lo=lo, hi=min(hi, 65536), s0=rng.random() < 0.5,
                empty=rng.choice([0, 0, 0, 2]) if batch > 4 else 0, lens_seed=rng.randrange(1 << 30))
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


def rows_of(case):
    return int(lengths_of(case).sum()) if "batch" in case and "lens_seed" in case else case.get("rows", case.get("batch"))


# ------------------------------------------------------------------ inputs

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EXTEND = {"factor": 4.0, "trained": 2048}           # the long-context scaling of positions past a trained length


def inputs(case, seed):
    """The tensors of a call, on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)

    def normal(*shape, mean=0.0, std=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(dtype)

    s, dt, n = {}, DT[case["dtype"]], rows_of(case)
    if case["op"] in ("turn", "turn_train"):
        qh, kh, d = case["qh"], case["kh"], case["d"]
        # a projection's rows [q | k | whatever else it makes]
        s["pre"] = normal(n, (qh + kh) * d + case["gap"], mean=0.05, std=1.4, dtype=dt)
        s["wq"], s["wk"] = normal(d, mean=1.0, std=0.2), normal(d, mean=1.0, std=0.2)
        if case["kind"] == "none":
            s["wq"] = s["wk"] = None
        s["positions"] = None
        if "reach" in case:
            s["positions"] = torch.randint(0, case["reach"], (n,), generator=g, device="cuda", dtype=torch.int32)
        if case["op"] == "turn_train":
            s["dq_out"], s["dk_out"] = normal(n, qh, d, dtype=dt), normal(n, kh, d, dtype=dt)
        return s
    nd, h, dk, dv = case["ndir"], case["heads"], case["dk"], case["dv"]
    # one projection's rows [q | k | v], the keys scaled so that the states stay near 1
    pre = torch.empty((n, nd * h * (2 * dk + dv)), dtype=dt, device="cuda")
    cut = nd * h * dk
    pre[:, :cut] = normal(n, cut, dtype=dt)
    pre[:, cut:2 * cut] = normal(n, cut, std=dk ** -0.5, dtype=dt)
    pre[:, 2 * cut:] = normal(n, nd * h * dv, dtype=dt)
    s["pre"] = pre
    # each head's memory: from a few frames to a few thousand
    s["log_decay"] = torch.tensor([[math.log1p(-2.0 ** -(2 + 9.0 * (e + 0.5 * i) / h)) for e in range(h)] for i in range(nd)],
                                  dtype=torch.float32, device="cuda")
    if case["op"] == "attend_step":
        s["state"] = normal(case["slots"], h, dk, dv, std=0.7)
        r = random.Random(int(seed) * 31 + 5)
        slots = r.sample(range(case["slots"]), n)
        slots = [-1 if k >= n - case["idle"] else v for k, v in enumerate(slots)]
        s["slots"] = torch.tensor(slots, dtype=torch.int32, device="cuda")
        return s
    s["s0"] = normal(nd, case["batch"], h, dk, dv, std=0.7) if case["s0"] else None
    if case["op"] == "attend_train":
        s["dy"] = normal(n, nd, h, dv, dtype=dt)
        s["ds_n"] = normal(nd, case["batch"], h, dk, dv) if case["s0"] else None
    return s


def split(case, pre):
    """q, k, v [rows, ndir, heads, size] of a projection's rows."""
    nd, h, dk, dv = case["ndir"], case["heads"], case["dk"], case["dv"]
    cut = nd * h * dk
    return (pre[:, :cut].unflatten(1, (nd, h, dk)), pre[:, cut:2 * cut].unflatten(1, (nd, h, dk)),
            pre[:, 2 * cut:].unflatten(1, (nd, h, dv)))


def pair(case, pre):
    """q and k [rows, heads, d] of a projection's rows."""
    qh, kh, d = case["qh"], case["kh"], case["d"]
    return pre[:, :qh * d].unflatten(1, (qh, d)), pre[:, qh * d:(qh + kh) * d].unflatten(1, (kh, d))


def scale_of(case):
    return case["dk"] ** -0.5


def frequencies(case):
    """Radians a position of each pair: base^(-2i/rotary), those that turn less than once within the trained length slowed
    down by the factor."""
    r = case["rotary"]
    f = 10000.0 ** (-np.arange(0, r, 2, dtype=np.float64) / max(r, 1))
    return np.where(f * EXTEND["trained"] < 2 * math.pi, f / EXTEND["factor"], f)


def prepare(case, seed):
    s = inputs(case, seed)
    s["case"] = case
    turn = case["op"] in ("turn", "turn_train")
    n, dt = rows_of(case), DT[case["dtype"]]
    if turn:
        s["out"] = [torch.empty((n, h, case["d"]), dtype=dt, device="cuda") for h in (case["qh"], case["kh"])]
        if case["op"] == "turn_train":
            s["dpre"] = torch.zeros_like(s["pre"])
            s["dw"] = [torch.empty_like(w) if w is not None else None for w in (s["wq"], s["wk"])]
    else:
        nd, h, dk, dv = case["ndir"], case["heads"], case["dk"], case["dv"]
        s["y"] = torch.empty((n, nd, h, dv), dtype=dt, device="cuda")
        if case["op"] == "attend_step":
            s["new_state"] = torch.zeros((case["slots"] + 1, h, dk, dv), device="cuda")
        else:
            s["s_n"] = torch.empty((nd, case["batch"], h, dk, dv), device="cuda")
        if case["op"] == "attend_train":
            s["dpre"] = torch.empty_like(s["pre"])
            s["ds0"] = torch.empty_like(s["s_n"]) if case["s0"] else None
    packed = "lens_seed" in case
    if own:     # the program's plan, operator descriptions and workspaces
        from padding_free_variable_gb300 import ops
        s["ops"] = ops
        s["plan"] = ops.Plan(lengths_of(case)) if packed else None
        if turn:
            s["shape"] = ops.qk_norm_shape(case["qh"], case["kh"], case["d"], case["kind"], case["rotary"], case["layout"],
                                           case["dtype"] == "bf16", EPS)
            s["table"] = ops.rotary_table(frequencies(case)) if case["rotary"] else None
            if case["op"] == "turn_train":
                s["scratch"] = torch.empty(ops.qk_norm_scratch_bytes(s["shape"], n), dtype=torch.uint8, device="cuda")
        else:
            s["shape"] = ops.la_shape(case["heads"], case["dk"], case["dv"], case["ndir"], case["dtype"] == "bf16",
                                      scale_of(case))
        return s
    if turn:
        s["freq"] = torch.from_numpy(frequencies(case)).cuda()
    if packed:
        order, top, bs, off = packing(lengths_of(case))
        steps = len(bs)
        if turn:
            s["positions"] = torch.from_numpy(np.repeat(np.arange(steps), bs)).cuda()
        else:
            # [ndir, batch (caller order), chunks * CHUNK] row of each step; rows past a sequence's end: one of zeros
            t = np.arange(max(1, -(-steps // CHUNK)) * CHUNK)
            at = np.full((case["ndir"], len(top), len(t)), n, dtype=np.int64)
            for j, length in enumerate(top):
                rows = off[t[:length]] + j
                at[0, order[j], :length] = rows
                if case["ndir"] == 2:
                    at[1, order[j], :length] = rows[::-1]
            s["at"] = torch.from_numpy(at).cuda()
            s["len"] = torch.from_numpy(lengths_of(case)).cuda()
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if op in ("attend", "attend_train"):
        return own_attend(s) if own else plain_attend(s)
    if op == "attend_step":
        return own_step(s) if own else plain_step(s)
    return own_turn(s) if own else plain_turn(s)


def own_attend(s):
    ops, case = s["ops"], s["case"]
    q, k, v = split(case, s["pre"])
    ops.la_forward(s["plan"], s["shape"], q, k, v, s["log_decay"], s["s0"], s["y"], s["s_n"])
    if case["op"] == "attend":
        return {"y": s["y"], "s_n": s["s_n"]}
    ops.la_backward(s["plan"], s["shape"], q, k, v, s["log_decay"], s["s0"], s["dy"], s["ds_n"], *split(case, s["dpre"]),
                    s["ds0"])
    return {"y": s["y"], "s_n": s["s_n"], "dpre": s["dpre"], "ds0": s["ds0"]}


def own_step(s):
    new = s["new_state"][:s["case"]["slots"]]
    s["ops"].la_step(s["shape"], *split(s["case"], s["pre"]), s["log_decay"], s["state"], new, s["y"], s["slots"])
    return {"y": s["y"], "state": new}


def own_turn(s):
    ops, case = s["ops"], s["case"]
    q, k = pair(case, s["pre"])
    ops.qk_norm_forward(s["shape"], q, k, s["wq"], s["wk"], s["table"], s["positions"], *s["out"], plan=s["plan"])
    if case["op"] == "turn":
        return {"q": s["out"][0], "k": s["out"][1]}
    ops.qk_norm_backward(s["shape"], q, k, s["wq"], s["wk"], s["table"], s["positions"], s["dq_out"], s["dk_out"],
                         *pair(case, s["dpre"]), *s["dw"], s["scratch"], plan=s["plan"])
    return {"q": s["out"][0], "k": s["out"][1], "dpre": s["dpre"], "dw": s["dw"]}


# The plain forms: elementary operations in 32 bits.  Sequences are laid out side by side, padded, in chunks of CHUNK
# steps: within a chunk every pair of steps, between chunks the state.

def plain_attend(s):
    case = s["case"]
    nd, h, dk, dv = case["ndir"], case["heads"], case["dk"], case["dv"]
    n, c = s["pre"].shape[0], scale_of(case)
    q, k, v = split(case, s["pre"])
    train = case["op"] == "attend_train"
    y = torch.zeros((n + 1, nd, h, dv), dtype=s["y"].dtype, device="cuda")
    s_n = torch.empty_like(s["s_n"])
    grads = [torch.zeros((n + 1, nd, h, m), dtype=y.dtype, device="cuda") for m in (dk, dk, dv)] if train else None
    ds0 = torch.empty_like(s_n) if train else None
    i = torch.arange(CHUNK, device="cuda")
    for d in range(nd):
        at = s["at"][d]
        b, m = at.shape[0], at.shape[1] // CHUNK
        live = (at < n).view(b, m, 1, CHUNK, 1)

        def chunks(x):      # [rows, nd, h, w] -> [b, chunks, h, CHUNK, w] in 32 bits, zero past a sequence's end
            w = x.shape[-1]
            rows = x[:, d][at.clamp_max(n - 1).flatten()].float().view(b, m, CHUNK, h, w).transpose(2, 3)
            return torch.where(live, rows, 0.0)

        def rows(x, out):   # the way back
            w = x.shape[-1]
            out[:, d].index_copy_(0, at.flatten(), x.transpose(2, 3).reshape(b * m * CHUNK, h, w).to(out.dtype))

        ld = s["log_decay"][d][:, None, None]                                       # [h, 1, 1]
        near = i[:, None] - i[None, :]
        inside = torch.where(near >= 0, torch.exp(ld * near.clamp_min(0)), 0.0)     # [h, CHUNK, CHUNK]
        size = (s["len"][:, None] - CHUNK * torch.arange(m, device="cuda")).clamp(0, CHUNK)     # [b, m] steps of a chunk
        keep = torch.exp(s["log_decay"][d] * size[..., None])[..., None, None]      # [b, m, h, 1, 1]
        left = (size[:, :, None, None, None] - 1 - i[None, None, None, :, None]).clamp_min(0)
        to_end = torch.exp(ld * left)                                               # [b, m, h, CHUNK, 1]
        from_start = torch.exp(ld * (i + 1)[None, :, None])                         # [h, CHUNK, 1]
        qs, ks, vs = chunks(q), chunks(k), chunks(v)
        kv = (ks * to_end).transpose(-1, -2) @ vs
        state = s["s0"][d] if s["s0"] is not None else torch.zeros((b, h, dk, dv), device="cuda")
        before = torch.empty((b, m, h, dk, dv), device="cuda")
        for e in range(m):
            before[:, e] = state
            state = keep[:, e] * state + kv[:, e]
        s_n[d] = state
        rows(c * (((qs @ ks.transpose(-1, -2)) * inside) @ vs + from_start * (qs @ before)), y)
        if not train:
            continue
        dy = chunks(s["dy"])
        dkv = (qs * from_start).transpose(-1, -2) @ dy
        err = s["ds_n"][d] if s["ds_n"] is not None else torch.zeros((b, h, dk, dv), device="cuda")
        after = torch.empty((b, m, h, dk, dv), device="cuda")
        for e in range(m - 1, -1, -1):
            after[:, e] = err
            err = keep[:, e] * err + c * dkv[:, e]
        ds0[d] = err
        p = (qs @ ks.transpose(-1, -2)) * inside
        dp = (dy @ vs.transpose(-1, -2)) * inside
        rows(c * (dp @ ks + from_start * (dy @ before.transpose(-1, -2))), grads[0])
        rows(c * (dp.transpose(-1, -2) @ qs) + to_end * (vs @ after.transpose(-1, -2)), grads[1])
        rows(c * (p.transpose(-1, -2) @ dy) + to_end * (ks @ after), grads[2])
    out = {"y": y[:n], "s_n": s_n}
    if train:
        out["dpre"] = torch.cat([g[:n].flatten(1) for g in grads], 1)
        out["ds0"] = ds0 if case["s0"] else None
    return out


def plain_step(s):
    case = s["case"]
    q, k, v = (x[:, 0].float() for x in split(case, s["pre"]))
    on = (s["slots"] >= 0)[:, None, None]
    at = torch.where(s["slots"] >= 0, s["slots"], case["slots"]).long()
    old = s["state"][at.clamp_max(case["slots"] - 1)]
    new = torch.exp(s["log_decay"][0])[:, None, None] * old + k[..., None] * v[..., None, :]
    s["new_state"][at] = new
    y = scale_of(case) * (q[..., None] * new).sum(-2)
    return {"y": torch.where(on, y, 0.0).to(s["y"].dtype)[:, None], "state": s["new_state"][:case["slots"]]}


def plain_turn(s):
    case = s["case"]
    d, r = case["d"], case["rotary"]
    angle = s["positions"].double()[:, None] * s["freq"] if r else None

    def first_second(x):
        return (x[..., :r // 2], x[..., r // 2:r]) if case["layout"] == "half" else (x[..., 0:r:2], x[..., 1:r:2])

    def turned(x, way):
        if not r:
            return x
        co, si = torch.cos(angle).float()[:, None], way * torch.sin(angle).float()[:, None]
        a, b = first_second(x)
        out = x.clone()
        a1, b1 = first_second(out)
        a1.copy_(a * co - b * si)
        b1.copy_(a * si + b * co)
        return out

    def hat_of(x):
        if case["kind"] == "none":
            return x, 1.0
        x = x - x.mean(-1, keepdim=True) if case["kind"] == "layer" else x
        rs = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        return x * rs, rs

    outs, grads, dws = [], [], []
    for x, w, dy in zip(pair(case, s["pre"]), (s["wq"], s["wk"]), (s.get("dq_out"), s.get("dk_out"))):
        hat, rs = hat_of(x.float())
        outs.append(turned(hat if w is None else hat * w, 1.0).to(x.dtype))
        if dy is None:
            continue
        g = turned(dy.float(), -1.0)
        dws.append((g * hat).sum((0, 1)) if w is not None else None)
        g = g if w is None else g * w
        if case["kind"] != "none":
            g = g - hat * (g * hat).mean(-1, keepdim=True) - (g.mean(-1, keepdim=True) if case["kind"] == "layer" else 0.0)
            g = g * rs
        grads.append(g.to(x.dtype).flatten(1))
    out = {"q": outs[0], "k": outs[1]}
    if grads:
        s["dpre"][:, :(case["qh"] + case["kh"]) * d] = torch.cat(grads, 1)
        out["dpre"], out["dw"] = s["dpre"], dws
    return out


# ------------------------------------------------------------------ what a pass has to move

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    n = rows_of(case)
    if case["op"] in ("turn", "turn_train"):
        values = n * (case["qh"] + case["kh"]) * case["d"]
        extra = (4 * n if "reach" in case else 0) + (0 if case["kind"] == "none" else 8 * case["d"]) + 8 * (case["rotary"] // 2)
        if case["op"] == "turn":        # q, k in; q', k' out
            return {"bytes": 2 * values * e + extra, "flops": 10.0 * values}
        return {"bytes": 4 * values * e + 2 * extra, "flops": 30.0 * values}    # q, k, dq', dk' in; q', k', dq, dk out
    h, dk, dv, nd = case["heads"], case["dk"], case["dv"], case["ndir"]
    if case["op"] == "attend_step":
        live = case["batch"] - case["idle"]
        return {"bytes": live * h * (8 * dk * dv + e * (2 * dk + dv)) + case["batch"] * (h * dv * e + 4),
                "flops": 5.0 * live * h * dk * dv}
    state = nd * case["batch"] * h * dk * dv * 4
    per = n * nd * h
    if case["op"] == "attend":          # q, k, v (and s_0) in; o and s_n out
        return {"bytes": per * (2 * dk + 2 * dv) * e + state * (2 if case["s0"] else 1), "flops": 4.0 * per * dk * dv}
    # q, k, v, dy (and s_0, ds_n) in; o, s_n and the gradients of q, k, v (and s_0) out
    return {"bytes": per * (4 * dk + 4 * dv) * e + state * (4 if case["s0"] else 1), "flops": 14.0 * per * dk * dv}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    """Frame by frame from the definition, in 64 bits; gradients by the chain rule, frame by frame backwards."""
    s = inputs(case, seed)
    if case["op"] in ("turn", "turn_train"):
        return exact_turn(case, s)
    h, dk, dv = case["heads"], case["dk"], case["dv"]
    c = float(scale_of(case))
    lam = torch.exp(s["log_decay"].double())[..., None, None]          # [nd, h, 1, 1]
    q, k, v = split(case, s["pre"].double())
    if case["op"] == "attend_step":
        y = torch.zeros_like(v)
        new = torch.zeros((case["slots"], h, dk, dv), dtype=torch.float64, device="cuda")
        on = torch.nonzero(s["slots"] >= 0)[:, 0]
        at = s["slots"][on].long()
        st = lam[0] * s["state"].double()[at] + torch.einsum("rhk,rhv->rhkv", k[on, 0], v[on, 0])
        new[at] = st
        y[on, 0] = c * torch.einsum("rhk,rhkv->rhv", q[on, 0], st)
        return {"y": y, "state": new}
    nd, nb = case["ndir"], case["batch"]
    order, top, bs, off = packing(lengths_of(case))
    steps = len(bs)
    if steps * nd * (2 if case["op"] == "attend_train" else 1) > 200000:
        return None
    order = torch.from_numpy(order).cuda()
    train = case["op"] == "attend_train"
    y, s_n = torch.empty_like(v), torch.empty((nd, nb, h, dk, dv), dtype=torch.float64, device="cuda")
    dq, dkey, dval = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dy = s["dy"].double() if train else None
    ds0 = torch.empty_like(s_n)
    for d in range(nd):
        state = torch.zeros((nb, h, dk, dv), dtype=torch.float64, device="cuda")
        if s["s0"] is not None:
            state = s["s0"][d].double()[order]
        for t in (range(steps) if d == 0 else range(steps - 1, -1, -1)):
            m, r = int(bs[t]), slice(int(off[t]), int(off[t + 1]))
            st = state[:m]
            st.mul_(lam[d]).addcmul_(k[r, d][..., None], v[r, d][..., None, :])
            y[r, d] = c * (q[r, d][..., None, :] @ st)[..., 0, :]
            if train:
                dq[r, d] = c * (st @ dy[r, d][..., None])[..., 0]
        s_n[d][order] = state
        if not train:
            continue
        err = torch.zeros_like(state)
        if s["ds_n"] is not None:
            err = s["ds_n"][d].double()[order]
        for t in (range(steps - 1, -1, -1) if d == 0 else range(steps)):
            m, r = int(bs[t]), slice(int(off[t]), int(off[t + 1]))
            e = err[:m]
            e.addcmul_(c * q[r, d][..., None], dy[r, d][..., None, :])
            dkey[r, d] = (e @ v[r, d][..., None])[..., 0]
            dval[r, d] = (k[r, d][..., None, :] @ e)[..., 0, :]
            e.mul_(lam[d])
        ds0[d][order] = err
    if not train:
        return {"y": y, "s_n": s_n}
    return {"y": y, "s_n": s_n, "dpre": torch.cat([x.flatten(1) for x in (dq, dkey, dval)], 1),
            "ds0": ds0 if case["s0"] else None}


def exact_turn(case, s):
    d, r = case["d"], case["rotary"]
    n = s["pre"].shape[0]
    if s["positions"] is None:
        _, _, bs, _ = packing(lengths_of(case))
        pos = torch.from_numpy(np.repeat(np.arange(len(bs)), bs)).cuda().double()
    else:
        pos = s["positions"].double()
    # the rotation as complex numbers of unit size, one for each row and pair
    unit = torch.polar(torch.ones((n, r // 2), dtype=torch.float64, device="cuda"),
                       pos[:, None] * torch.from_numpy(frequencies(case)).cuda())[:, None]
    left = torch.arange(r // 2, device="cuda") * (1 if case["layout"] == "half" else 2)
    right = left + (r // 2 if case["layout"] == "half" else 1)

    def rotate(x, by):
        out = x.clone()
        z = torch.complex(x[..., left], x[..., right]) * by
        out[..., left], out[..., right] = z.real, z.imag
        return out

    outs, grads, dws = [], [], []
    for x, w, dy in zip(pair(case, s["pre"].double()), (s["wq"], s["wk"]), (s.get("dq_out"), s.get("dk_out"))):
        w = torch.ones(d, dtype=torch.float64, device="cuda") if w is None else w.double()
        mean = x.sum(-1, keepdim=True) / d if case["kind"] == "layer" else torch.zeros_like(x[..., :1])
        u = x - mean
        dev = torch.ones_like(mean) if case["kind"] == "none" else torch.sqrt((u ** 2).sum(-1, keepdim=True) / d + EPS)
        outs.append(rotate(u / dev * w, unit))
        if dy is None:
            continue
        g = rotate(dy.double(), unit.conj())
        dws.append((g * u / dev).sum((0, 1)) if case["kind"] != "none" else None)
        g = g * w
        if case["kind"] == "layer":
            g = g - g.sum(-1, keepdim=True) / d
        if case["kind"] != "none":
            g = g / dev - u * (g * u).sum(-1, keepdim=True) / (d * dev ** 3)
        grads.append(g.flatten(1))
    out = {"q": outs[0], "k": outs[1]}
    if grads:
        dpre = torch.zeros_like(s["pre"], dtype=torch.float64)
        dpre[:, :(case["qh"] + case["kh"]) * d] = torch.cat(grads, 1)
        out["dpre"], out["dw"] = dpre, dws
    return out
