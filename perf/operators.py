"""Cases that measure the state-space sequence operators: the selective scan
and the short causal convolution in front of it, for prompts (batches of equal
length and ragged ones), for training (forward and backward) and for single
tokens over a cache of states.

`own` false: plain torch operations.  `own` true: the library's calls.

A selective scan is the solve of a block lower-bidiagonal system along a chain:
    dt' = softplus(dt + dt_bias)                     per row t and channel d
    h_t = exp(dt'_t A) h_{t-1} + dt'_t x_t B_t       N states per channel
    y_t = (sum_n C_t h_t + D x_t) * silu(z_t)
and the causal convolution is y_t = silu(bias + sum_j weight_j x_{t-K+1+j}).
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _lib():
    from sparse_spd_selected_b200 import selinv
    return selinv


def listed():
    return [
        # one user's next token: nothing but latency
        {"name": "conv token 1", "op": "conv_step", "batch": 1, "slots": 1, "D": 2048, "K": 4, "type": "bf16"},
        # a full serving batch, its states in a larger cache
        {"name": "conv token 192", "op": "conv_step", "batch": 192, "slots": 256, "D": 4096, "K": 4, "type": "bf16"},
        # prompts of several users in one packed row, some continued from a state
        {"name": "conv prompts ragged", "op": "conv", "rows": 12345, "seqs": 24, "D": 4096, "K": 4, "type": "f16"},
        # a training step's layer
        {"name": "conv train", "op": "conv_train", "batch": 8, "L": 2048, "D": 4096, "K": 4, "type": "bf16"},
        # odd sizes in single precision
        {"name": "conv train odd", "op": "conv_train", "batch": 3, "L": 1021, "D": 1030, "K": 3, "type": "f32"},
        {"name": "scan token 1", "op": "scan_step", "batch": 1, "slots": 1, "D": 2048, "N": 16, "G": 1, "type": "bf16"},
        {"name": "scan token 192", "op": "scan_step", "batch": 192, "slots": 256, "D": 4096, "N": 16, "G": 1,
         "type": "bf16"},
        # one user's prompt: few channels for the whole GPU
        {"name": "scan prompt", "op": "scan", "batch": 1, "L": 4096, "D": 2048, "N": 16, "G": 1, "type": "bf16"},
        # prompts of several users in one packed row, each from a state of its own
        {"name": "scan prompts ragged", "op": "scan", "rows": 12345, "seqs": 24, "D": 2048, "N": 16, "G": 1,
         "type": "f16"},
        # a long document on a narrow layer
        {"name": "scan long", "op": "scan", "batch": 1, "L": 50001, "D": 512, "N": 16, "G": 1, "type": "bf16"},
        # a training step's layer
        {"name": "scan train", "op": "scan_train", "batch": 4, "L": 2048, "D": 4096, "N": 16, "G": 1, "type": "bf16"},
        # odd sizes, a state that is no power of two, two groups of channels, single precision
        {"name": "scan train odd", "op": "scan_train", "batch": 3, "L": 517, "D": 1250, "N": 12, "G": 2,
         "type": "f32"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_step", "conv", "conv_train", "scan_step", "scan", "scan", "scan_train", "scan_train"])
    c = {"op": op, "type": rng.choice(["bf16", "bf16", "f16", "f32"])}
    wide = rng.random() < 0.6
    d = _spread(rng, 8, 512) * 8 if wide else _spread(rng, 50, 4096)
    if op.endswith("step"):
        batch = _spread(rng, 1, 192)
        c.update(batch=batch, slots=batch + rng.choice([0, 1, 7, 40]) if batch > 1 else 1)
    elif op in ("conv", "scan") and rng.random() < 0.5:
        seqs = _spread(rng, 2, 64)
        c.update(rows=max(seqs, _spread(rng, 200, 30000)), seqs=seqs)
    else:
        batch = rng.choice([1, 1, 2, 3, 4, 8])
        c.update(batch=batch, L=max(1, _spread(rng, 50, 30000) // batch))
    if op.startswith("conv"):
        c["K"] = rng.choice([2, 3, 4, 4, 4])
        room = 60_000_000
        n = 1
    else:
        c["N"] = n = rng.choice([16, 16, 16, 8, 12, 32, 64])
        c["G"] = rng.choice([1, 1, 1, 2, 4])
        room = 400_000_000 if op != "scan_train" else 300_000_000
    rows = c.get("rows") or c["batch"] * c.get("L", 1)
    room = min(room, n * (30_000_000 if c["type"] == "f32" else 60_000_000))
    if rows * d * n > room:
        d = max(8, room // (rows * n) // 8 * 8)
    c["D"] = d // c["G"] * c["G"] if c.get("G", 1) > 1 else d
    return c


def _lengths(case, seed):
    """Ragged lengths with the given sum: spread over a factor of some tens, one of them a single row."""
    g = torch.Generator().manual_seed(seed * 7 + 1)
    s, rows = case["seqs"], case["rows"]
    w = torch.exp(3.0 * torch.rand(s, generator=g, dtype=torch.float64))
    n = torch.clamp((w / w.sum() * (rows - s)).floor().long(), min=0) + 1
    n[0] = 1
    n[s - 1] += rows - int(n.sum())
    return n.tolist()


def prepare(case, seed):
    dev, t = torch.device("cuda"), TYPES[case["type"]]
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    op, d = case["op"], case["D"]
    s = {"op": op, "type": t}
    step, train = op.endswith("step"), op.endswith("train")
    if step:
        lead = (case["batch"],)
        if case["slots"] > 1:
            s["index"] = torch.randperm(case["slots"], generator=g, device=dev)[:case["batch"]].to(torch.int32)
        else:
            s["index"] = None
    elif "rows" in case:
        s["lengths"] = _lengths(case, seed)
        lead = (case["rows"],)
    else:
        s["lengths"] = [case["L"]] * case["batch"]
        lead = (case["batch"], case["L"])
    s["lead"] = lead
    if not step:
        n = torch.tensor(s["lengths"], device=dev)
        ends = torch.cumsum(n, 0)
        rows = int(sum(s["lengths"]))
        # the sequence of each row, its first row, and the row where each sequence ends
        s["seq"] = torch.searchsorted(ends, torch.arange(rows, device=dev), right=True)
        s["first"] = (ends - n)[s["seq"]]
        s["ends"] = ends
        if own and "rows" in case:
            s["plan"] = _lib().SequencePlan(s["lengths"])
        else:
            s["plan"] = None
    ragged = "rows" in case
    if op.startswith("conv"):
        k = case["K"]
        # x is one half of a projection's output, as such a layer has it
        s["x"] = normal(*lead, 2 * d).to(t)[..., :d]
        s["weight"] = ((2 * uniform(d, k) - 1) / math.sqrt(k)).to(t)
        s["bias"] = (0.2 * normal(d)).to(t)
        if step:
            s["cache"] = normal(case["slots"], k - 1, d).to(t)
            s["cache_out"] = s["cache"].clone()
            s["row"] = s["index"].long() if s["index"] is not None else torch.arange(case["batch"], device=dev)
        s["state"] = normal(case["seqs"], k - 1, d).to(t) if ragged else None
    else:
        n, grp = case["N"], case["G"]
        xz = normal(*lead, 2 * d).to(t)
        s["x"], s["z"] = xz[..., :d], xz[..., d:]
        s["dt"] = (0.5 * normal(*lead, d)).to(t)
        # B and C are parts of one projection's output
        bc = normal(*lead, 2 * grp * n + 8).to(t)
        s["B"] = bc[..., 8:8 + grp * n].unflatten(-1, (grp, n))
        s["C"] = bc[..., 8 + grp * n:].unflatten(-1, (grp, n))
        s["A"] = -(torch.arange(1, n + 1, device=dev) * torch.exp(0.3 * normal(d, n)))
        s["D"] = 1 + 0.2 * normal(d)
        step_size = torch.exp(math.log(1e-3) + (math.log(1e-1) - math.log(1e-3)) * uniform(d))
        s["dt_bias"] = step_size + torch.log(-torch.expm1(-step_size))
        if step:
            s["cache"] = normal(case["slots"], d, n)
            s["cache_out"] = s["cache"].clone()
            s["row"] = s["index"].long() if s["index"] is not None else torch.arange(case["batch"], device=dev)
        s["state"] = 0.5 * normal(case["seqs"], d, n) if ragged else None
    if train:
        s["yb"] = normal(*lead, d).to(t)
    return s


# ---- the library's calls -------------------------------------------------


def _run_own(s):
    v, op = _lib(), s["op"]
    if op == "conv_step":
        y = v.causal_conv_step(s["cache"], s["x"], s["weight"], s["bias"], silu=True, index=s["index"],
                               cache_out=s["cache_out"], check=False)
        return [y, s["cache_out"]]
    if op == "scan_step":
        y = v.selective_scan_step(s["cache"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], z=s["z"],
                                  dt_bias=s["dt_bias"], softplus=True, index=s["index"], cache_out=s["cache_out"],
                                  check=False)
        return [y, s["cache_out"]]
    if op == "conv":
        r = v.causal_conv(s["x"], s["weight"], s["bias"], silu=True, state=s["state"], plan=s["plan"])
        return [r["y"], r["state"]]
    if op == "conv_train":
        r = v.causal_conv(s["x"], s["weight"], s["bias"], silu=True, want_state=False)
        b = v.causal_conv_backward(s["x"], s["weight"], s["yb"], bias=s["bias"], silu=True)
        return [r["y"], b["xb"], b["weightb"], b["biasb"]]
    more = dict(z=s["z"], dt_bias=s["dt_bias"], softplus=True, state=s["state"], plan=s["plan"])
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    if op == "scan":
        r = v.selective_scan(*args, s["D"], **more)
        return [r["y"], r["state"]]
    r = v.selective_scan(*args, s["D"], keep=True, want_state=False, **more)
    b = v.selective_scan_backward(r["kept"], *args, s["yb"], D=s["D"], **more)
    return [r["y"]] + [b[k] for k in ("xb", "dtb", "Ab", "Bb", "Cb", "Db", "zb", "dt_biasb")]


# ---- the plain form ------------------------------------------------------


def _silu_slope(v):
    p = torch.sigmoid(v)
    return p * (1 + v * (1 - p))


def _taps(s, k):
    """For each row the places of its k taps in [x; the initial states; a row of zeros]."""
    rows = s["seq"].numel()
    back = torch.arange(rows, device=s["seq"].device)[:, None] + torch.arange(1 - k, 1, device=s["seq"].device)
    before = s["first"][:, None] - back
    if s["state"] is None:
        return torch.where(before > 0, rows, back)
    return torch.where(before > 0, rows + s["seq"][:, None] * (k - 1) + (k - 1) - before, back)


def _run_conv(s):
    t, (d, k) = s["type"], s["weight"].shape
    w, b = s["weight"].float(), s["bias"].float()
    if s["op"] == "conv_step":
        win = torch.cat([s["cache"][s["row"]], s["x"][:, None]], 1)
        s["cache_out"][s["row"]] = win[:, 1:]
        pre = (win.float() * w.t()).sum(1) + b
        return [(pre * torch.sigmoid(pre)).to(t), s["cache_out"]]
    x = s["x"].reshape(-1, d)
    rows = x.shape[0]
    states = x.new_zeros(0, d) if s["state"] is None else s["state"].reshape(-1, d)
    every = torch.cat([x, states, x.new_zeros(1, d)])
    at = _taps(s, k)
    win = every[at].float()
    pre = (win * w.t()).sum(1) + b
    y = (pre * torch.sigmoid(pre)).to(t).reshape(*s["lead"], d)
    if s["op"] == "conv":
        # the last k - 1 inputs of each sequence: the taps of its last row but the oldest, moved by one
        last = s["ends"] - 1
        return [y, every[at[last]][:, 1:]]
    prb = s["yb"].reshape(-1, d).float() * _silu_slope(pre)
    # row t is a tap of the rows t .. t + k - 1 of its sequence
    ahead = torch.arange(rows, device=x.device)[:, None] + torch.arange(k, device=x.device)
    ahead = torch.where(ahead < s["ends"][s["seq"]][:, None], ahead, rows)
    xb = (torch.cat([prb, prb.new_zeros(1, d)])[ahead] * w.flip(1).t()).sum(1)
    return [y, xb.to(t).reshape(*s["lead"], d), (win * prb[:, None]).sum(0).t().contiguous(), prb.sum(0)]


def _doubling(a, u, k=1):
    """h_t = a_t h_{t-1} + u_t along the first axis, h before the first row zero: each pass joins runs of k rows
    to runs of 2 k."""
    if k >= a.shape[0]:
        return u
    u = torch.cat([u[:k], u[k:] + a[k:] * u[:-k]])
    return _doubling(torch.cat([a[:k], a[k:] * a[:-k]]), u, 2 * k) if 2 * k < a.shape[0] else u


def _spreads(v, d):
    """[rows, G, N] of the groups for each of the d channels: [rows, d, N]."""
    return v.float().repeat_interleave(d // v.shape[-2], dim=-2)


def _run_scan(s):
    t, (d, n) = s["type"], s["A"].shape
    grp = s["B"].shape[-2]
    flat = {k: s[k].reshape(-1, *s[k].shape[len(s["lead"]):]) for k in ("x", "dt", "B", "C", "z")}
    x, z = flat["x"].float(), flat["z"].float()
    raw = flat["dt"].float() + s["dt_bias"]
    dt = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    bs, cs = _spreads(flat["B"], d), _spreads(flat["C"], d)
    a = torch.exp(dt[..., None] * s["A"])
    u = (dt * x)[..., None] * bs
    if s["op"] == "scan_step":
        h = a * s["cache"][s["row"]] + u
        s["cache_out"][s["row"]] = h
        y = (h * cs).sum(-1) + s["D"] * x
        return [(y * z * torch.sigmoid(z)).to(t), s["cache_out"]]
    rows = x.shape[0]
    starts = (s["first"] == torch.arange(rows, device=x.device)).nonzero()[:, 0]
    if s["state"] is not None:
        u[starts] += a[starts] * s["state"]
    kept = a.clone()
    kept[starts] = 0
    h = _doubling(kept, u)
    y = (h * cs).sum(-1) + s["D"] * x
    gate = z * torch.sigmoid(z)
    out = (y * gate).to(t).reshape(*s["lead"], d)
    if s["op"] == "scan":
        return [out, h[s["ends"] - 1]]
    yb = s["yb"].reshape(-1, d).float()
    zb = yb * y * _silu_slope(z)
    yb = yb * gate
    # g_t = C_t yb_t + a_{t+1} g_{t+1}: the same recurrence, from the last row to the first
    after = torch.cat([kept[1:], torch.zeros_like(kept[:1])])
    g = _doubling(after.flip(0), (cs * yb[..., None]).flip(0)).flip(0)
    del after
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    q = g * kept * before
    if s["state"] is not None:
        q[starts] = g[starts] * a[starts] * s["state"]
    dux = (g * bs).sum(-1)
    dtb = dux * x + (q * s["A"]).sum(-1)
    xb = dux * dt + s["D"] * yb
    rawb = dtb * torch.sigmoid(raw)
    ab = (q * dt[..., None]).sum(0)
    bb = (g * (dt * x)[..., None]).reshape(rows, grp, d // grp, n).sum(2)
    cb = (h * yb[..., None]).reshape(rows, grp, d // grp, n).sum(2)
    shape = s["lead"]
    return [out, xb.to(t).reshape(*shape, d), rawb.to(t).reshape(*shape, d), ab, bb.to(t).reshape(*shape, grp, n),
            cb.to(t).reshape(*shape, grp, n), (yb * x).sum(0), zb.to(t).reshape(*shape, d), rawb.sum(0)]


def run(s):
    if own:
        return _run_own(s)
    return _run_conv(s) if s["op"].startswith("conv") else _run_scan(s)


# ---- the definition, in 64 bits, one row after another -------------------


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"].startswith("conv"):
        return _exact_conv(s)
    return _exact_scan(s)


def _exact_conv(s):
    w, b = s["weight"].double(), s["bias"].double()
    d, k = w.shape
    x = s["x"].double()

    def weigh(ext):
        return torch.nn.functional.conv1d(ext.t()[None], w[:, None], b, groups=d)[0].t()

    if s["op"] == "conv_step":
        new = s["cache"].double().clone()
        ys = []
        for i, r in enumerate(s["row"].tolist()):
            ext = torch.cat([new[r], x[i:i + 1]])
            ys.append((ext * w.t()).sum(0) + b)
            new[r] = ext[1:]
        y = torch.stack(ys)
        return [y / (1 + torch.exp(-y)), new]
    x = x.reshape(-1, d)
    outs, lasts, xbs, wb, bb, at = [], [], [], torch.zeros_like(w), torch.zeros_like(b), 0
    yb = s["yb"].double().reshape(-1, d) if "yb" in s else None
    for i, n in enumerate(s["lengths"]):
        head = x.new_zeros(k - 1, d) if s["state"] is None else s["state"][i].double()
        ext = torch.cat([head, x[at:at + n]])
        pre = weigh(ext)
        p = 1 / (1 + torch.exp(-pre))
        outs.append(pre * p)
        lasts.append(ext[n:])
        if yb is not None:
            prb = yb[at:at + n] * (p + pre * p * (1 - p))
            eb = torch.zeros_like(ext)
            for j in range(k):
                eb[j:j + n] += prb * w[:, j]
                wb[:, j] += (prb * ext[j:j + n]).sum(0)
            bb += prb.sum(0)
            xbs.append(eb[k - 1:])
        at += n
    y = torch.cat(outs).reshape(*s["lead"], d)
    if s["op"] == "conv":
        return [y, torch.stack(lasts)]
    return [y, torch.cat(xbs).reshape(*s["lead"], d), wb, bb]


def _exact_scan(s):
    dev = s["x"].device
    a_, skip, bias = s["A"].double(), s["D"].double(), s["dt_bias"].double()
    d, n = a_.shape
    grp = s["B"].shape[-2]
    of = torch.arange(d, device=dev) // (d // grp)
    if s["op"] == "scan_step":
        new = s["cache"].double().clone()
        ys = []
        for i, r in enumerate(s["row"].tolist()):
            step = torch.logaddexp(s["dt"][i].double() + bias, torch.zeros_like(bias))
            xi, zi = s["x"][i].double(), s["z"][i].double()
            h = torch.exp(step[:, None] * a_) * new[r] + (step * xi)[:, None] * s["B"][i].double()[of]
            new[r] = h
            ys.append(((h * s["C"][i].double()[of]).sum(1) + skip * xi) * zi / (1 + torch.exp(-zi)))
        return [torch.stack(ys), new]
    lengths = s["lengths"]
    count, longest = len(lengths), max(lengths)
    rows = sum(lengths)
    train = "yb" in s
    if train and rows * d * n * 8 > 20e9:
        return None
    # row r of every sequence that is long enough, all at once
    first = torch.cumsum(torch.tensor([0] + lengths[:-1]), 0)
    order = sorted(range(count), key=lambda i: -lengths[i])
    alive = [sum(1 for v in lengths if v > r) for r in range(longest)]
    start = first[order].to(dev)
    names = ("x", "dt", "B", "C", "z") + (("yb",) if train else ())
    flat = {k: s[k].reshape(-1, *s[k].shape[len(s["lead"]):]) for k in names}
    h = a_.new_zeros(count, d, n) if s["state"] is None else s["state"].double()[order].clone()
    y = torch.empty(rows, d, dtype=torch.float64, device=dev)
    past = torch.empty(rows, d, n, dtype=torch.float64, device=dev) if train else None
    for r in range(longest):
        m = alive[r]
        at = start[:m] + r
        step = torch.logaddexp(flat["dt"][at].double() + bias, torch.zeros_like(bias))
        xr, zr = flat["x"][at].double(), flat["z"][at].double()
        if train:
            past[at] = h[:m]
        h[:m] = torch.exp(step[..., None] * a_) * h[:m] + (step * xr)[..., None] * flat["B"][at].double()[:, of]
        y[at] = ((h[:m] * flat["C"][at].double()[:, of]).sum(-1) + skip * xr) * zr / (1 + torch.exp(-zr))
    if not train:
        back = torch.empty_like(h)
        back[order] = h
        return [y.reshape(*s["lead"], d), back]
    xb, dtb, zb = torch.empty_like(y), torch.empty_like(y), torch.empty_like(y)
    bb = torch.empty(rows, grp, n, dtype=torch.float64, device=dev)
    cb = torch.empty_like(bb)
    ab, db, bias_b = torch.zeros_like(a_), torch.zeros_like(skip), torch.zeros_like(bias)
    g = a_.new_zeros(count, d, n)          # the cotangent that row r + 1 hands to row r
    for r in range(longest - 1, -1, -1):
        m = alive[r]
        at = start[:m] + r
        raw = flat["dt"][at].double() + bias
        step = torch.logaddexp(raw, torch.zeros_like(bias))
        xr, zr, yr = flat["x"][at].double(), flat["z"][at].double(), flat["yb"][at].double()
        br, cr = flat["B"][at].double()[:, of], flat["C"][at].double()[:, of]
        decay, prev = torch.exp(step[..., None] * a_), past[at]
        now = decay * prev + (step * xr)[..., None] * br
        p = 1 / (1 + torch.exp(-zr))
        inner = (now * cr).sum(-1) + skip * xr
        zb[at] = yr * inner * p * (1 + zr * (1 - p))
        yr = yr * zr * p
        total = cr * yr[..., None] + g[:m]
        u = (total * br).sum(-1)
        moved = total * decay * prev
        rawb = (u * xr + (moved * a_).sum(-1)) / (1 + torch.exp(-raw))
        xb[at], dtb[at] = u * step + skip * yr, rawb
        ab += (moved * step[..., None]).sum(0)
        db += (yr * xr).sum(0)
        bias_b += rawb.sum(0)
        bb[at] = (total * (step * xr)[..., None]).reshape(m, grp, d // grp, n).sum(2)
        cb[at] = (now * yr[..., None]).reshape(m, grp, d // grp, n).sum(2)
        g[:m] = total * decay
    f = s["lead"]
    y = y.reshape(*f, d)
    return [y, xb.reshape(*f, d), dtb.reshape(*f, d), ab, bb.reshape(*f, grp, n), cb.reshape(*f, grp, n), db,
            zb.reshape(*f, d), bias_b]


# ---- what one pass cannot do without -------------------------------------


def work(case):
    e = 4 if case["type"] == "f32" else 2
    d, op = case["D"], case["op"]
    rows = case.get("rows") or case["batch"] * case.get("L", 1)
    seqs = case.get("seqs", 0) if "rows" in case else 0
    if op.startswith("conv"):
        k = case["K"]
        w = e * d * (k + 1)
        if op == "conv_step":
            return {"bytes": e * d * rows * (2 + 2 * (k - 1)) + w, "flops": rows * d * (2 * k + 5)}
        if op == "conv":
            last = (seqs or case["batch"]) * (k - 1) * d * e
            return {"bytes": 2 * e * rows * d + w + last + seqs * (k - 1) * d * e, "flops": rows * d * (2 * k + 5)}
        return {"bytes": 4 * e * rows * d + w + 4 * d * (k + 1), "flops": rows * d * (6 * k + 16)}
    n, grp = case["N"], case["G"]
    consts = 4 * d * (n + 2)
    if op == "scan_step":
        return {"bytes": rows * (4 * e * d + 2 * e * grp * n + 8 * d * n) + consts, "flops": rows * d * (7 * n + 20)}
    if op == "scan":
        states = 4 * d * n * ((seqs or case["batch"]) + seqs)
        return {"bytes": rows * (4 * e * d + 2 * e * grp * n) + consts + states, "flops": rows * d * (7 * n + 20)}
    return {"bytes": rows * (8 * e * d + 4 * e * grp * n) + 2 * consts, "flops": rows * d * (26 * n + 50)}
