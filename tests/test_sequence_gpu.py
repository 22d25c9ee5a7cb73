"""The selective scan and the causal convolution on the GPU against their plain float64 forms: element types, sizes
around every tile edge, ragged sequences, states, single tokens, gradients, strides, streams and captured graphs.

A result may differ from the plain one, computed from the same rounded inputs, by half a unit of its own type (its
last rounding) and by the roundings of the arithmetic: their number along the longest path times the unit roundoff
times the magnitude of the terms (sequence_plain)."""
import numpy as np
import pytest
import torch

from sparse_spd_selected_b200 import selinv
from tests import sequence_plain as plain

pytestmark = pytest.mark.gpu

TYPES = {"f64": torch.float64, "f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def arith(t):
    return torch.float64 if t == torch.float64 else torch.float32


def unit(t):
    """Unit roundoff of a type: half its eps."""
    return torch.finfo(t).eps / 2


def dev(a, t):
    return torch.as_tensor(np.ascontiguousarray(a)).to("cuda", t)


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(name, got, ref, mag, bound):
    """|got - ref| <= bound * mag + half a unit of got's type (and its smallest step)."""
    info = torch.finfo(got.dtype)
    assert tuple(got.shape) == ref.shape, name
    tol = bound * mag + unit(got.dtype) * np.abs(ref) * (1 + 2 * bound) + unit(got.dtype) * bound * mag + info.smallest_normal
    off = np.abs(host(got) - ref)
    assert np.isfinite(off).all() and (off <= tol).all(), (name, float((off / tol).max()), float(off.max()))


def scan_inputs(seed, t, lead, d, n, groups, gate=True, skip=True, bias=True, softplus=True, states=None):
    g = np.random.default_rng(seed)
    v = {"x": dev(g.standard_normal(lead + (d,)), t)}
    v["dt"] = dev(0.5 * g.standard_normal(lead + (d,)) if softplus else g.uniform(0.01, 0.5, lead + (d,)), t)
    v["A"] = dev(-np.exp(g.uniform(-2, 1, (d, n))), arith(t))
    v["B"] = dev(g.standard_normal(lead + (groups, n)), t)
    v["C"] = dev(g.standard_normal(lead + (groups, n)), t)
    v["D"] = dev(g.standard_normal(d), arith(t)) if skip else None
    v["z"] = dev(g.standard_normal(lead + (d,)), t) if gate else None
    v["dt_bias"] = dev(g.uniform(-3, 0, d) if softplus else g.uniform(0, 0.3, d), arith(t)) if bias else None
    v["state"] = dev(g.standard_normal(states + (d, n)), arith(t)) if states is not None else None
    yb = dev(g.standard_normal(lead + (d,)), t)
    stateb = dev(g.standard_normal(states + (d, n)), arith(t)) if states is not None else None
    return v, yb, stateb


ROWWISE = ("x", "dt", "B", "C", "z", "y", "xb", "dtb", "Bb", "Cb", "zb")


def scan_plain(v, yb, stateb, lengths, softplus, mag):
    """The plain scan of sequences one after another in flat rows; parameters' cotangents summed."""
    w = {k: host(a) for k, a in v.items()}
    outs, at = [], 0
    for i, m in enumerate(lengths):
        s = {k: (a[at:at + m] if k in ROWWISE and a is not None else a) for k, a in w.items()}
        s["state"] = None if w["state"] is None else w["state"][i]
        outs.append(plain.scan(**s, softplus=softplus, yb=host(yb)[at:at + m],
                               stateb=None if stateb is None else host(stateb)[i], mag=mag))
        at += m
    r = {}
    for k in outs[0]:
        if k in ROWWISE:
            r[k] = np.concatenate([o[k] for o in outs])
        elif k in ("state", "stateb"):
            r[k] = np.stack([o[k] for o in outs])
        else:
            r[k] = sum(o[k] for o in outs)
    return r


def check_scan(seed, kind, lengths, d, n, groups=1, ragged=False, tail=0, **options):
    t, softplus = TYPES[kind], options.get("softplus", True)
    with_state = options.pop("with_state", False)
    rows = sum(lengths)
    lead = (rows + tail,) if ragged else (len(lengths), lengths[0])
    v, yb, stateb = scan_inputs(seed, t, lead, d, n, groups, states=(len(lengths),) if with_state else None, **options)
    plan = selinv.SequencePlan(lengths) if ragged else None
    more = dict(z=v["z"], dt_bias=v["dt_bias"], softplus=softplus, state=v["state"], plan=plan)
    args = (v["x"], v["dt"], v["A"], v["B"], v["C"])
    r = selinv.selective_scan(*args, v["D"], keep=True, **more)
    b = selinv.selective_scan_backward(r["kept"], *args, yb, D=v["D"], stateb=stateb, **more)
    flat = lambda a: None if a is None else a.reshape((-1,) + a.shape[len(lead):])[:rows]   # noqa: E731
    fv = {k: flat(a) if k in ROWWISE else a for k, a in v.items()}
    ref = scan_plain(fv, flat(yb), stateb, lengths, softplus, False)
    mag = scan_plain(fv, flat(yb), stateb, lengths, softplus, True)
    longest = max(lengths)
    u = unit(arith(t))
    row_bound = plain.scan_bound(longest, n, d, u)
    sum_bound = plain.scan_bound(longest, n, d + rows, u)
    near("y", flat(r["y"]), ref["y"], mag["y"], row_bound)
    near("state", r["state"], ref["state"], mag["state"], row_bound)
    for k in ("xb", "dtb", "Bb", "Cb", "zb"):
        if b[k] is not None:
            near(k, flat(b[k]), ref[k], mag[k], row_bound)
    for k in ("Ab", "Db", "dt_biasb"):
        if b[k] is not None:
            near(k, b[k], ref[k], mag[k], sum_bound)
    if with_state:
        near("stateb", b["stateb"], ref["stateb"], mag["stateb"], row_bound)
    else:
        assert b["stateb"] is None
    if tail:
        for a in (r["y"], b["xb"], b["dtb"], b["Bb"], b["Cb"]):
            assert not host(a[rows:]).any()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16", "f64"])
@pytest.mark.parametrize("lines,rows,d,n,groups", [
    (1, 1, 1, 1, 1), (2, 3, 5, 2, 1), (1, 15, 8, 4, 2), (3, 16, 33, 16, 1), (2, 17, 32, 16, 4), (1, 33, 130, 16, 1),
    (2, 40, 24, 12, 3), (1, 50, 40, 32, 1), (2, 21, 12, 64, 2), (1, 19, 9, 37, 1), (2, 18, 64, 8, 1),
])
def test_scan_sizes(cuda_ok, kind, lines, rows, d, n, groups):
    check_scan(100 + rows, kind, [rows] * lines, d, n, groups, with_state=lines == 2)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("d,n", [(2400, 16), (2401, 12), (1600, 32), (9000, 8), (19000, 3), (1230, 64)])
def test_scan_wide_tiles(cuda_ok, kind, d, n):
    """Enough channels for the tiles of 4 x 4 states per thread: 600 warps and more."""
    check_scan(200 + n, kind, [18] * 8, d, n, groups=1 if d % 2 else 2, with_state=True)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f64"])
@pytest.mark.parametrize("lines,n", [(37, 16), (50, 12), (50, 7)])
def test_scan_whole_lines(cuda_ok, kind, lines, n):
    """Lines that are not cut, one or two blocks per multiprocessor, of channels that end within a tile."""
    check_scan(52, kind, [18] * lines, 490, n)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("d,groups", [(34, 1), (35, 1), (70, 2), (68, 2), (1, 1)])
def test_scan_rows_off_16_bytes(cuda_ok, kind, d, groups):
    """Rows of 16-bit elements on words and on odd places, and channels that end in the middle of a word."""
    check_scan(53, kind, [19, 19], d, 16, groups)


@pytest.mark.parametrize("kind", ["f32", "f16", "f64"])
@pytest.mark.parametrize("rows,d,n", [(700, 8, 16), (1030, 33, 5), (257, 16, 64), (130, 3, 4)])
def test_scan_segments(cuda_ok, kind, rows, d, n):
    """Few channels and many rows: lines are cut and the segments' states handed on."""
    check_scan(300 + rows, kind, [rows] * 2, d, n, with_state=True)


@pytest.mark.parametrize("kind", ["f32", "f64"])
def test_scan_growth_beyond_a_segments_range(cuda_ok, kind):
    """Steps below zero let states grow, over the 32 rows of one segment by more than the type's range: nothing stays
    nothing, and a small state a finite one."""
    t, rows, d, n = TYPES[kind], 512, 6, 4
    step, small = (3.0, 1e-30) if kind == "f32" else (23.0, 1e-250)
    v, yb, stateb = scan_inputs(78, t, (1, rows), d, n, 1, softplus=False, bias=False, skip=False, states=(1,))
    v["x"].zero_()
    v["A"].fill_(-1)
    v["dt"].zero_()
    v["dt"][:, 64:96] = -step
    v["state"].fill_(small)
    v["state"][:, ::2] = 0
    yb.zero_()
    yb[:, -1] = small
    stateb.zero_()
    args = (v["x"], v["dt"], v["A"], v["B"], v["C"])
    r = selinv.selective_scan(*args, z=v["z"], state=v["state"], keep=True)
    b = selinv.selective_scan_backward(r["kept"], *args, yb, z=v["z"], state=v["state"], stateb=stateb)
    # the decays' arguments come to 32 steps: an error of a unit each is that many units of the state
    u = unit(arith(t))
    bound = plain.scan_bound(rows, n, d, u) + 8 * 32 * step * u
    flat = {k: a[0] if k in ROWWISE and a is not None else a for k, a in v.items()}
    ref, mag = (scan_plain(flat, yb[0], stateb, [rows], False, m) for m in (False, True))
    assert np.isfinite(host(r["y"])).all() and not host(r["state"])[:, ::2].any()
    near("y", r["y"][0], ref["y"], mag["y"], bound)
    near("state", r["state"], ref["state"], mag["state"], bound)
    near("stateb", b["stateb"], ref["stateb"], mag["stateb"], bound)


@pytest.mark.parametrize("options", [dict(gate=False), dict(skip=False), dict(bias=False), dict(softplus=False),
                                     dict(gate=False, skip=False, bias=False, softplus=False)])
def test_scan_without_options(cuda_ok, options):
    check_scan(400, "f32", [37, 37], 20, 16, **options)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f64"])
@pytest.mark.parametrize("lengths", [
    [1], [0, 5, 0], [1] * 40, [16, 16, 16], [15, 17, 1, 0, 0, 31, 2], [3, 200, 1, 1, 1, 150, 64, 0], [513],
])
@pytest.mark.parametrize("with_state", [False, True])
def test_scan_ragged(cuda_ok, kind, lengths, with_state):
    check_scan(500 + len(lengths), kind, lengths, 24, 16, groups=2, ragged=True, tail=3, with_state=with_state)


def test_scan_ragged_wide_tiles(cuda_ok):
    check_scan(600, "bf16", [5, 1, 0, 40, 16, 2], 20000, 16, ragged=True, with_state=True)


def test_scan_without_rows(cuda_ok):
    v, yb, stateb = scan_inputs(1, torch.float32, (2, 0), 4, 3, 1, states=(2,))
    r = selinv.selective_scan(*(v[k] for k in ("x", "dt", "A", "B", "C", "D")), z=v["z"], state=v["state"], keep=True)
    assert r["y"].shape == (2, 0, 4) and torch.equal(r["state"], v["state"])
    b = selinv.selective_scan_backward(r["kept"], *(v[k] for k in ("x", "dt", "A", "B", "C")), yb, D=v["D"], z=v["z"],
                                       state=v["state"], stateb=stateb)
    assert torch.equal(b["stateb"], stateb) and not b["Ab"].any() and not b["Db"].any()
    plan = selinv.SequencePlan([0, 0])
    x = v["x"][0]
    r = selinv.selective_scan(x, v["dt"][0], v["A"], v["B"][0], v["C"][0], plan=plan, state=v["state"])
    assert torch.equal(r["state"], v["state"])
    r = selinv.selective_scan(x, v["dt"][0], v["A"], v["B"][0], v["C"][0], plan=plan)
    assert not r["state"].any()


def conv_plain(v, yb, stateb, lengths, silu, mag):
    x, outs, at = host(v["x"]), [], 0
    for i, m in enumerate(lengths):
        outs.append(plain.conv(x[at:at + m], host(v["weight"]), host(v["bias"]), silu,
                               None if v["state"] is None else host(v["state"])[i], host(yb)[at:at + m],
                               None if stateb is None else host(stateb)[i], mag))
        at += m
    r = {}
    for k in outs[0]:
        if k in ("y", "xb"):
            r[k] = np.concatenate([o[k] for o in outs])
        elif k in ("state", "stateb"):
            r[k] = np.stack([o[k] for o in outs])
        else:
            r[k] = sum(o[k] for o in outs)
    return r


def check_conv(seed, kind, lengths, d, k, silu=True, ragged=False, tail=0, with_state=False, with_bias=True):
    t = TYPES[kind]
    g = np.random.default_rng(seed)
    rows = sum(lengths)
    lead = (rows + tail,) if ragged else (len(lengths), lengths[0])
    v = {"x": dev(g.standard_normal(lead + (d,)), t), "weight": dev(g.uniform(-1, 1, (d, k)), t),
         "bias": dev(g.standard_normal(d), t) if with_bias else None,
         "state": dev(g.standard_normal((len(lengths), k - 1, d)), t) if with_state else None}
    yb = dev(g.standard_normal(lead + (d,)), t)
    stateb = dev(g.standard_normal((len(lengths), k - 1, d)), t) if with_state else None
    plan = selinv.SequencePlan(lengths) if ragged else None
    r = selinv.causal_conv(v["x"], v["weight"], v["bias"], silu=silu, state=v["state"], plan=plan)
    b = selinv.causal_conv_backward(v["x"], v["weight"], yb, bias=v["bias"], stateb=stateb, silu=silu, state=v["state"],
                                    plan=plan)
    flat = lambda a: a.reshape(-1, d)[:rows]   # noqa: E731
    fv = dict(v, x=flat(v["x"]))
    ref = conv_plain(fv, flat(yb), stateb, lengths, silu, False)
    mag = conv_plain(fv, flat(yb), stateb, lengths, silu, True)
    bound = plain.conv_bound(0, k, unit(arith(t)))
    near("y", flat(r["y"]), ref["y"], mag["y"], bound)
    assert np.array_equal(host(r["state"]), ref["state"])
    near("xb", flat(b["xb"]), ref["xb"], mag["xb"], bound)
    sums = plain.conv_bound(rows, k, unit(arith(t)))
    near("weightb", b["weightb"], ref["weightb"], mag["weightb"], sums)
    near("biasb", b["biasb"], ref["biasb"], mag["biasb"], sums)
    if with_state:
        near("stateb", b["stateb"], ref["stateb"], mag["stateb"], bound)
    if tail:
        assert not host(r["y"][rows:]).any() and not host(b["xb"][rows:]).any()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16", "f64"])
@pytest.mark.parametrize("lines,rows,d,k", [(1, 1, 1, 2), (2, 2, 3, 4), (3, 3, 8, 4), (1, 4, 16, 3), (2, 65, 129, 4),
                                            (1, 300, 40, 4), (2, 33, 24, 2), (1, 37, 11, 8), (2, 19, 16, 5)])
def test_conv_sizes(cuda_ok, kind, lines, rows, d, k):
    check_conv(700 + rows, kind, [rows] * lines, d, k, with_state=lines == 2, silu=rows != 3, with_bias=rows != 4)


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("lengths", [[1], [0, 2, 0], [1] * 40, [2, 1, 3, 0, 70, 4, 33, 1], [260, 3]])
@pytest.mark.parametrize("with_state", [False, True])
def test_conv_ragged(cuda_ok, kind, lengths, with_state):
    check_conv(800 + len(lengths), kind, lengths, 20, 4, ragged=True, tail=2, with_state=with_state)


def test_conv_without_rows(cuda_ok):
    w = dev(np.ones((4, 3)), torch.float32)
    s = dev(np.arange(16.0).reshape(2, 2, 4), torch.float32)
    r = selinv.causal_conv(torch.zeros(2, 0, 4, device="cuda"), w, state=s)
    assert r["y"].shape == (2, 0, 4) and torch.equal(r["state"], s)
    r = selinv.causal_conv(torch.zeros(0, 4, device="cuda"), w, state=s, plan=selinv.SequencePlan([0, 0]))
    assert torch.equal(r["state"], s)
    assert selinv.causal_conv(torch.zeros(0, 3, 4, device="cuda"), w)["y"].shape == (0, 3, 4)


# ---- single tokens ----------------------------------------------------------


@pytest.mark.parametrize("kind", ["f32", "bf16", "f64"])
@pytest.mark.parametrize("batch,d,n,groups", [(1, 1, 1, 1), (3, 33, 16, 1), (5, 64, 12, 2), (2, 40, 64, 1), (4, 300, 5, 3)])
def test_scan_step(cuda_ok, kind, batch, d, n, groups):
    t = TYPES[kind]
    v, _, _ = scan_inputs(900 + d, t, (batch,), d, n, groups, states=(batch,))
    cache = v["state"].clone()
    y = selinv.selective_scan_step(cache, v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], z=v["z"],
                                   dt_bias=v["dt_bias"], softplus=True)
    yb = torch.zeros_like(v["x"])
    ref = scan_plain(v, yb, None, [1] * batch, True, False)
    mag = scan_plain(v, yb, None, [1] * batch, True, True)
    bound = plain.scan_bound(1, n, 0, unit(arith(t)))
    near("y", y, ref["y"], mag["y"], bound)
    near("state", cache, ref["state"], mag["state"], bound)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_steps_over_slots(cuda_ok, kind):
    """Slots in any order, skipped rows, a second array for the new states, and slots that no row names."""
    t = TYPES[kind]
    rng = np.random.default_rng(5)
    slots, d, n, k = 7, 20, 16, 4
    index = torch.tensor([4, -1, 0, 6], dtype=torch.int32, device="cuda")
    row = [4, 0, 6]
    v, _, _ = scan_inputs(950, t, (4,), d, n, 1, states=(slots,))
    args = (v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"])
    more = dict(z=v["z"], dt_bias=v["dt_bias"], softplus=True)
    cache = v["state"].clone()
    new = torch.full_like(cache, 7.0)
    y = selinv.selective_scan_step(cache, *args, index=index, cache_out=new, **more)
    assert torch.equal(cache, v["state"])
    part = v["state"][row].clone()
    live = [0, 2, 3]
    sub = lambda a: a[live].contiguous()    # noqa: E731
    want = selinv.selective_scan_step(part, sub(v["x"]), sub(v["dt"]), v["A"], sub(v["B"]), sub(v["C"]), v["D"],
                                      z=sub(v["z"]), dt_bias=v["dt_bias"], softplus=True)
    assert torch.equal(y[live], want) and not y[1].any()
    assert torch.equal(new[row], part)
    assert bool((new[[1, 2, 3, 5]] == 7.0).all())
    selinv.selective_scan_step(cache, *args, index=index, **more)
    assert torch.equal(cache[row], part) and torch.equal(cache[[1, 2, 3, 5]], v["state"][[1, 2, 3, 5]])

    w, b = dev(rng.standard_normal((d, k)), t), dev(rng.standard_normal(d), t)
    c0 = dev(rng.standard_normal((slots, k - 1, d)), t)
    cache = c0.clone()
    y = selinv.causal_conv_step(cache, v["x"], w, b, silu=True, index=index)
    whole = selinv.causal_conv(v["x"][live].reshape(3, 1, d).contiguous(), w, b, silu=True, state=c0[row].contiguous())
    assert torch.equal(y[live], whole["y"][:, 0]) and not y[1].any()
    assert torch.equal(cache[row], whole["state"]) and torch.equal(cache[[1, 2, 3, 5]], c0[[1, 2, 3, 5]])


def test_bad_slots_are_reported_and_left_alone(cuda_ok):
    d, n = 40, 16
    v, _, _ = scan_inputs(960, torch.float32, (5,), d, n, 1, states=(4,))
    args = (v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"])
    for index, info in (([0, 1, 4, 2, 3], {2: "outside"}), ([0, 1, 0, 2, 1], {2: "earlier", 4: "earlier"}),
                        ([-2, 0, 1, 2, 3], {0: "outside"})):
        cache = v["state"].clone()
        ix = torch.tensor(index, dtype=torch.int32, device="cuda")
        with pytest.raises(selinv.SlotError) as e:
            selinv.selective_scan_step(cache, *args, index=ix)
        assert {r for r, s in enumerate(e.value.info) if s != -1} == set(info)
        good = [r for r in range(5) if r not in info]
        part = v["state"][[index[r] for r in good]].clone()
        sub = lambda a: a[good].contiguous()    # noqa: E731
        want = selinv.selective_scan_step(part, sub(v["x"]), sub(v["dt"]), v["A"], sub(v["B"]), sub(v["C"]), v["D"])
        assert torch.equal(cache[[index[r] for r in good]], part)
        cache = v["state"].clone()
        y = selinv.selective_scan_step(cache, *args, index=ix, check=False)
        assert torch.equal(y[good], want) and not y[list(info)].any()
        w = dev(np.ones((d, 3)), torch.float32)
        with pytest.raises(selinv.SlotError):
            selinv.causal_conv_step(torch.zeros(4, 2, d, device="cuda"), v["x"], w, index=ix)


# ---- as they are used together ----------------------------------------------


def layer_weights(g, t, d, n, k):
    return {"weight": dev(g.uniform(-0.5, 0.5, (d, k)), t), "bias": dev(0.1 * g.standard_normal(d), t),
            "A": dev(-np.exp(g.uniform(-2, 1, (d, n))), arith(t)), "D": dev(g.standard_normal(d), arith(t)),
            "dt_bias": dev(g.uniform(-3, 0, d), arith(t)), "to_bc": dev(0.2 * g.standard_normal((d, 2 * n)), t),
            "to_dt": dev(0.2 * g.standard_normal((d, d)), t)}


def layer(w, xz, n, conv_state=None, state=None, plan=None, ad=False):
    d = xz.shape[-1] // 2
    x, z = xz[..., :d], xz[..., d:]
    if ad:
        c, conv_state = selinv.causal_conv_ad(x, w["weight"], w["bias"], silu=True, state=conv_state, plan=plan)
    else:
        r = selinv.causal_conv(x, w["weight"], w["bias"], silu=True, state=conv_state, plan=plan)
        c, conv_state = r["y"], r["state"]
    bc, dt = c @ w["to_bc"], c @ w["to_dt"]
    B, C = bc[..., None, :n], bc[..., None, n:]
    args = (c, dt, w["A"], B, C, w["D"])
    more = dict(z=z, dt_bias=w["dt_bias"], softplus=True, state=state, plan=plan)
    if ad:
        y, state = selinv.selective_scan_ad(*args, **more)
    else:
        r = selinv.selective_scan(*args, **more)
        y, state = r["y"], r["state"]
    return y, conv_state, state


def test_prompts_then_tokens(cuda_ok):
    """A ragged batch of prompts, its states put into slots, then tokens one by one: the same as the whole sequences at
    once.  Both sides round the same products, in another order of rows, so they agree to the scan's own bound."""
    g = np.random.default_rng(7)
    t, d, n, k, steps = torch.float32, 48, 16, 4, 5
    w = layer_weights(g, t, d, n, k)
    lengths = [9, 1, 30]
    whole = [dev(g.standard_normal((m + steps, 2 * d)), t) for m in lengths]
    want = [layer(w, xz[None], n)[0][0] for xz in whole]
    packed = torch.cat([xz[:m] for xz, m in zip(whole, lengths)])
    y, conv_state, state = layer(w, packed, n, plan=selinv.SequencePlan(lengths))
    at = 0
    # matrix products of other sizes may round otherwise: 2^-24 * 4 * d relative to their terms, carried through the scan
    tol = 64 * d * unit(t) * (plain.PER_ROW + max(lengths))
    for m, ref in zip(lengths, want):
        assert float((y[at:at + m] - ref[:m]).abs().max()) <= tol * float(ref.abs().max())
        at += m
    index = torch.tensor([5, 2, 0], dtype=torch.int32, device="cuda")
    cache, conv_cache = torch.zeros(6, d, n, device="cuda"), torch.zeros(6, k - 1, d, device="cuda")
    cache[index.long()], conv_cache[index.long()] = state, conv_state
    for s in range(steps):
        xz = torch.stack([a[m + s] for a, m in zip(whole, lengths)])
        x, z = xz[:, :d], xz[:, d:]
        c = selinv.causal_conv_step(conv_cache, x, w["weight"], w["bias"], silu=True, index=index)
        bc = c @ w["to_bc"]
        y = selinv.selective_scan_step(cache, c, c @ w["to_dt"], w["A"], bc[:, None, :n], bc[:, None, n:], w["D"], z=z,
                                       dt_bias=w["dt_bias"], softplus=True, index=index)
        for r, (m, ref) in enumerate(zip(lengths, want)):
            assert float((y[r] - ref[m + s]).abs().max()) <= tol * float(ref.abs().max())


def test_chunked_prompt_equals_whole(cuda_ok):
    v, _, _ = scan_inputs(970, torch.float64, (1, 90), 24, 16, 1, states=(1,))
    more = dict(dt_bias=v["dt_bias"], softplus=True)
    whole = selinv.selective_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], z=v["z"], state=v["state"], **more)
    state, ys = v["state"], []
    for a, b in ((0, 1), (1, 33), (33, 90)):
        cut = {k: v[k][:, a:b] for k in ("x", "dt", "B", "C", "z")}      # strided, not copied
        r = selinv.selective_scan(cut["x"], cut["dt"], v["A"], cut["B"], cut["C"], v["D"], z=cut["z"], state=state, **more)
        state = r["state"]
        ys.append(r["y"])
    y = torch.cat(ys, 1)
    assert float((y - whole["y"]).abs().max()) <= 1e-12 * float(whole["y"].abs().max())
    assert float((state - whole["state"]).abs().max()) <= 1e-12 * float(whole["state"].abs().max())


def test_layer_gradients(cuda_ok):
    """Gradients through both operators and the products between them, against differences of the loss in float64
    (central: their error is the third derivative times eps^2, and the loss's rounding over eps)."""
    g = np.random.default_rng(8)
    t, d, n = torch.float64, 6, 4
    w = layer_weights(g, t, d, n, 3)
    xz = dev(g.standard_normal((2, 7, 2 * d)), t)
    wt = dev(g.standard_normal((2, 7, d)), t)
    leaves = {**{k: a.requires_grad_(True) for k, a in w.items()}, "xz": xz.requires_grad_(True)}

    def loss(ad):
        y, c, s = layer(w, xz, n, ad=ad)
        return (y * wt).sum() + s.sum() + (c * c).sum()

    loss(True).backward()
    rng = np.random.default_rng(9)
    for name, leaf in leaves.items():
        step = dev(rng.standard_normal(tuple(leaf.shape)), t)
        eps = 1e-6
        with torch.no_grad():
            leaf += eps * step
            up = float(loss(False))
            leaf -= 2 * eps * step
            down = float(loss(False))
            leaf += eps * step
        want = (up - down) / (2 * eps)
        got = float((leaf.grad * step).sum())
        assert abs(got - want) <= 1e-6 * (1 + abs(want)), name


@pytest.mark.parametrize("softplus,gate", [(True, True), (False, False)])
def test_gradcheck(cuda_ok, softplus, gate):
    v, _, _ = scan_inputs(980, torch.float64, (2, 5), 4, 3, 2, gate=gate, softplus=softplus, states=(2,))
    keys = [k for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "state") if v[k] is not None]

    def f(*a):
        w = dict(zip(keys, a))
        return selinv.selective_scan_ad(w["x"], w["dt"], w["A"], w["B"], w["C"], w["D"], z=w.get("z"),
                                        dt_bias=w["dt_bias"], softplus=softplus, state=w["state"])

    assert torch.autograd.gradcheck(f, [v[k].clone().requires_grad_(True) for k in keys])
    g = np.random.default_rng(3)
    a = [dev(g.standard_normal(s), torch.float64).requires_grad_(True) for s in ((9, 5), (5, 4), (5,), (3, 3, 5))]
    plan = selinv.SequencePlan([2, 6, 1])
    assert torch.autograd.gradcheck(lambda x, w, b, s: selinv.causal_conv_ad(x, w, b, silu=True, state=s, plan=plan), a)


def test_gradients_of_expanded_and_repeated_inputs(cuda_ok):
    """One row's dt for every row (stride 0), one tensor as x and z, and a loss whose cotangent is one number expanded."""
    v, _, _ = scan_inputs(990, torch.float64, (1, 6), 4, 3, 1)
    x = v["x"].clone().requires_grad_(True)
    row = v["dt"][:, :1].clone().requires_grad_(True)
    y, _ = selinv.selective_scan_ad(x, row.expand(1, 6, 4), v["A"], v["B"], v["C"], z=x)
    y.sum().backward()
    x2 = v["x"].clone().requires_grad_(True)
    z2 = v["x"].clone().requires_grad_(True)
    dt2 = row.detach().expand(1, 6, 4).contiguous().requires_grad_(True)
    y2, _ = selinv.selective_scan_ad(x2, dt2, v["A"], v["B"], v["C"], z=z2)
    y2.backward(torch.ones_like(y2))
    assert torch.allclose(x.grad, x2.grad + z2.grad, rtol=1e-14)
    assert torch.allclose(row.grad, dt2.grad.sum(1, keepdim=True), rtol=1e-13)


@pytest.mark.parametrize("scan", [False, True])
@pytest.mark.parametrize("dims", [(0,), (1,), (0, 1)])
def test_gradients_of_sums_over_leading_dimensions(cuda_ok, dims, scan):
    """The cotangent of y then repeats along some of the leading dimensions."""
    v, _, _ = scan_inputs(991, torch.float64, (2, 3, 6), 4, 3, 1)
    w = torch.randn(4, 3, dtype=torch.float64, device="cuda")
    grads = []
    for dense in (False, True):
        x = v["x"].clone().requires_grad_(True)
        u, _ = selinv.causal_conv_ad(x, w, silu=True)
        y = selinv.selective_scan_ad(v["x"], u, v["A"], v["B"], v["C"], z=v["z"], softplus=True)[0] if scan else u
        if dense:
            y.backward((2 * y.detach().sum(dims, keepdim=True)).expand(y.shape).contiguous())
        else:
            (y.sum(dims) ** 2).sum().backward()
        grads.append(x.grad)
    assert torch.allclose(grads[0], grads[1], rtol=1e-12, atol=1e-14)


# ---- strides, streams, graphs -------------------------------------------------


@pytest.mark.parametrize("shift", [0, 1, 3])
def test_strided_inputs_and_outputs(cuda_ok, shift):
    """Slices of wider arrays at any offset give what contiguous copies give."""
    t, rows, d, n = torch.bfloat16, 35, 40, 16
    g = np.random.default_rng(11)
    wide = dev(g.standard_normal((2, rows, 3 * d + 2 * n + 7)), t)
    cut = lambda at, m: wide[..., shift + at:shift + at + m]    # noqa: E731
    x, dt, z = cut(0, d), cut(d, d), cut(2 * d, d)
    B, C = cut(3 * d, n).unflatten(-1, (2, n // 2)), cut(3 * d + n, n).unflatten(-1, (2, n // 2))
    A = dev(-np.exp(g.standard_normal((d, n // 2))), torch.float32)
    w = dev(g.standard_normal((d, 4)), t)
    c = lambda a: a.contiguous()    # noqa: E731
    want = selinv.selective_scan(c(x), c(dt), A, c(B), c(C), z=c(z), softplus=True, keep=True)
    out = torch.full((2, rows, d + 5), 3.0, dtype=t, device="cuda")
    got = selinv.selective_scan(x, dt, A, B, C, z=z, softplus=True, keep=True, out={"y": out[..., shift:shift + d]})
    assert torch.equal(got["y"], want["y"]) and torch.equal(got["state"], want["state"])
    assert bool((out[..., :shift] == 3).all()) and bool((out[..., shift + d:] == 3).all())
    yb = cut(5, d)
    gw = selinv.selective_scan_backward(want["kept"], c(x), c(dt), A, c(B), c(C), c(yb), z=c(z), softplus=True)
    gg = selinv.selective_scan_backward(got["kept"], x, dt, A, B, C, yb, z=z, softplus=True)
    for k, a in gw.items():
        assert (a is None and gg[k] is None) or torch.equal(a, gg[k]), k
    cw, cg = selinv.causal_conv(c(x), w, silu=True), selinv.causal_conv(x, w, silu=True)
    assert torch.equal(cw["y"], cg["y"])
    bw, bg = selinv.causal_conv_backward(c(x), w, c(yb), silu=True), selinv.causal_conv_backward(x, w, yb, silu=True)
    assert torch.equal(bw["xb"], bg["xb"]) and torch.equal(bw["weightb"], bg["weightb"])


def test_rows_behind_the_plan_stay(cuda_ok):
    t = torch.float32
    v, yb, _ = scan_inputs(12, t, (20,), 8, 16, 1)
    for a in (v["x"], v["dt"], v["z"], v["B"], v["C"], yb):
        a[15:] = float("nan")
    plan = selinv.SequencePlan([10, 5])
    out = {"y": torch.full((20, 8), 5.0, device="cuda")}
    r = selinv.selective_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], z=v["z"], plan=plan, out=out, keep=True)
    assert bool((out["y"][15:] == 5).all()) and bool(torch.isfinite(out["y"]).all()) and bool(torch.isfinite(r["state"]).all())
    b = selinv.selective_scan_backward(r["kept"], v["x"], v["dt"], v["A"], v["B"], v["C"], yb, D=v["D"], z=v["z"], plan=plan)
    assert all(bool(torch.isfinite(a).all()) for a in b.values() if a is not None)
    w = torch.ones(8, 4, device="cuda")
    c = selinv.causal_conv(v["x"], w, plan=plan)
    assert bool(torch.isfinite(c["y"]).all()) and not c["y"][15:].any()
    cb = selinv.causal_conv_backward(v["x"], w, yb, plan=plan)
    assert bool(torch.isfinite(cb["xb"]).all()) and bool(torch.isfinite(cb["weightb"]).all())


def test_sequences_do_not_reach_one_another(cuda_ok):
    """A sequence of infinities and NaN between two others leaves them as they are, forward and backward."""
    lengths = [70, 90, 40]
    for d in (8, 20000):
        v, yb, _ = scan_inputs(13, torch.float32, (200,), d, 4, 1)
        plan = selinv.SequencePlan(lengths)
        run = lambda: selinv.selective_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], z=v["z"], plan=plan, keep=True)  # noqa: E731
        back = lambda r: selinv.selective_scan_backward(r["kept"], v["x"], v["dt"], v["A"], v["B"], v["C"], yb, D=v["D"],  # noqa: E731
                                                        z=v["z"], plan=plan)
        r0 = run()
        b0 = back(r0)
        v["x"][70:160:2] = float("inf")
        v["B"][71:160:3] = float("nan")
        yb[75:160:4] = float("inf")
        r1 = run()
        b1 = back(r1)
        keep = torch.cat([torch.arange(70), torch.arange(160, 200)]).cuda()
        assert torch.equal(r0["y"][keep], r1["y"][keep]) and torch.equal(r0["state"][[0, 2]], r1["state"][[0, 2]])
        for k in ("xb", "dtb", "Bb", "Cb", "zb"):
            assert torch.equal(b0[k][keep], b1[k][keep]), k


def test_results_repeat_bit_for_bit(cuda_ok):
    v, yb, _ = scan_inputs(14, torch.bfloat16, (2, 300), 200, 16, 1)
    args = (v["x"], v["dt"], v["A"], v["B"], v["C"])
    runs = []
    for _ in range(3):
        r = selinv.selective_scan(*args, v["D"], z=v["z"], keep=True)
        b = selinv.selective_scan_backward(r["kept"], *args, yb, D=v["D"], z=v["z"])
        runs.append([r["y"], r["state"]] + [b[k] for k in ("xb", "dtb", "Ab", "Bb", "Cb", "Db", "zb")])
    for other in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(runs[0], other))


def test_given_stream(cuda_ok):
    s = torch.cuda.Stream()
    v, yb, _ = scan_inputs(15, torch.float32, (2, 200), 40, 16, 1)
    args = (v["x"], v["dt"], v["A"], v["B"], v["C"])
    want = selinv.selective_scan(*args, v["D"], z=v["z"], keep=True)
    wb = selinv.selective_scan_backward(want["kept"], *args, yb, D=v["D"], z=v["z"])
    torch.cuda.synchronize()
    got = selinv.selective_scan(*args, v["D"], z=v["z"], keep=True, stream=s)
    gb = selinv.selective_scan_backward(got["kept"], *args, yb, D=v["D"], z=v["z"], stream=s)
    s.synchronize()
    assert torch.equal(want["y"], got["y"]) and torch.equal(wb["Ab"], gb["Ab"]) and torch.equal(wb["Bb"], gb["Bb"])
    assert torch.cuda.current_stream() != s


def test_captured_graph(cuda_ok):
    """Forward, backward and a step captured once and replayed on new contents; two graphs on one pool."""
    v, yb, _ = scan_inputs(16, torch.float32, (1, 700), 24, 16, 1)
    args = (v["x"], v["dt"], v["A"], v["B"], v["C"])
    w = torch.randn(24, 4, device="cuda")
    cache = torch.randn(3, 24, 16, device="cuda")
    new = torch.empty_like(cache)
    index = torch.tensor([2, 0], dtype=torch.int32, device="cuda")

    def run():
        c = selinv.causal_conv(v["x"], w, silu=True)["y"]
        r = selinv.selective_scan(c, *args[1:], v["D"], z=v["z"], keep=True)
        b = selinv.selective_scan_backward(r["kept"], c, *args[1:], yb, D=v["D"], z=v["z"])
        cb = selinv.causal_conv_backward(v["x"], w, b["xb"], silu=True)
        y = selinv.selective_scan_step(cache, v["x"][0, :2], v["dt"][0, :2], v["A"], v["B"][0, :2], v["C"][0, :2],
                                       index=index, cache_out=new, check=False)
        return [r["y"], r["state"], b["Ab"], b["Bb"], b["dtb"], cb["xb"], cb["weightb"], y, new]

    run()
    torch.cuda.synchronize()
    pool = torch.cuda.graph_pool_handle()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(run())
        graphs.append(g)
    v["x"].normal_()
    yb.normal_()
    cache.normal_()
    want = [a.clone() for a in run()]
    for g, o in zip(graphs, outs):
        new.zero_()
        g.replay()
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(want, o)):
            if i < len(want) - 1:
                assert torch.equal(p, q), i
        assert torch.equal(want[-1][[2, 0]], new[[2, 0]])
    with pytest.raises(ValueError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            selinv.selective_scan_step(cache, v["x"][0, :2], v["dt"][0, :2], v["A"], v["B"][0, :2], v["C"][0, :2], index=index)


# ---- refusals -----------------------------------------------------------------


def test_refusals(cuda_ok):
    v, yb, _ = scan_inputs(17, torch.float32, (2, 6), 8, 4, 2, states=(2,))
    args = dict(x=v["x"], dt=v["dt"], A=v["A"], B=v["B"], C=v["C"])

    def refuse(error, **change):
        a = {**args, **change}
        pos = [a.pop(k) for k in ("x", "dt", "A", "B", "C")]
        with pytest.raises(error):
            selinv.selective_scan(*pos, **a)

    refuse(ValueError, x=v["x"].cpu())
    refuse(TypeError, x=v["x"].int())
    refuse(TypeError, dt=v["dt"].half())
    refuse(ValueError, dt=v["dt"][:, :5])
    refuse(TypeError, A=v["A"].double())
    refuse(ValueError, A=v["A"].t())
    refuse(ValueError, B=v["B"][:, :, 0])
    refuse(ValueError, B=v["B"][..., :3])
    refuse(ValueError, B=v["B"].repeat(1, 1, 2, 1)[:, :, :3], C=v["C"].repeat(1, 1, 2, 1)[:, :, :3])
    refuse(ValueError, x=v["x"].transpose(1, 2).contiguous().transpose(1, 2))
    refuse(ValueError, D=torch.ones(9, device="cuda"))
    refuse(TypeError, state=v["state"].half())
    refuse(ValueError, state=v["state"][:1])
    refuse(ValueError, plan=selinv.SequencePlan([6]))
    refuse(ValueError, out={"state": v["state"]}, state=v["state"])
    refuse(ValueError, out={"y": v["x"]})
    refuse(ValueError, out={"y": torch.empty(1, 6, 8, device="cuda").expand(2, 6, 8)})
    big = torch.zeros(2, 6, 2, 65, device="cuda")
    refuse(selinv.SelinvError, A=torch.zeros(8, 65, device="cuda"), B=big, C=big)
    x = v["x"][0]
    with pytest.raises(ValueError):
        selinv.selective_scan(x, v["dt"][0], v["A"], v["B"][0], v["C"][0], plan=selinv.SequencePlan([7]))
    with pytest.raises(ValueError):
        selinv.SequencePlan([3, -1])
    r = selinv.selective_scan(*args.values(), keep=True)
    with pytest.raises(ValueError):
        selinv.selective_scan_backward(r["kept"][:-1], *args.values(), yb)
    with pytest.raises(ValueError):
        selinv.selective_scan_backward(r["kept"], *args.values(), yb[:, :5])
    w = torch.ones(8, 4, device="cuda")
    for bad in (torch.ones(8, 9, device="cuda"), torch.ones(8, 1, device="cuda")):
        with pytest.raises(selinv.SelinvError):
            selinv.causal_conv(v["x"], bad)
    with pytest.raises(TypeError):
        selinv.causal_conv(v["x"], w.half())
    with pytest.raises(ValueError):
        selinv.causal_conv(v["x"], w, state=torch.zeros(2, 4, 8, device="cuda"))
    with pytest.raises(ValueError):
        selinv.causal_conv(v["x"], w, out={"y": v["x"]})
    cache = torch.zeros(3, 3, 8, device="cuda")
    with pytest.raises(TypeError):
        selinv.causal_conv_step(cache, x, w, index=torch.zeros(6, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        selinv.causal_conv_step(cache, x, w)
    with pytest.raises(ValueError):
        selinv.causal_conv_step(cache, x[:2], w, cache_out=torch.zeros(4, 3, 8, device="cuda"))
    whole = torch.zeros(5, 3, 8, device="cuda")
    with pytest.raises(ValueError):
        selinv.causal_conv_step(whole[:3], x[:2], w, cache_out=whole[1:4])


def test_differentiable_calls_are_refused_in_a_capture(cuda_ok):
    """While an eager graph of the same leaves lives, too; the leaves and the eager graph are usable afterwards."""
    v, yb, _ = scan_inputs(18, torch.float32, (1, 9), 8, 4, 1)
    x = v["x"].clone().requires_grad_(True)
    w = torch.ones(8, 4, device="cuda", requires_grad=True)
    call = lambda: selinv.selective_scan_ad(x, v["dt"], v["A"], v["B"], v["C"])[0]     # noqa: E731
    y = call()
    c, _ = selinv.causal_conv_ad(x, w)
    torch.cuda.synchronize()
    for bad in (call, lambda: selinv.causal_conv_ad(x, w)):
        g = torch.cuda.CUDAGraph()
        with pytest.raises(ValueError):
            with torch.cuda.graph(g):
                bad()
    g = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(g):
        z = call()
    g.replay()
    (y.sum() + c.sum()).backward()
    torch.cuda.synchronize()
    assert torch.equal(z, y.detach()) and bool(torch.isfinite(x.grad).all()) and bool(torch.isfinite(w.grad).all())


def test_two_streams_at_once(cuda_ok):
    """Calls in flight together, of shapes that are cut differently, give what they give alone."""
    cases = [scan_inputs(20 + i, torch.float32, (2, rows), d, 16, 1)[:2] for i, (rows, d) in enumerate(((500, 40), (300, 900)))]

    def run(v, yb):
        args = (v["x"], v["dt"], v["A"], v["B"], v["C"])
        r = selinv.selective_scan(*args, v["D"], z=v["z"], keep=True)
        b = selinv.selective_scan_backward(r["kept"], *args, yb, D=v["D"], z=v["z"])
        return [r["y"], r["state"], b["xb"], b["Ab"], b["Bb"], b["Cb"]]

    want = [run(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(5):
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(run(*c))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


def test_workspace_is_the_callers(cuda_ok):
    """A workspace of the right size serves call after call; a smaller one is refused."""
    v, yb, _ = scan_inputs(22, torch.float32, (1, 600), 16, 16, 1)
    args = (v["x"], v["dt"], v["A"], v["B"], v["C"])
    want = selinv.selective_scan(*args, keep=True)
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        got = selinv.selective_scan(*args, keep=True, workspace=ws)
        b = selinv.selective_scan_backward(got["kept"], *args, yb, workspace=ws)
    assert torch.equal(got["y"], want["y"]) and bool(torch.isfinite(b["Ab"]).all())
    with pytest.raises(ValueError):
        selinv.selective_scan(*args, workspace=ws[:16])
    with pytest.raises(ValueError):
        selinv.selective_scan_backward(got["kept"], *args, yb, workspace=ws[:16])


def test_against_the_selected_inverse(cuda_ok):
    """Two rows of the scan are the solve of a block lower-bidiagonal system: the blocks that bidiag returns give them."""
    v, _, _ = scan_inputs(23, torch.float64, (1, 2), 3, 4, 1, gate=False, skip=False)
    step = torch.nn.functional.softplus(v["dt"][0] + v["dt_bias"])
    decay = torch.exp(step[1][:, None] * v["A"])
    eye = torch.eye(4, dtype=torch.float64, device="cuda").expand(3, 2, 4, 4).contiguous()
    lower = -torch.diag_embed(decay)[:, None].contiguous()
    g = selinv.bidiag(eye, lower)
    u = (step * v["x"][0])[:, :, None] * v["B"][0]                  # [row, channel, state]
    h1 = (g["G_lower"][:, 0] @ u[0][..., None] + g["G_diag"][:, 1] @ u[1][..., None])[..., 0]
    r = selinv.selective_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], dt_bias=v["dt_bias"], softplus=True)
    assert torch.allclose(r["state"][0], h1, rtol=1e-13, atol=1e-14)


def test_outputs_that_overlap_each_other_are_refused(cuda_ok):
    v, yb, _ = scan_inputs(18, torch.float32, (2, 6), 8, 4, 2, states=(2,))
    args = (v["x"], v["dt"], v["A"], v["B"], v["C"])
    kept = selinv.selective_scan(*args, keep=True)["kept"]
    one, bc = torch.empty_like(v["x"]), torch.empty_like(v["B"])
    for out in ({"xb": one, "dtb": one}, {"Bb": bc, "Cb": bc}, {"xb": one, "Bb": one.view(2, 6, 2, 4)}):
        with pytest.raises(ValueError):
            selinv.selective_scan_backward(kept, *args, yb, out=out)
    state = torch.empty(2, 8, 4, device="cuda")
    with pytest.raises(ValueError):
        selinv.selective_scan(*args, out={"state": state, "y": state.view(-1)[:1].expand(2, 6, 8)})
    flat = torch.empty(2 * 6 * 8 + 10, device="cuda")
    with pytest.raises(ValueError):
        selinv.causal_conv(v["x"], torch.ones(8, 4, device="cuda"),
                           out={"y": flat[:96].view(2, 6, 8), "state": flat[58:106].view(2, 3, 8)})


def test_offsets_beyond_32_bits(cuda_ok):
    """A cache of more than 2^31 elements, and rows and lines that lie as far apart: the same results as close by."""
    big = torch.empty(2 ** 31 + 2 ** 29 + 2 ** 21, device="cuda")
    v, yb, _ = scan_inputs(19, torch.float32, (3, 2), 64, 16, 1)
    args = [v["x"], v["dt"], v["A"], v["B"], v["C"]]
    far = big.as_strided((3, 2, 64), (2 ** 30, 2 ** 29, 1)).copy_(v["x"])
    r, s = (selinv.selective_scan(x, *args[1:], z=v["z"], keep=True) for x in (v["x"], far))
    assert torch.equal(r["y"], s["y"]) and torch.equal(r["state"], s["state"])
    out = {"xb": far}
    b = selinv.selective_scan_backward(r["kept"], *args, yb, z=v["z"])
    selinv.selective_scan_backward(r["kept"], *args, yb, z=v["z"], out=out)
    assert torch.equal(b["xb"], far)
    w = torch.randn(64, 4, device="cuda")
    far.copy_(v["x"])
    assert torch.equal(selinv.causal_conv(far, w)["y"], selinv.causal_conv(v["x"], w)["y"])
    x, dt, z, B, C = (v[k][:, 0].contiguous() for k in ("x", "dt", "z", "B", "C"))
    for shape, step in (((64, 16), lambda c, i: selinv.selective_scan_step(c, x, dt, v["A"], B, C, z=z, index=i)),
                        ((3, 64), lambda c, i: selinv.causal_conv_step(c, x, w, index=i))):
        size = shape[0] * shape[1]
        slots = big.numel() // size
        cache, near_by = big[:slots * size].view(slots, *shape), torch.randn(3, *shape, device="cuda")
        at = torch.tensor([slots - 1, 1, slots - 2], dtype=torch.int32, device="cuda")
        cache[at.long()] = near_by
        y = step(near_by, torch.arange(3, dtype=torch.int32, device="cuda"))
        assert torch.equal(step(cache, at), y) and torch.equal(cache[at.long()], near_by)
