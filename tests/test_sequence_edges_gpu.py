"""Edges of the sequence operators on the GPU: empty plans, rows and widths at the limits, infinities, arguments far from
zero, and calls that have to be refused."""
import numpy as np
import pytest
import torch

from sparse_spd_selected_b200 import selinv
from tests import sequence_plain as plain
from tests.test_sequence_gpu import TYPES, arith, check_scan, dev, host, near, scan_inputs, unit

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_state", [False, True])
@pytest.mark.parametrize("tail", [0, 3])
def test_backward_of_sequences_without_rows(cuda_ok, with_state, tail):
    """A plan of sequences without rows: the final states' cotangents are the initial ones', all else is zero."""
    v, yb, stateb = scan_inputs(31, torch.float32, (tail,), 12, 5, 2, states=(2,))
    state = v["state"] if with_state else None
    plan = selinv.SequencePlan([0, 0])
    args = (v["x"], v["dt"], v["A"], v["B"], v["C"])
    more = dict(D=v["D"], z=v["z"], dt_bias=v["dt_bias"], softplus=True, state=state, plan=plan)
    r = selinv.selective_scan(*args, keep=True, **more)
    b = selinv.selective_scan_backward(r["kept"], *args, yb, stateb=stateb, **more)
    for k in ("xb", "dtb", "Bb", "Cb", "zb", "Ab", "Db", "dt_biasb"):
        assert not b[k].any(), k
    assert torch.equal(b["stateb"], stateb) if with_state else b["stateb"] is None
    w = torch.ones(12, 4, device="cuda")
    cs, csb = (dev(np.random.default_rng(i).standard_normal((2, 3, 12)), torch.float32) for i in (1, 2))
    c = selinv.causal_conv_backward(v["x"], w, yb, bias=v["D"], stateb=csb, state=cs if with_state else None, plan=plan)
    assert not c["xb"].any() and not c["weightb"].any() and not c["biasb"].any()
    assert torch.equal(c["stateb"], csb) if with_state else c["stateb"] is None


def test_gradients_of_sequences_without_rows(cuda_ok):
    v, _, stateb = scan_inputs(32, torch.float32, (0,), 12, 5, 2, states=(2,))
    leaves = {k: a.requires_grad_(True) for k, a in v.items()}
    y, state = selinv.selective_scan_ad(**leaves, softplus=True, plan=selinv.SequencePlan([0, 0]))
    ((state * stateb).sum() + y.sum()).backward()
    assert torch.equal(v["state"].grad, stateb)
    for k in ("A", "D", "dt_bias"):
        assert not v[k].grad.any(), k


MOST_ROWS = 2 ** 31 - 65


def repeated(value, *shape):
    return torch.full((1,) * len(shape), value, dtype=torch.float16, device="cuda").expand(*shape)


@pytest.mark.parametrize("rows", [MOST_ROWS, MOST_ROWS - 1400])
def test_scan_of_the_longest_lines(cuda_ok, rows):
    """One channel and one state over as many rows as a line may have: every row is written, and the final state.  The
    inputs are one row, repeated: h = a h + u with a = 1/2, u = 1/4, B = C = 1, so y is 1/2 but for the first rows."""
    x, dt, one = repeated(0.25, rows, 1), repeated(1.0, rows, 1), repeated(1.0, rows, 1, 1)
    A = torch.full((1, 1), -float(np.log(2.0)), device="cuda")
    out = {"y": torch.full((rows, 1), float("nan"), dtype=torch.float16, device="cuda")}
    r = selinv.selective_scan(x, dt, A, one, one, out=out)
    y = out["y"]
    # a is off by some units of float, y's last rounding is half a unit of float16
    assert abs(float(r["state"]) - 0.5) < 1e-6
    assert float((y[64:] - 0.5).abs().max()) <= 2.0 ** -11 and bool(torch.isfinite(y[:64]).all())


@pytest.mark.parametrize("rows", [MOST_ROWS, MOST_ROWS - 63])
def test_conv_of_the_longest_lines(cuda_ok, rows):
    """One channel over as many rows as a line may have, forward and backward; all sums are exact but weightb's."""
    x = repeated(0.5, rows, 1)
    w = torch.tensor([[1.0, 2.0, -4.0]], dtype=torch.float16, device="cuda")
    out = {"y": torch.full((rows, 1), float("nan"), dtype=torch.float16, device="cuda")}
    state = torch.full((2, 1), 0.25, dtype=torch.float16, device="cuda")
    r = selinv.causal_conv(x, w, state=state, out=out)
    assert bool((out["y"][2:] == -0.5).all()) and out["y"][:2, 0].tolist() == [-1.25, -0.75]
    assert r["state"][:, 0].tolist() == [0.5, 0.5]
    out = {"xb": out["y"].fill_(float("nan"))}
    b = selinv.causal_conv_backward(x, w, repeated(0.25, rows, 1), state=state, out=out)
    assert bool((out["xb"][:-2] == -0.25).all()) and out["xb"][-2:, 0].tolist() == [-0.5, -1.0]
    assert b["stateb"][:, 0].tolist() == [0.25, 0.75]
    # the sums: rows of 1/8 (less the states' rows), in chunks of at most 128 rows and 8 strands of those
    count = -(-rows // 128)
    bound = (128 + count / 8 + 8) * 2.0 ** -24
    ref = np.array([[2 * 0.25 * 0.25 + (rows - 2) * 0.125, 0.25 * 0.25 + (rows - 1) * 0.125, rows * 0.125]])
    assert (np.abs(host(b["weightb"]) - ref) <= bound * ref).all()
    assert abs(float(b["biasb"]) - 0.25 * rows) <= bound * 0.25 * rows


@pytest.mark.parametrize("kind,n,groups", [("bf16", 16, 1), ("f32", 32, 1), ("bf16", 64, 1), ("f32", 64, 4), ("f64", 32, 1)])
def test_scan_of_the_widest_layers(cuda_ok, kind, n, groups):
    """2^20 channels, forward and backward, at one row without a state: h = dt' x B in closed form."""
    t, d = TYPES[kind], 2 ** 20
    g = torch.Generator("cuda").manual_seed(n)
    x, dt, yb = (torch.randn(1, d, generator=g, device="cuda").to(t) for _ in range(3))
    B, C = (torch.randn(1, groups, n, generator=g, device="cuda").to(t) for _ in range(2))
    A, D = -torch.ones(d, n, dtype=arith(t), device="cuda"), torch.ones(d, dtype=arith(t), device="cuda")
    r = selinv.selective_scan(x, dt, A, B, C, D, softplus=True, keep=True)
    b = selinv.selective_scan_backward(r["kept"], x, dt, A, B, C, yb, D=D, softplus=True)
    x, dt, yb, B, C = (host(a)[0] for a in (x, dt, yb, B, C))

    def closed(f):
        step, slope = np.logaddexp(dt, 0), plain.sigmoid(dt)
        xs, ys, bs, cs = f(x), f(yb), f(B), f(C)
        bc = np.repeat((bs * cs).sum(1), d // groups)
        per = lambda v: v.reshape(groups, -1).sum(1)[:, None]      # noqa: E731
        return {"y": (bc * step + 1) * xs, "xb": (step * bc + 1) * ys, "dtb": xs * bc * ys * slope,
                "Bb": cs * per(ys * step * xs), "Cb": bs * per(ys * step * xs),
                "state": (step * xs)[-1000:, None] * bs[-1]}

    ref, mag = closed(lambda v: v), closed(np.abs)
    u = unit(arith(t))
    for k, got, width in (("y", r["y"][0], 0), ("state", r["state"][-1000:], 0), ("xb", b["xb"][0], 0), ("dtb", b["dtb"][0], 0),
                          ("Bb", b["Bb"][0], d), ("Cb", b["Cb"][0], d)):
        near(k, got, ref[k], mag[k], plain.scan_bound(1, n, width, u))
    assert not b["Ab"].any()


def same_infinities(name, got, ref, mag, bound):
    """Where the definition is finite the result is near it, where it is infinite it is that infinity."""
    got, finite = got.detach(), np.isfinite(ref) & np.isfinite(mag)
    assert tuple(got.shape) == ref.shape, name
    near(name, got[torch.from_numpy(finite).cuda()], ref[finite], mag[finite], bound)
    inf = np.isinf(ref)
    bad = host(got)[inf] != ref[inf]
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(inf)[bad][:4].tolist(), host(got)[inf][bad][:4])


@pytest.mark.parametrize("kind", ["f32", "bf16", "f64"])
@pytest.mark.parametrize("rows,d,n", [(60, 5, 1), (60, 40, 3), (37, 133, 12), (37, 7, 16), (50, 70, 33), (260, 6, 3)])
@pytest.mark.parametrize("what", ["x", "yb", "B", "C", "dt", "last"])
def test_infinities_stay_what_they_are(cuda_ok, kind, rows, d, n, what):
    """One infinite input of a line, all others positive: what the definition leaves finite or infinite is so in every
    output, whatever states and channels a tile has that do not exist."""
    t = TYPES[kind]
    v, yb, _ = scan_inputs(33, t, (1, rows), d, n, 1)
    for a in (v["x"], v["B"], v["C"], v["D"], v["z"], yb):
        a.copy_(0.5 + a.abs())
    at = rows // 2
    if what in ("x", "dt"):
        v[what][0, at, d - 1] = float("inf")
    elif what == "yb":
        yb[0, at, d - 1] = float("inf")
    elif what == "last":        # a state that no row takes up
        v["x"][0, rows - 1, 0] = float("inf")
    else:
        v[what][0, at, 0, n - 1] = float("inf")
    args, more = [v[k] for k in ("x", "dt", "A", "B", "C")], dict(z=v["z"], dt_bias=v["dt_bias"], softplus=True)
    r = selinv.selective_scan(*args, v["D"], keep=True, **more)
    b = selinv.selective_scan_backward(r["kept"], *args, yb, D=v["D"], **more)
    w = {k: host(a) if k in ("A", "D", "dt_bias", "state") else host(a)[0] for k, a in v.items()}
    with np.errstate(all="ignore"):
        ref, mag = (plain.scan(**w, softplus=True, yb=host(yb)[0], mag=m) for m in (False, True))
    u = unit(arith(t))
    bound, sums = plain.scan_bound(rows, n, d, u), plain.scan_bound(rows, n, d + rows, u)
    same_infinities("y", r["y"][0], ref["y"], mag["y"], bound)
    same_infinities("state", r["state"][0], ref["state"], mag["state"], bound)
    for k in ("xb", "dtb", "Bb", "Cb", "zb"):
        same_infinities(k, b[k][0], ref[k], mag[k], bound)
    for k in ("Ab", "Db", "dt_biasb"):
        same_infinities(k, b[k], ref[k], mag[k], sums)


@pytest.mark.parametrize("n", [3, 12])
def test_infinities_in_prompts_and_tokens(cuda_ok, n):
    """A prompt and single tokens agree on what becomes of an infinite input."""
    v, _, _ = scan_inputs(34, torch.float32, (40, 1), 9, n, 1)
    for k in ("B", "C", "D", "z"):
        v[k].abs_()
    v["x"][7, 0, 4] = float("inf")
    v["x"][20, 0, 6] = float("-inf")
    more = dict(dt_bias=v["dt_bias"], softplus=True)
    line = {k: v[k].transpose(0, 1) for k in ("x", "dt", "B", "C", "z")}
    r = selinv.selective_scan(line["x"], line["dt"], v["A"], line["B"], line["C"], v["D"], z=line["z"], **more)
    cache = torch.zeros(1, 9, n, device="cuda")
    for i in range(40):
        y = selinv.selective_scan_step(cache, v["x"][i], v["dt"][i], v["A"], v["B"][i], v["C"][i], v["D"], z=v["z"][i], **more)
        p = r["y"][:, i]
        assert torch.equal(torch.isinf(y), torch.isinf(p)) and not torch.isnan(p).any(), i
        assert torch.allclose(p, y, rtol=1e-4, atol=1e-5)
    assert torch.allclose(cache, r["state"], rtol=1e-4, atol=1e-5) and torch.isinf(cache).sum() == 2 * n


@pytest.mark.parametrize("kind", ["f32", "f64"])
def test_infinite_states_outlive_their_decay(cuda_ok, kind):
    """A line cut into segments, each of which decays a state by more than the type's range: an infinite state, and an
    infinite cotangent of one, stay infinite over all of them, as row after row, and other channels' vanish."""
    t, rows, d, n = TYPES[kind], 600, 6, 4
    step = 3.0 if kind == "f32" else 30.0
    v, yb, stateb = scan_inputs(35, t, (1, rows), d, n, 1, softplus=False, bias=False, skip=False, states=(1,))
    v["A"].fill_(-2)
    v["dt"].fill_(step)
    for a in (v["x"], v["B"], v["C"], v["z"], yb):
        a.copy_(0.5 + a.abs())
    v["x"][0, 5, 1] = float("inf")
    stateb[0, 3] = float("inf")
    args = [v[k] for k in ("x", "dt", "A", "B", "C")]
    assert selinv.lib().selinv_selective_scan_workspace_size(
        selinv._scan_inputs(*args, None, v["z"], None, False, v["state"], None)[0]) > 0      # it is cut
    r = selinv.selective_scan(*args, z=v["z"], state=v["state"], keep=True)
    b = selinv.selective_scan_backward(r["kept"], *args, yb, z=v["z"], state=v["state"], stateb=stateb)
    w = {k: host(a) if a is None or k == "A" else host(a)[0] for k, a in v.items()}
    with np.errstate(all="ignore"):
        ref, mag = (plain.scan(**w, yb=host(yb)[0], stateb=host(stateb)[0], mag=m) for m in (False, True))
    assert np.isinf(ref["state"][1]).all() and np.isinf(ref["stateb"][3]).all() and np.isfinite(ref["state"][0]).all()
    # the decays' arguments are 2 steps a row: an error of three units each is that many units of what is left of a state
    u = unit(arith(t))
    bound = plain.scan_bound(1, n, d, u) + 8 * 2 * step * u
    for k in ("y", "xb", "zb"):
        same_infinities(k, r[k][0] if k == "y" else b[k][0], ref[k], mag[k], bound)
    same_infinities("state", r["state"][0], ref["state"], mag["state"], bound)
    same_infinities("stateb", b["stateb"][0], ref["stateb"], mag["stateb"], bound)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f64"])
@pytest.mark.parametrize("k", [2, 4, 7])
def test_conv_infinities_next_to_a_chunks_end(cuda_ok, kind, k):
    """Each channel has one infinite input, in a row of its own: the chunk before it, which reads it for its last rows'
    cotangents, does not make something else of weightb."""
    t, rows = TYPES[kind], 200
    g = np.random.default_rng(36)
    x, yb = (dev(0.5 + g.random((1, rows, rows)), t) for _ in range(2))
    weight = dev(0.5 + g.random((rows, k)), t)
    x[0].diagonal().fill_(float("inf"))
    r = selinv.causal_conv(x, weight)
    b = selinv.causal_conv_backward(x, weight, yb)
    with np.errstate(all="ignore"):
        ref, mag = (plain.conv(host(x)[0], host(weight), yb=host(yb)[0], mag=m) for m in (False, True))
    u = unit(arith(t))
    same_infinities("y", r["y"][0], ref["y"], mag["y"], plain.conv_bound(0, k, u))
    same_infinities("xb", b["xb"][0], ref["xb"], mag["xb"], plain.conv_bound(0, k, u))
    for key in ("weightb", "biasb"):
        same_infinities(key, b[key], ref[key], mag[key], plain.conv_bound(rows, k, u))


def relative(got, ref):
    """Errors in units of float's rounding (2^-24), relative to each value."""
    return np.abs(host(got).reshape(ref.shape) - ref) / np.abs(ref) / 2.0 ** -24


def spread_out(lo, hi, count, seed):
    """Values over a range, and close to zero and to the whole numbers within it."""
    g = np.random.default_rng(seed)
    v = np.concatenate([g.uniform(lo, hi, count), g.uniform(max(lo, -1.0), min(hi, 1.0), count // 4),
                        np.arange(np.ceil(lo), np.floor(hi) + 1), [2.0 ** -i for i in range(40) if lo <= 2.0 ** -i <= hi],
                        [-2.0 ** -i for i in range(40) if lo <= -2.0 ** -i <= hi]])
    return v.astype(np.float32)


def row_of(dt, z=None, A=None, state=None, x=1.0, D=None):
    """One row with a channel per value of dt, one state, B = C = 1: forward with its kept states, and the arguments."""
    d = dt.numel()
    one = torch.ones(1, 1, 1, device="cuda")
    xs = torch.full((1, d), x, device="cuda")
    A = torch.zeros(d, 1, device="cuda") if A is None else A
    args = (xs, dt[None], A, one, one)
    return args, dict(z=None if z is None else z[None], D=D, state=state)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_steps_from_16_bits_far_from_zero(cuda_ok, kind):
    """Steps that the float biases carry far from zero: 1.3 units of |x| more, for the argument's roundings."""
    v = spread_out(-86.5, 86.5, 40000, 1)
    ref = np.logaddexp(v.astype(np.float64), 0)
    t = TYPES[kind]
    one, x = torch.ones(1, 1, 1, dtype=t, device="cuda"), torch.ones(1, v.size, dtype=t, device="cuda")
    args = (x, torch.zeros_like(x), torch.zeros(v.size, 1, device="cuda"), one, one)
    more = dict(dt_bias=torch.from_numpy(v).cuda(), softplus=True)
    cache = torch.zeros(1, v.size, 1, device="cuda")
    selinv.selective_scan_step(cache, *args, **more)
    for name, got in (("state", selinv.selective_scan(*args, **more)["state"]), ("cache", cache)):
        assert (relative(got, ref) <= 12 + 1.3 * np.abs(v)).all(), name


def test_steps_far_from_zero(cuda_ok):
    """softplus over its whole range, to a few units relative to the step itself, in every kernel that forms it.

    With A = 0, x = B = 1 and no state the state is the step, with C = 1 and yb = 1 so is xb.  Its roundings: the power of
    two 4 units, the correction of its argument 1, the polynomial 1 for its fit and 3 for its arithmetic, the sum 1, and
    the kernels' products 2."""
    v = spread_out(-86.5, 86.5, 40000, 1)
    ref = np.logaddexp(v.astype(np.float64), 0)
    dt = torch.from_numpy(v).cuda()
    args, more = row_of(dt)
    r = selinv.selective_scan(*args, softplus=True, keep=True)
    b = selinv.selective_scan_backward(r["kept"], *args, torch.ones_like(args[0]), softplus=True)
    cache = torch.zeros(1, v.size, 1, device="cuda")
    selinv.selective_scan_step(cache, *args, softplus=True)
    for name, got in (("state", r["state"]), ("xb", b["xb"]), ("cache", cache)):
        off = relative(got, ref)
        assert off.max() <= 12, (name, off.max(), v[off.argmax()])
    # dt's cotangent is the sigmoid: the argument of its power is off by 1.3 units of itself, so e^-x by 1.3 |x|; 4 for the
    # power, 1 for the sum, 2 for the reciprocal and 1 for the product
    off = relative(b["dtb"], 1 / (1 + np.exp(-v.astype(np.float64))))
    assert (off <= 8 + 1.3 * np.abs(v)).all(), (off - 1.3 * np.abs(v)).max()


def test_gates_far_from_zero(cuda_ok):
    """silu over its whole range: y of a state that is not read and D = x = 1 in the scan, of a single tap in the
    convolution.  The sigmoid's roundings are those above, with 2 more products."""
    v = spread_out(-86.5, 100.0, 40000, 2)
    w = v.astype(np.float64)
    keep = w != 0
    ref = w / (1 + np.exp(-w))
    bound = 10 + 1.3 * np.abs(w)
    z = torch.from_numpy(v).cuda()
    zero = torch.zeros_like(z)
    args, more = row_of(zero, z=z, D=torch.ones_like(z))
    y = selinv.selective_scan(*args, **more)["y"]
    token = selinv.selective_scan_step(torch.zeros(1, v.size, 1, device="cuda"), *args, more["D"], z=more["z"])
    taps = torch.tensor([[0.0, 1.0]], device="cuda").expand(v.size, 2).contiguous()
    conv = selinv.causal_conv(z[None], taps, silu=True)["y"]
    tap = selinv.causal_conv_step(torch.zeros(1, 1, v.size, device="cuda"), z[None], taps, silu=True)
    for name, got in (("scan", y), ("scan step", token), ("conv", conv), ("conv step", tap)):
        off = relative(got[0].cpu()[keep], ref[keep])
        assert (off <= bound[keep]).all(), (name, (off - bound[keep]).max())
        assert not host(got)[0][~keep].any(), name
    assert torch.equal(selinv.causal_conv(torch.full((1, 8), -1e4, device="cuda"), taps[:8], silu=True)["y"],
                       torch.zeros(1, 8, device="cuda"))


def test_decays_far_from_zero(cuda_ok):
    """exp(dt' A) over its whole range: of a state of one with x = 0 it is what is left.  The argument is off by 2.3 units of
    itself (A log2 e, the product, log2 e's own rounding), the power by 4, the state's product by 1, 1 to spare."""
    v = spread_out(-86.0, 0.0, 40000, 3)
    v = v[v < 0]
    dt, A = torch.from_numpy(-v).cuda(), -torch.ones(v.size, 1, device="cuda")
    state = torch.ones(v.size, 1, device="cuda")
    ref = np.exp(v.astype(np.float64))
    args, more = row_of(dt, A=A, x=0.0, state=state)
    r = selinv.selective_scan(*args, **more, keep=True)
    b = selinv.selective_scan_backward(r["kept"], *args, torch.ones_like(args[0]), state=state)
    cache = state.clone()[None]
    selinv.selective_scan_step(cache, *args)
    for name, got in (("state", r["state"]), ("stateb", b["stateb"]), ("cache", cache)):
        off = relative(got, ref)
        assert (off <= 6 + 2.3 * np.abs(v)).all(), (name, (off - 2.3 * np.abs(v)).max())


@pytest.mark.parametrize("kind", ["f32", "bf16", "f64"])
@pytest.mark.parametrize("rows,d", [(700, 8), (40, 3000)])
def test_rows_without_a_step_leave_the_state(cuda_ok, kind, rows, d):
    """dt' = 0, as in a padded batch: the state stays bit for bit what it is, and so does its cotangent on the way back."""
    t, n = TYPES[kind], 5
    v, yb, stateb = scan_inputs(37, t, (1, rows), d, n, 1, softplus=False, bias=False, states=(1,))
    v["dt"].zero_()
    yb.zero_()
    args = [v[k] for k in ("x", "dt", "A", "B", "C")]
    r = selinv.selective_scan(*args, v["D"], z=v["z"], state=v["state"], keep=True)
    b = selinv.selective_scan_backward(r["kept"], *args, yb, D=v["D"], z=v["z"], state=v["state"], stateb=stateb)
    assert torch.equal(r["state"], v["state"]) and torch.equal(b["stateb"], stateb)
    assert not b["xb"].any() and not b["Ab"].any() and not b["Bb"].any()
    cache = v["state"].clone()
    selinv.selective_scan_step(cache, v["x"][:, 0], v["dt"][:, 0], v["A"], v["B"][:, 0], v["C"][:, 0])
    assert torch.equal(cache, v["state"])


def test_workspaces_that_cannot_be_are_refused(cuda_ok):
    """On the host, in pieces, off 16 bytes, or shared with an input or an output: refused before anything is launched."""
    v, yb, _ = scan_inputs(38, torch.float32, (1, 600), 16, 16, 1)
    args = [v[k] for k in ("x", "dt", "A", "B", "C")]
    r = selinv.selective_scan(*args, keep=True)
    size = 1 << 22
    ws = torch.zeros(2 * size, dtype=torch.uint8, device="cuda")
    inner = ws[:600 * 16 * 4].view(torch.float32).view(1, 600, 16)
    w = torch.ones(16, 4, device="cuda")
    forward = lambda **k: selinv.selective_scan(*args, **k)                                     # noqa: E731
    backward = lambda **k: selinv.selective_scan_backward(r["kept"], *args, yb, **k)            # noqa: E731
    conv = lambda **k: selinv.causal_conv_backward(v["x"], w, yb, **k)                          # noqa: E731
    for call, key in ((forward, "y"), (backward, "xb"), (conv, "xb")):
        for bad in (torch.zeros(size, dtype=torch.uint8), ws[::2], ws[4:size], "here", np.zeros(size, np.uint8)):
            with pytest.raises(ValueError):
                call(workspace=bad)
        with pytest.raises(ValueError):
            call(workspace=ws, out={key: inner})
        call(workspace=ws[size:], out={key: inner})
        call(workspace=ws.view(torch.float64))
    whole = torch.zeros(size + 600 * 16, device="cuda")
    x = whole[-600 * 16:].view(1, 600, 16)
    for call in (lambda k: selinv.selective_scan(x, *args[1:], workspace=k),
                 lambda k: selinv.selective_scan_backward(r["kept"], x, *args[1:], yb, workspace=k),
                 lambda k: selinv.causal_conv_backward(x, w, yb, workspace=k)):
        with pytest.raises(ValueError):
            call(whole)
        call(whole[:size])


def test_missing_tensors_are_refused(cuda_ok):
    """What a call cannot do without, given as None or as something else: a ValueError that names it."""
    v, yb, _ = scan_inputs(39, torch.float32, (2, 6), 8, 4, 2, states=(2,))
    full = {k: v[k] for k in ("x", "dt", "A", "B", "C")}
    kept = selinv.selective_scan(*full.values(), keep=True)["kept"]
    token = {k: a if k == "A" else a[:, 0] for k, a in full.items()}
    w, x = torch.ones(8, 4, device="cuda"), v["x"]
    cache = torch.zeros(2, 3, 8, device="cuda")
    for bad in (None, [1.0], np.zeros(3)):
        for k in full:
            for call in (lambda a: selinv.selective_scan(*a), lambda a: selinv.selective_scan_backward(kept, *a, yb)):
                with pytest.raises(ValueError, match=f"^{k} "):
                    call(list({**full, k: bad}.values()))
            with pytest.raises(ValueError, match=f"{k} must|{k} \\["):
                selinv.selective_scan_step(v["state"].clone(), *{**token, k: bad}.values())
        for call in (lambda: selinv.selective_scan_backward(kept, *full.values(), bad), lambda: selinv.causal_conv(bad, w),
                     lambda: selinv.selective_scan_backward(bad, *full.values(), yb), lambda: selinv.causal_conv(x, bad),
                     lambda: selinv.causal_conv_backward(x, w, bad), lambda: selinv.causal_conv_step(cache, bad, w),
                     lambda: selinv.causal_conv_step(bad, x[:, 0], w), lambda: selinv.causal_conv_step(cache, x[:, 0], bad)):
            with pytest.raises(ValueError):
                call()
    with pytest.raises(ValueError):
        selinv.causal_conv_step(cache, x[:, 0], w, cache_out=[1.0])
    with pytest.raises(ValueError):
        selinv.causal_conv(x[0], w, plan=[4, 2])


def test_steps_whose_inputs_lie_in_the_cache_are_refused(cuda_ok):
    """Rows are done in no order, so an input that another row's new state replaces is no input.  What lies beside the
    cache, or in a cache that is only read, is one."""
    whole = torch.randn(6, 3, 8, device="cuda")
    cache, w = whole[:4], torch.ones(8, 4, device="cuda")
    index = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    x = torch.randn(3, 8, device="cuda")
    conv = lambda x, c=cache, w=w, i=index, **k: selinv.causal_conv_step(c, x, w, index=i, **k)     # noqa: E731
    for bad in (dict(x=cache[1:, -1]), dict(x=cache[:3, 0], cache_out=cache), dict(x=whole[3:, 0]),
                dict(x=x, w=cache.view(-1)[:32].view(8, 4)), dict(x=x, i=cache.view(torch.int32).view(-1)[:3])):
        with pytest.raises(ValueError, match="overlap"):
            conv(**bad)
    before = cache.clone()
    other = torch.zeros_like(cache)
    y = conv(cache[:3, -1].clone(), cache_out=other)
    assert torch.equal(conv(cache[:3, -1], cache_out=other.clone()), y) and torch.equal(cache, before)
    conv(whole[4:, 0].expand(2, 8)[[0, 1, 0]])
    conv(torch.empty_strided((3, 8), (24, 1), device="cuda").copy_(x))
    v, _, _ = scan_inputs(40, torch.float32, (3, 1), 8, 2, 2)
    a = {k: b[:, 0] if k in ("x", "dt", "B", "C", "z") else b for k, b in v.items() if k != "state"}
    states = torch.randn(5, 8, 2, device="cuda")
    flat = states.view(-1)
    part = {"x": flat[8:32].view(3, 8), "dt": flat[56:80].view(3, 8), "B": flat[2:14].view(3, 2, 2),
            "C": flat[-12:].view(3, 2, 2), "A": states[1], "z": flat[:24].view(3, 8), "D": flat[70:78], "dt_bias": flat[:8]}
    for k, bad in part.items():
        with pytest.raises(ValueError, match=f"^{k} must not overlap"):
            selinv.selective_scan_step(states, **{**a, k: bad}, index=index)
        ok = selinv.selective_scan_step(states, **{**a, k: bad}, index=index, cache_out=torch.empty_like(states))
        assert torch.equal(ok, selinv.selective_scan_step(states.clone(), **{**a, k: bad.clone()}, index=index)), k
    assert selinv.selective_scan_step(states, **{k: b[:0] if k in ("x", "dt", "B", "C", "z") else b
                                                 for k, b in a.items()}).shape == (0, 8)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lines,rows,d,n,cut", [
    # blocks of the forward at one lane per channel, on 148 multiprocessors: 258, 157 and 213 leave lines whole, with one
    # lane, two and two
    (2, 18, 16400, 16, False), (1, 18, 20001, 16, False), (3, 18, 9000, 7, False),
    # 112, 60 and 3 have them cut, with one lane, two and four
    (1, 260, 14300, 5, True), (1, 260, 7600, 9, True), (1, 150, 300, 16, True),
    # more states: no fewer than two lanes, or four
    (1, 150, 300, 20, True), (1, 150, 70, 40, True), (2, 18, 2400, 33, False),
])
def test_scan_dispatch(cuda_ok, kind, lines, rows, d, n, cut):
    """Sizes on each side of the rules that choose lanes and segments, with channels that end inside a tile."""
    shape = selinv._SCAN_INPUTS.pack(selinv.F32 if kind == "f32" else selinv.BF16, 0, lines, rows, d, n, 1, 0, 0, 0,
                                     *[0, 0, 0] * 5, 0, 0, 0, 0, 0, 0)
    assert (selinv.lib().selinv_selective_scan_workspace_size(shape) > 0) == cut
    check_scan(41, kind, [rows] * lines, d, n, with_state=True)
