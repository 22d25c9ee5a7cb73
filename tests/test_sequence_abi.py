"""The sequence operators' C entry points reject bad arguments before anything is launched (no GPU needed), size their
buffers, and the binding's layout and refusals that need no device."""
import ctypes

import pytest
import torch

from sparse_spd_selected_b200 import build, selinv

FAKE = 1 << 20      # never dereferenced: validation fails first, or there is nothing to do


@pytest.fixture(scope="module")
def lib():
    build.build()
    return selinv.lib()


def scan_inputs(**change):
    v = dict(dtype=selinv.F32, flags=0, lines=2, rows=8, d=6, n=4, groups=2, sequences=0, live=0, table=0, x=FAKE, xl=48,
             xr=6, dt=FAKE, dtl=48, dtr=6, z=0, zl=0, zr=0, B=FAKE, Bl=64, Br=8, C=FAKE, Cl=64, Cr=8, Bg=4, Cg=4, A=FAKE,
             D=0, bias=0, state=0)
    v.update(change)
    return selinv._SCAN_INPUTS.pack(*v.values())


VIEW = selinv._VIEW.pack(FAKE, 48, 6)


def scan(lib, view=VIEW, state=0, kept=0, ws=0, nbytes=0, **change):
    return lib.selinv_selective_scan(scan_inputs(**change), view, state, kept, ws, nbytes, 0)


def test_scan_rejects(lib):
    bad = selinv.ERR_INVALID_ARG
    for change in (dict(dtype=4), dict(dtype=-1), dict(flags=2), dict(lines=-1), dict(rows=-1), dict(d=0), dict(n=0),
                   dict(groups=0), dict(groups=4), dict(x=0), dict(dt=0), dict(B=0), dict(C=0), dict(A=0), dict(x=FAKE + 2),
                   dict(z=FAKE + 1), dict(A=FAKE + 2), dict(D=FAKE + 1), dict(state=FAKE + 2), dict(xr=-6), dict(Bg=-1),
                   dict(xr=1 << 31), dict(view=selinv._VIEW.pack(0, 48, 6)), dict(state=FAKE + 2), dict(kept=FAKE + 1),
                   dict(ws=FAKE + 8)):
        assert scan(lib, **change) == bad, change
    assert lib.selinv_selective_scan(None, VIEW, 0, 0, 0, 0, 0) == bad
    assert scan(lib, n=65) == selinv.ERR_UNSUPPORTED
    assert scan(lib, d=(1 << 20) + 2) == selinv.ERR_UNSUPPORTED
    assert scan(lib, rows=(1 << 31)) == selinv.ERR_UNSUPPORTED
    # tables: one line, at most as many sequences with rows as sequences and as rows
    for change in (dict(lines=2), dict(live=5, sequences=4), dict(live=9, sequences=9), dict(live=0, sequences=1),
                   dict(live=1, sequences=-1), dict(table=FAKE + 4, live=1, sequences=1)):
        assert scan(lib, **{**dict(lines=1, table=FAKE, live=1, sequences=1), **change}) == bad, change
    assert scan(lib, lines=1, rows=4096, d=8, groups=2, ws=0) == selinv.ERR_WORKSPACE


def test_scan_backward_rejects(lib):
    bad = selinv.ERR_INVALID_ARG

    def call(g=None, ws=0, nbytes=0, **change):
        v = dict(kept=FAKE, yb=FAKE, ybl=48, ybr=6, stateb=0, xb=FAKE, xbl=48, xbr=6, dtb=FAKE, dtbl=48, dtbr=6, zb=0, zbl=0,
                 zbr=0, Bb=FAKE, Bbl=64, Bbr=8, Cb=FAKE, Cbl=64, Cbr=8, Bbg=4, Cbg=4, Ab=FAKE, Db=0, bias=0, state=0)
        v.update(g or {})
        return lib.selinv_selective_scan_backward(scan_inputs(**change), selinv._SCAN_GRADS.pack(*v.values()), ws, nbytes, 0)

    for g in (dict(kept=0), dict(yb=0), dict(xb=0), dict(dtb=0), dict(Bb=0), dict(Cb=0), dict(Ab=0), dict(Ab=FAKE + 2),
              dict(Bbg=-4), dict(stateb=FAKE + 1)):
        assert call(g) == bad, g
    assert call(z=FAKE, zl=48, zr=6) == bad             # a gate, but nowhere for its cotangent
    assert call() == selinv.ERR_WORKSPACE
    assert call(n=65) == selinv.ERR_UNSUPPORTED


def test_scan_buffers(lib):
    kept = lib.selinv_selective_scan_kept_size
    assert kept(scan_inputs(rows=1)) == 2 * 1 * 6 * 4 * 4
    assert kept(scan_inputs(rows=17)) == 2 * 2 * 6 * 4 * 4
    assert kept(scan_inputs(rows=16, dtype=selinv.F64)) == 2 * 1 * 6 * 4 * 8
    assert kept(scan_inputs(rows=16, dtype=selinv.BF16)) == 2 * 1 * 6 * 4 * 4
    f = lib.selinv_selective_scan_workspace_size
    assert f(scan_inputs(rows=16)) == 0                                  # too short to be cut
    assert f(scan_inputs(lines=64, d=4096, groups=1, rows=4096)) == 0    # fills the GPU as it is
    assert f(scan_inputs(lines=1, rows=4096)) > 0                        # few channels: cut into segments
    assert lib.selinv_selective_scan_backward_workspace_size(scan_inputs()) > 0


def step(**change):
    v = dict(dtype=selinv.F32, flags=0, batch=3, slots=3, d=6, n=4, groups=2, x=FAKE, dt=FAKE, z=0, B=FAKE, C=FAKE, xr=6,
             dtr=6, zr=0, Br=8, Cr=8, Bg=4, Cg=4, yr=6, A=FAKE, D=0, bias=0, cache=FAKE, out=FAKE, y=FAKE, index=0, info=0)
    v.update(change)
    return selinv._SCAN_STEP.pack(*v.values())


def test_steps_reject(lib):
    bad = selinv.ERR_INVALID_ARG
    f = lib.selinv_selective_scan_step
    for change in (dict(dtype=9), dict(flags=4), dict(batch=-1), dict(slots=2), dict(d=0), dict(n=0), dict(groups=5),
                   dict(x=0), dict(cache=0), dict(out=0), dict(y=0), dict(A=0), dict(x=FAKE + 1), dict(index=FAKE + 2),
                   dict(info=FAKE + 1), dict(xr=-1)):
        assert f(step(**change), 0) == bad, change
    assert f(step(n=65), 0) == selinv.ERR_UNSUPPORTED
    assert f(step(batch=0), 0) == selinv.OK
    assert f(None, 0) == bad

    def conv(**change):
        v = dict(dtype=selinv.F32, flags=0, batch=3, slots=3, d=6, k=4, x=FAKE, weight=FAKE, bias=0, cache=FAKE, xr=6, yr=6,
                 out=FAKE, y=FAKE, index=0, info=0)
        v.update(change)
        return lib.selinv_causal_conv_step(selinv._CONV_STEP.pack(*v.values()), 0)

    for change in (dict(dtype=5), dict(flags=1), dict(slots=2), dict(weight=0), dict(cache=0), dict(x=FAKE + 2), dict(yr=-1)):
        assert conv(**change) == bad, change
    assert conv(k=1) == selinv.ERR_UNSUPPORTED and conv(k=9) == selinv.ERR_UNSUPPORTED
    assert conv(batch=0) == selinv.OK


def test_conv_rejects(lib):
    bad = selinv.ERR_INVALID_ARG

    def inputs(**change):
        v = dict(dtype=selinv.F16, flags=0, lines=2, rows=8, d=6, k=4, sequences=0, live=0, table=0, x=FAKE, xl=48, xr=6,
                 weight=FAKE, bias=0, state=0)
        v.update(change)
        return selinv._CONV_INPUTS.pack(*v.values())

    f = lib.selinv_causal_conv
    for change in (dict(dtype=7), dict(flags=1), dict(lines=-1), dict(d=0), dict(k=0), dict(x=0), dict(weight=0),
                   dict(x=FAKE + 1), dict(state=FAKE + 1), dict(table=FAKE)):
        assert f(inputs(**change), VIEW, 0, 0) == bad, change
    assert f(inputs(), selinv._VIEW.pack(0, 48, 6), 0, 0) == bad
    for k in (1, 9):
        assert f(inputs(k=k), VIEW, 0, 0) == selinv.ERR_UNSUPPORTED
    g = lib.selinv_causal_conv_backward
    grads = dict(yb=FAKE, ybl=48, ybr=6, stateb=0, xb=FAKE, xbl=48, xbr=6, weightb=FAKE, biasb=0, state=0)
    for change in (dict(yb=0), dict(xb=0), dict(weightb=0), dict(weightb=FAKE + 2), dict(stateb=FAKE + 1)):
        assert g(inputs(), selinv._CONV_GRADS.pack(*{**grads, **change}.values()), 0, 0, 0) == bad, change
    assert g(inputs(), selinv._CONV_GRADS.pack(*grads.values()), 0, 0, 0) == selinv.ERR_WORKSPACE
    assert lib.selinv_causal_conv_backward_workspace_size(inputs()) >= 2 * 5 * 6 * 4


def test_no_lines_is_nothing_to_do(lib):
    assert scan(lib, lines=0) == selinv.OK


def test_binding_refuses_what_is_not_on_a_gpu():
    x = torch.zeros(2, 6, 8)
    with pytest.raises(ValueError):
        selinv.causal_conv(x, torch.zeros(8, 4))
    with pytest.raises(ValueError):
        selinv.selective_scan(x, x, torch.zeros(8, 4), torch.zeros(2, 6, 1, 4), torch.zeros(2, 6, 1, 4))
    with pytest.raises(ValueError):
        selinv.selective_scan_step(torch.zeros(2, 8, 4), x[:, 0], x[:, 0], torch.zeros(8, 4), torch.zeros(2, 1, 4),
                                   torch.zeros(2, 1, 4))
    with pytest.raises(ValueError):
        selinv.causal_conv_step(torch.zeros(2, 3, 8), x[:, 0], torch.zeros(8, 4))


def test_views_and_plans_on_the_host():
    t = torch.zeros(4, 3, 5, 7)
    assert selinv._view("t", t, 1)[1:] == (35, 7)
    assert selinv._view("t", t[:, :, 1:3, 2:5], 1)[1:] == (35, 7)
    assert selinv._view("t", t[:, 1:2], 1)[1:] == (105, 7)
    assert selinv._view("t", t, 2)[1:] == (105, 35)
    with pytest.raises(ValueError):
        selinv._view("t", t[:, :2], 1)                       # two leading strides that do not make one
    with pytest.raises(ValueError):
        selinv._view("t", t.transpose(2, 3), 1)              # channels not contiguous
    with pytest.raises(ValueError):
        selinv._view("t", t[:1].expand(4, 3, 5, 7), 1, True)     # an output that overlaps itself
    plan = selinv.SequencePlan([0, 3, 0, 2], device="cpu")
    assert plan.rows == 5 and plan.live == 2 and plan.table.tolist() == [0, 3, 5, 1, 3, 0, 2]
    a = torch.zeros(6, 8)
    selinv._apart("y", a[:, :4], (("x", a[:, 4:]),))
    for other in (a[:, 2:6], a[1:], a):
        with pytest.raises(ValueError):
            selinv._apart("y", a[:, :4], (("x", other),))


def test_repeated_leading_dimensions_are_refused():
    """A stride of 0 within the leading dimensions does not make one even stride with those outside it."""
    t = torch.zeros(4, 1, 5, 7)
    with pytest.raises(ValueError):
        selinv._view("t", t.expand(4, 3, 5, 7), 1)
    with pytest.raises(ValueError):
        selinv._view("t", t[:, 0].expand(3, 4, 5, 7), 1)
    assert selinv._view("t", t[:1].expand(4, 1, 5, 7), 1)[1:] == (0, 7)
    assert selinv._view("t", t[:1].expand(4, 3, 5, 7), 1)[1:] == (0, 7)
    assert selinv._view_or_copy(t.expand(4, 3, 5, 7)).is_contiguous()


def test_slices_of_one_array_are_told_apart():
    a = torch.zeros(6, 40)
    x, b, c = a[:, :16], a[:, 16:28].view(6, 2, 6), a[:, 28:].view(6, 2, 6)
    for name, t, others in (("b", b, (x, c)), ("c", c, (x, b)), ("x", x, (b, c)), ("x", x[1:4], (b[2:], x[4:]))):
        selinv._apart(name, t, [("u", u) for u in others])
    for t, u in ((b, a[:, 20:30].view(6, 2, 5)), (b, b[:, :1].expand(6, 2, 6)), (x, x), (x, a), (a.view(-1)[10:20], x),
                 (x, a.view(-1)[10:20]), (x, a[:, :1].expand(6, 16)), (x, a.view(torch.int32)[:, 16:])):
        with pytest.raises(ValueError):
            selinv._apart("t", t, [("u", u)])
    selinv._apart("x", x, [("u", a.view(-1)[17:39])])         # one piece inside a row's gap


def test_structures_match_the_header():
    """The packed structures have the header's sizes: every field is 8 bytes."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "selinv.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    sizes = {"selinv_view": 24}
    for body, name in re.findall(r"typedef struct \{([^}]*)\} (selinv_\w+);", src):
        total = 0
        for decl in body.split(";"):
            decl = decl.strip()
            if decl:
                kind = next((k for k in ("selinv_view",) if decl.startswith(k)), None)
                total += (24 if kind else 8) * (decl.count(",") + 1)
        sizes[name] = total
    for name, packed in (("selinv_scan_inputs", selinv._SCAN_INPUTS), ("selinv_scan_grads", selinv._SCAN_GRADS),
                         ("selinv_scan_step", selinv._SCAN_STEP), ("selinv_conv_inputs", selinv._CONV_INPUTS),
                         ("selinv_conv_grads", selinv._CONV_GRADS), ("selinv_conv_step", selinv._CONV_STEP),
                         ("selinv_view", selinv._VIEW)):
        assert packed.size == sizes[name], name
        assert ctypes.sizeof(ctypes.c_void_p) == 8
