"""The selective scan and the causal convolution from their definitions, in
float64 with numpy, one row after another, forward and backward; and bounds on
what rounding can do to a computation in fewer bits.

With `mag` the same formulas run on absolute values (the decays keep their
signs): what comes out bounds the sum of the magnitudes of all terms of an
output, so that an output of a chain of correctly rounded steps is off by at
most (roundings along the longest path) * (unit roundoff) * (that magnitude).
"""
import numpy as np


def sigmoid(v):
    return 1 / (1 + np.exp(-v))


def silu_slope(v):
    p = sigmoid(v)
    return p * (1 + v * (1 - p))


def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=False, state=None, yb=None, stateb=None, mag=False):
    """One sequence: x, dt, z, yb [rows, d], B, C [rows, groups, n], A [d, n], state, stateb [d, n].  Returns a dict of
    the forward's outputs and, with yb, of every cotangent."""
    f = np.abs if mag else (lambda v: v)
    rows, d = x.shape
    n, groups = A.shape[1], B.shape[1]
    of = np.arange(d) // (d // groups)
    raw = dt + (0 if dt_bias is None else dt_bias)
    step = np.logaddexp(raw, 0) if softplus else raw
    slope = sigmoid(raw) if softplus else np.ones_like(raw)
    decay = np.exp(step[:, :, None] * A)
    x, step, A = f(x), f(step), f(A)
    B, C = f(B[:, of]), f(C[:, of])
    D = np.zeros(d) if D is None else f(D)
    gate = np.ones_like(x) if z is None else f(z * sigmoid(z))
    h0 = np.zeros((d, n)) if state is None else f(state)
    u = (step * x)[:, :, None] * B
    h = np.empty((rows, d, n))
    now = h0
    for t in range(rows):
        now = decay[t] * now + u[t]
        h[t] = now
    inner = (h * C).sum(2) + D * x
    out = {"y": inner * gate, "state": now}
    if yb is None:
        return out
    yb = f(yb)
    ybg = yb * gate
    past = np.concatenate([h0[None], h])[:rows]
    g = np.empty_like(h)
    carry = np.zeros((d, n)) if stateb is None else f(stateb)
    for t in range(rows - 1, -1, -1):
        g[t] = C[t] * ybg[t][:, None] + carry
        carry = decay[t] * g[t]
    q = g * decay * past
    gb = (g * B).sum(2)
    rawb = (x * gb + (q * A).sum(2)) * slope
    per = (rows, groups, d // groups, n)
    out.update(xb=step * gb + D * ybg, dtb=rawb, Ab=(q * step[:, :, None]).sum(0), Db=(ybg * x).sum(0),
               Bb=(g * (step * x)[:, :, None]).reshape(per).sum(2), Cb=(h * ybg[:, :, None]).reshape(per).sum(2),
               dt_biasb=rawb.sum(0), stateb=carry)
    if z is not None:
        # silu' = p (1 + z (1 - p)) passes through zero at z = -1.278: the rounding of its sum is relative to
        # 1 + |z| (1 - p), so that is what bounds its terms
        p = sigmoid(z)
        out["zb"] = yb * inner * (p * (1 + np.abs(z) * (1 - p)) if mag else silu_slope(z))
    return out


def conv(x, weight, bias=None, silu=False, state=None, yb=None, stateb=None, mag=False):
    """One sequence: x, yb [rows, d], weight [d, k], state, stateb [k-1, d]."""
    f = np.abs if mag else (lambda v: v)
    rows, d = x.shape
    k = weight.shape[1]
    ext = np.concatenate([np.zeros((k - 1, d)) if state is None else state, x])
    pre = np.zeros((rows, d)) + (0 if bias is None else bias)
    for j in range(k):
        pre = pre + ext[j:j + rows] * weight[:, j]
    slope = silu_slope(pre) if silu else np.ones_like(pre)
    if mag:
        # the magnitude of pre's terms, carried through silu (its slope is at most 1.1)
        m = np.zeros((rows, d)) + (0 if bias is None else np.abs(bias))
        for j in range(k):
            m = m + np.abs(ext[j:j + rows] * weight[:, j])
        out = {"y": 1.1 * m + 0 * pre if silu else m, "state": np.abs(ext[rows:])}
        slope = 1.1 + 0.5 * m if silu else slope       # silu'' is at most 1/2
    else:
        out = {"y": pre * sigmoid(pre) if silu else pre, "state": ext[rows:]}
    if yb is None:
        return out
    ext, weight = f(ext), f(weight)
    prb = f(yb) * slope
    eb = np.zeros_like(ext)
    wb = np.zeros_like(weight)
    for j in range(k):
        eb[j:j + rows] += prb * weight[:, j]
        wb[:, j] = (prb * ext[j:j + rows]).sum(0)
    if stateb is not None:
        eb[rows:] += f(stateb)
    out.update(xb=eb[k - 1:], weightb=wb, biasb=prb.sum(0), stateb=eb[:k - 1])
    return out


# Roundings per row on the longest path of a scan in float: the step (softplus: 8), times A, times log2 e, the power of
# two (2^-22: 4 units) with its argument's error times the argument (at most 8 in the tests, so 8 * 3), two products
# and two sums.  Forward and backward chains have `rows` such steps each; the sums over n and over channels add their
# depth, the gates 8.
PER_ROW = 8 + 3 + 4 + 24 + 4


def scan_bound(rows, n, width, unit):
    return (2 * PER_ROW * (rows + 2) + n + width + 16) * unit


# the taps' sum, silu (two roundings of its exponential's argument times at most 8, 8 more) and the sums over rows
def conv_bound(rows, k, unit):
    return (4 * k + 40 + rows) * unit
