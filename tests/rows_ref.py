"""Plain fp64 forms of the row operators, with their error bounds.

Every bound has two parts: half a step of the output's type, and the fp32
arithmetic before it. The second is K 2^-24 times the same formula taken over
absolute values, where K counts the roundings of one term:

- gate: forming gate + bias, its product with log2(e), the exponential, the
  sum 1 + e, the reciprocal and the last product are at most 1/2, 1, 2, 1/2, 2
  and 1/2 units of 2^-24 (instructions with one ulp count 2), of which the
  first two enter the exponent, so that they weigh |gate + bias| times: K =
  6 + 2 |gate + bias|.
- a step of the recurrence multiplies and adds: 2 more for h, the same again
  where the products of a block of rows are formed first and applied to the
  carried state later (4). The error of a step decays like the state, so it
  obeys the same recurrence.
- a row's sum of squares over at most 32 values per lane, then 6 levels over
  the lanes and 4 over the wavefronts: depth 48, halved by the square root;
  the root and reciprocal 4 more.
- a sum over rows, of n terms in any order: n units of the sum of absolute
  values (with fewer than that in fact).
"""

import numpy as np

U = 2.0 ** -24
HALF = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
# half the smallest subnormal step
TINY = {"float32": 2.0 ** -127, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -127}


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def rounded(value, err32, dtype):
    """Bound of an output of that type whose fp32 value is off by err32."""
    half = HALF[dtype]
    return err32 + half * (np.abs(value) + err32) + TINY[dtype]


def scan(x, g, off, bias=None, state=None, dh=None, dstate_out=None, dtype="float32"):
    """Outputs and bounds of the gated scan, as dicts; with dh its gradient
    too. Rows behind the last sequence are left NaN."""
    rows, c = x.shape
    n = len(off) - 1
    x = x.astype(np.float64)
    gb = g.astype(np.float64) + (0.0 if bias is None else bias.astype(np.float64))
    a, u = sigmoid(gb), sigmoid(-gb)
    k = 6.0 + 2.0 * np.abs(gb) + 4.0
    if bias is not None:
        k = k + 2.0 * np.abs(bias.astype(np.float64))
    h0 = np.zeros((n, c)) if state is None else state.astype(np.float64)
    h = np.full((rows, c), np.nan)
    prev, prev_err, prev_abs = h.copy(), h.copy(), h.copy()
    err = h.copy()
    out_state, err_state = h0.copy(), np.zeros((n, c))
    for j in range(n):
        v, e, m = h0[j], np.zeros(c), np.abs(h0[j])
        for t in range(off[j], off[j + 1]):
            prev[t], prev_err[t], prev_abs[t] = v, e, m
            v = a[t] * v + u[t] * x[t]
            m = a[t] * m + u[t] * np.abs(x[t])
            e = a[t] * e + k[t] * U * m
            h[t], err[t] = v, e
        out_state[j], err_state[j] = v, e
    val = dict(h=h, state_out=out_state)
    tol = dict(h=rounded(h, err, dtype), state_out=rounded(out_state, err_state, "float32"))
    if dh is None:
        return val, tol
    dx, dg = np.full((rows, c), np.nan), np.full((rows, c), np.nan)
    ex, eg, ag = dx.copy(), dx.copy(), np.zeros((rows, c))
    ds, es = np.zeros((n, c)), np.zeros((n, c))
    for j in range(n):
        carry = np.zeros(c) if dstate_out is None else dstate_out[j].astype(np.float64)
        e, m = np.zeros(c), np.abs(carry)
        for t in range(off[j + 1] - 1, off[j] - 1, -1):
            d = dh[t].astype(np.float64) + carry
            m = np.abs(dh[t].astype(np.float64)) + m
            e = e + 2 * U * m
            kt = k[t] * U
            dx[t] = u[t] * d
            ex[t] = u[t] * (e + kt * m)
            dg[t] = a[t] * u[t] * (prev[t] - x[t]) * d
            span = prev_abs[t] + np.abs(x[t])
            eg[t] = a[t] * u[t] * (prev_err[t] * m + span * e + 3 * kt * span * m)
            ag[t] = np.abs(dg[t]) + eg[t]
            carry = a[t] * d
            m = a[t] * m
            e = a[t] * e + kt * m
        ds[j], es[j] = carry, e
    last = int(off[-1])
    val.update(dx=dx, dgate=dg, dstate=ds, dbias=dg[:last].sum(0))
    tol.update(dx=rounded(dx, ex, dtype), dgate=rounded(dg, eg, dtype),
               dstate=rounded(ds, es, "float32"),
               dbias=eg[:last].sum(0) + last * U * ag.sum(0) + TINY["float32"])
    return val, tol


def norm(res, h=None, gate=None, w_post=None, scale=None, w_pre=None, eps=1e-6, dy=None, dz=None,
         grad=False, dtype="float32"):
    """Outputs and bounds of the block norm; with grad its gradients too."""
    f = np.float64
    res = res.astype(f)
    rows, c = res.shape
    one = np.ones(c)
    w_post = one if w_post is None else w_post.astype(f)
    scale = one if scale is None else scale.astype(f)
    w_pre = one if w_pre is None else w_pre.astype(f)
    ksum = 48 / 2 + 4.0
    y, ya = res, np.abs(res)
    ey = np.zeros_like(res)
    if h is not None:
        h = h.astype(f)
        r1 = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
        n = h * r1 * w_post
        kt = ksum + 4.0
        act, slope = np.ones_like(h), np.zeros_like(h)
        ko = np.zeros_like(h)
        if gate is not None:
            o = gate.astype(f)
            sg, ug = sigmoid(o), sigmoid(-o)
            act, slope = o * sg, sg * (1.0 + o * ug)
            ko = 8.0 + 2.0 * np.abs(o)
        t = n * act
        y = res + scale * t
        ya = np.abs(res) + np.abs(scale * t)
        et = (kt + ko) * U * np.abs(t)
        ey = np.abs(scale) * et + 3 * U * ya
    val, tol = {}, {}
    if h is not None:
        val["y"], tol["y"] = y, rounded(y, ey, dtype)
    r2 = 1.0 / np.sqrt((y * y).mean(1, keepdims=True) + eps)
    # relative error of r2: half that of the mean square, which takes y's
    m2 = (y * y).mean(1, keepdims=True) + eps
    er2 = ksum * U + (np.abs(y) * ey).mean(1, keepdims=True) / m2
    z = y * r2 * w_pre
    ez = np.abs(r2 * w_pre) * ey + np.abs(z) * (er2 + 3 * U)
    val["z"], tol["z"] = z, rounded(z, ez, dtype)
    if not grad:
        return val, tol
    d, ed = np.zeros_like(y), np.zeros_like(y)
    if dz is not None:
        dz = dz.astype(f)
        q = dz * w_pre
        mean = (q * y).mean(1, keepdims=True)
        mean_abs = np.abs(q * y).mean(1, keepdims=True)
        emean = (np.abs(q) * ey).mean(1, keepdims=True) + (2 * ksum) * U * mean_abs
        d = r2 * q - y * r2 ** 3 * mean
        ed = (np.abs(r2 * q) * (er2 + 4 * U) + ey * r2 ** 3 * np.abs(mean)
              + np.abs(y) * r2 ** 3 * (emean + np.abs(mean) * (3 * er2 + 6 * U)))
        p = dz * y * r2
        ep = np.abs(dz * r2) * ey + np.abs(p) * (er2 + 3 * U)
        val["dw_pre"] = p.sum(0)
        tol["dw_pre"] = ep.sum(0) + rows * U * (np.abs(p) + ep).sum(0)
    if dy is not None:
        ed = ed + 2 * U * (np.abs(d) + np.abs(dy.astype(f)))
        d = d + dy.astype(f)
    val["dres"], tol["dres"] = d, rounded(d, ed, dtype)
    if h is None:
        return val, tol
    da = np.abs(d) + ed
    if gate is not None:
        v = d * scale * n * slope
        # slope = s (1 + o u): its two terms may cancel
        sa = sg * (1.0 + np.abs(o) * ug)
        ev = np.abs(scale * n) * (ed * np.abs(slope) + da * sa * (kt + ko + 6) * U)
        val["dgate"], tol["dgate"] = v, rounded(v, ev, dtype)
    p = d * t
    ep = ed * np.abs(t) + da * (et + 2 * U * np.abs(t))
    val["dscale"] = p.sum(0)
    tol["dscale"] = ep.sum(0) + rows * U * (np.abs(p) + ep).sum(0)
    q = d * scale * act
    eq = np.abs(scale * act) * (ed + da * (ko + 4) * U)
    p = q * h * r1
    ep = eq * np.abs(h * r1) + np.abs(p) * (ksum + 4) * U
    val["dw_post"] = p.sum(0)
    tol["dw_post"] = ep.sum(0) + rows * U * (np.abs(p) + ep).sum(0)
    q, eq = q * w_post, eq * np.abs(w_post) + 2 * U * np.abs(q * w_post)
    mean = (q * h).mean(1, keepdims=True)
    emean = (eq * np.abs(h)).mean(1, keepdims=True)
    emean = emean + 2 * ksum * U * np.abs(q * h).mean(1, keepdims=True)
    v = r1 * q - h * r1 ** 3 * mean
    ev = (r1 * eq + np.abs(r1 * q) * (ksum + 4) * U
          + np.abs(h) * r1 ** 3 * (emean + np.abs(mean) * (3 * ksum + 8) * U))
    val["dh"], tol["dh"] = v, rounded(v, ev, dtype)
    return val, tol
