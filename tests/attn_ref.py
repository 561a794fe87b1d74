"""Plain fp64 forms of linear attention and the group norm, with their error
bounds, as in rows_ref.py: half a step of the output's type, and the fp32
arithmetic before it as K 2^-24 times the same formula over absolute values.

Linear attention. A term of o_i is lambda^(i-j) (q_i . k_j) v_j. Its weight is
formed row by row, or as one exponential a chunk and more when the state is
carried: each of the i - j + 1 steps gives at most 6 + 2 |log_decay| roundings
(the power: the exponent's product, of which |log_decay| an ulp, an exponential
of 2, the products it enters). The products are summed over dk values, over the
64 rows of a chunk and over dk values again: that many additions, and 8 for the
scale and the sums' joins. Products on the matrix cores take their operands in
bf16 pieces. Rows of 16 bits: what is not a row operand itself (a weighted row,
a score, the state) is two pieces or three, which leave up to 2^-18 of it, 64
units of 2^-24, for each of the three such roundings that a term meets; an fp16 row is two
pieces too, and the product of two second pieces is left out, 64 more for each
of the three products. fp32 rows: three pieces each, which leave 2^-26 and drop
products below 2^-25: a unit for each of six.
"""

import numpy as np

from tests.rows_ref import TINY, U, rounded, sigmoid

PIECES = {"float32": 6.0, "bfloat16": 3 * 64.0, "float16": 6 * 64.0}


def _powers(g, n):
    """e^(g n), 1 at n = 0 whatever g is, 0 at negative n."""
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.exp(np.where(n > 0, g * n, 0.0))
    return np.where(n >= 0, p, 0.0)


def _job(a, b, c, g, w0, first, beta, gamma, pieces):
    """One head of one sequence: o_i = beta a_i W_i, W_i = lambda W_{i-1} +
    gamma b_i c_i^T, the first row decaying w0 `first` times (0 or 1). Returns
    o, its fp32 error, the last W and its error."""
    n = len(a)
    i = np.arange(n)
    kappa = 6.0 + 2.0 * min(abs(g), 50.0)
    deep = a.shape[1] * 2 + 64 + 8 + pieces
    age = i[:, None] - i
    d = _powers(g, age)
    p, pa = a @ b.T, np.abs(a) @ np.abs(b).T
    steps = kappa * np.maximum(age + 1, 0) + deep
    enter = _powers(g, i + first)[:, None]
    ca, w0a = np.abs(c), np.abs(w0)
    o = gamma * ((p * d) @ c) + enter * (a @ w0)
    e = abs(gamma) * ((pa * d * steps) @ ca)
    e = e + (kappa * (i + 2) + deep)[:, None] * enter * (np.abs(a) @ w0a)
    if n == 0:
        return beta * o, abs(beta) * U * e, w0, np.zeros_like(w0)
    leave = _powers(g, n - 1 - i)[:, None]
    whole = _powers(g, np.array(n - 1 + first))
    w = gamma * ((b * leave).T @ c) + whole * w0
    ew = abs(gamma) * ((np.abs(b) * leave * (kappa * (n - i) + deep)[:, None]).T @ ca)
    ew = ew + (kappa * (n + 1) + deep) * whole * w0a
    return beta * o, abs(beta) * U * e, w, U * ew


def attention(q, k, v, log_decay, off, qk_heads, scale, state=None, do=None, dstate_out=None,
              dtype="float32"):
    """Outputs and bounds of linear attention, as dicts; with do its gradient
    too. Rows behind the last sequence are left NaN."""
    f = np.float64
    heads = len(log_decay)
    rows, share = q.shape[0], heads // qk_heads
    dk, dv = q.shape[1] // qk_heads, v.shape[1] // heads
    n_seq = len(off) - 1
    q, k = (t.astype(f).reshape(rows, qk_heads, dk) for t in (q, k))
    v = v.astype(f).reshape(rows, heads, dv)
    g = log_decay.astype(f)
    zero = np.zeros((n_seq, heads, dk, dv))
    s0 = zero if state is None else state.astype(f)
    pieces = PIECES[dtype]
    o, eo = np.full((rows, heads, dv), np.nan), np.full((rows, heads, dv), np.nan)
    out, eout = s0.copy(), zero.copy()
    if do is not None:
        do = do.astype(f).reshape(rows, heads, dv)
        t0 = zero if dstate_out is None else dstate_out.astype(f)
        dq, dk_ = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
        eq, ek = dq.copy(), dq.copy()
        aq, ak = dq.copy(), dq.copy()
        dv_, ev = o.copy(), o.copy()
        ds, es = t0.copy(), zero.copy()
    for j in range(n_seq):
        at = slice(int(off[j]), int(off[j + 1]))
        for x in ((dq, dk_, eq, ek, aq, ak) if do is not None else ()):
            x[at] = 0.0
        for h in range(heads):
            hq = h // share
            a, b, c = q[at, hq], k[at, hq], v[at, h]
            if len(a) == 0:
                continue
            o[at, h], eo[at, h], out[j, h], eout[j, h] = _job(a, b, c, g[h], s0[j, h], 1, scale,
                                                              1.0, pieces)
            if do is None:
                continue
            d = do[at, h]
            x, e, _, _ = _job(d, c, b, g[h], s0[j, h].T, 1, scale, 1.0, pieces)
            dq[at, hq] += x
            eq[at, hq] += e
            aq[at, hq] += np.abs(x)
            x, e, _, _ = _job(c[::-1], d[::-1], a[::-1], g[h], t0[j, h].T, 0, 1.0, scale, pieces)
            dk_[at, hq] += x[::-1]
            ek[at, hq] += e[::-1]
            ak[at, hq] += np.abs(x[::-1])
            x, e, w, ew = _job(b[::-1], a[::-1], d[::-1], g[h], t0[j, h], 0, 1.0, scale, pieces)
            dv_[at, h], ev[at, h] = x[::-1], e[::-1]
            lam = _powers(g[h], np.array(1.0))
            ds[j, h] = lam * w
            es[j, h] = lam * (ew + 6 * U * np.abs(w))

    def flat(x):
        return x.reshape(rows, -1)

    val = dict(o=flat(o), state_out=out)
    tol = dict(o=rounded(flat(o), flat(eo), dtype), state_out=rounded(out, eout, "float32"))
    if do is not None:
        val.update(dq=flat(dq), dk=flat(dk_), dv=flat(dv_), dstate=ds)
        tol.update(dq=rounded(flat(dq), flat(eq + share * U * aq), dtype),
                   dk=rounded(flat(dk_), flat(ek + share * U * ak), dtype),
                   dv=rounded(flat(dv_), flat(ev), dtype), dstate=rounded(ds, es, "float32"))
    return val, tol


# Group norm: sums of fp32 values over at most 32 rows or lanes each, joined in
# 6 levels over the lanes and 10 over wavefronts and parts (where they are not
# fp64): 48 roundings, of |x| in a mean, of (x - mean)^2 in a variance.
DEPTH = 48.0


def group_norm(x, groups, weight=None, bias=None, gate=None, silu=False, off=None, eps=1e-5,
               dy=None, dtype="float32"):
    """Outputs and bounds of the group norm; with dy its gradients too. Rows
    behind the last sequence are left NaN."""
    f = np.float64
    rows, c = x.shape
    width = c // groups
    w = (np.ones(c) if weight is None else weight.astype(f)).reshape(groups, width)
    b = (np.zeros(c) if bias is None else bias.astype(f)).reshape(groups, width)
    x = x.astype(f).reshape(rows, groups, width)
    units = ([slice(i, i + 1) for i in range(rows)] if off is None else
             [slice(int(off[i]), int(off[i + 1])) for i in range(len(off) - 1)])
    last = rows if off is None else int(off[-1])

    def over(t):
        """Means over each unit's groups, for every value."""
        m = np.full(t.shape, np.nan)
        if off is None:
            m[:] = t.mean(2, keepdims=True)
        else:
            for u in units:
                if u.stop > u.start:
                    m[u] = t[u].mean((0, 2), keepdims=True)
        return m

    mean = over(x)
    em = DEPTH * U * over(np.abs(x - mean)) + 4 * U * np.abs(mean)
    xc = x - mean
    exc = em + U * np.abs(xc)
    var = over(xc * xc)
    root = 1.0 / np.sqrt(var + eps)
    # the mean square of centred values takes the mean's error to second order,
    # and their own
    ev = DEPTH * U * var + em * em + 2 * over(np.abs(xc) * U * np.abs(xc)) + U * var
    er = 0.5 * ev / (var + eps) + 4 * U
    xh = xc * root
    exh = root * exc + np.abs(xh) * er
    n = xh * w + b
    en = np.abs(w) * exh + 2 * U * (np.abs(xh * w) + np.abs(n))
    act, slope, ea, es = n, np.ones_like(n), en, np.zeros_like(n)
    if silu:
        s, u = sigmoid(n), sigmoid(-n)
        act, slope = n * s, s * (1.0 + n * u)
        k = (8.0 + 2.0 * np.abs(n)) * U
        ea = np.abs(slope) * en + 0.5 * en * en + k * np.abs(act)
        sa = s * (1.0 + np.abs(n) * u)
        # the slope of the slope is at most 1/2
        es = 0.5 * en + (k + 6 * U) * sa
    gated, gslope, eg, egs = 1.0, 0.0, 0.0, 0.0
    if gate is not None:
        g = gate.astype(f).reshape(rows, groups, width)
        s, u = sigmoid(g), sigmoid(-g)
        gated, gslope = g * s, s * (1.0 + g * u)
        k = (8.0 + 2.0 * np.abs(g)) * U
        eg, egs = k * np.abs(gated), (k + 6 * U) * s * (1.0 + np.abs(g) * u)
    y = act * gated
    ey = ea * np.abs(gated) + np.abs(act) * eg + 2 * U * np.abs(y)

    def flat(t):
        return t.reshape(rows, -1)

    val = dict(y=flat(y))
    tol = dict(y=rounded(flat(y), flat(ey), dtype))
    if dy is None:
        return val, tol
    dy = dy.astype(f).reshape(rows, groups, width)
    dn = dy * gated * slope
    edn = np.abs(dy) * (np.abs(gated) * es + eg * np.abs(slope)) + 3 * U * np.abs(dn)
    if gate is not None:
        dg = dy * act * gslope
        edg = np.abs(dy) * (ea * np.abs(gslope) + np.abs(act) * egs) + 3 * U * np.abs(dg)
        val["dgate"], tol["dgate"] = flat(dg), rounded(flat(dg), flat(edg), dtype)
    p = dn * xh
    ep = edn * np.abs(xh) + np.abs(dn) * exh + 2 * U * np.abs(p)
    if weight is not None:
        val["dweight"] = p[:last].sum(0).reshape(-1)
        tol["dweight"] = (ep[:last].sum(0)
                          + 33 * U * (np.abs(p) + ep)[:last].sum(0)).reshape(-1) + TINY["float32"]
    if bias is not None:
        val["dbias"] = dn[:last].sum(0).reshape(-1)
        tol["dbias"] = (edn[:last].sum(0)
                        + 33 * U * (np.abs(dn) + edn)[:last].sum(0)).reshape(-1) + TINY["float32"]
    q = dn * w
    eq = edn * np.abs(w) + U * np.abs(q)
    m1, m2 = over(q), over(q * xh)
    em1 = over(eq) + DEPTH * U * over(np.abs(q))
    em2 = over(eq * np.abs(xh) + np.abs(q) * exh) + DEPTH * U * over(np.abs(q * xh))
    dx = root * (q - m1 - xh * m2)
    span = np.abs(q) + np.abs(m1) + np.abs(xh * m2)
    edx = root * (eq + em1 + exh * np.abs(m2) + np.abs(xh) * em2 + span * (er + 5 * U))
    val["dx"], tol["dx"] = flat(dx), rounded(flat(dx), flat(edx), dtype)
    return val, tol
