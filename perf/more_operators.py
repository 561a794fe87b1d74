"""Measured cases of two more operators over packed rows: linear attention
with a decay for each head, and the group norm with an activation, each forward
and with its gradient.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges,
``prepare`` makes what a caller has in hand, ``run`` makes one pass (plain
torch operations in fp32, or the library's calls where ``own`` is set),
``exact`` the same outputs in fp64 and ``work`` the bytes and operations a
pass cannot do without.
"""

import math

import numpy as np
import torch

own = False

_DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
_EPS = 1e-5


# -------------------------------------------------------------------- cases

def listed():
    return [
        # One frame of one stream: a recogniser's step between pushes, latency only.
        dict(name="attn_1x1_f32", op="attn", train=False, dtype="float32", n_seq=1, rows=1,
             heads=8, qk_heads=8, dk=64, dv=64, lengths="equal", joint=False, state=True),
        # A push of 512 streams at the 80 ms clock: 8 frames each, states carried.
        dict(name="attn_512x8_bf16", op="attn", train=False, dtype="bfloat16", n_seq=512,
             rows=4096, heads=8, qk_heads=8, dk=64, dv=64, lengths="equal", joint=True,
             state=True),
        # The 64 x 30 s batch of frames through one layer, q, k and v slices of one product.
        dict(name="attn_64x2998_bf16", op="attn", train=False, dtype="bfloat16", n_seq=64,
             rows=64 * 2998, heads=8, qk_heads=8, dk=64, dv=64, lengths="equal", joint=True,
             state=False),
        # The longest recording (87 min) on its own: one sequence, one row per frame.
        dict(name="attn_521998_f32", op="attn", train=False, dtype="float32", n_seq=1,
             rows=521998, heads=2, qk_heads=2, dk=64, dv=64, lengths="equal", joint=False,
             state=True),
        # Training on the 64 x 30 s batch with wide heads: forward and gradients.
        dict(name="attn_64x2998_train_bf16", op="attn", train=True, dtype="bfloat16", n_seq=64,
             rows=64 * 2998, heads=4, qk_heads=4, dk=128, dv=128, lengths="equal", joint=True,
             state=False),
        # Training on ragged clips, odd head widths, q and k shared by three heads each.
        dict(name="attn_ragged_train_f16", op="attn", train=True, dtype="float16", n_seq=48,
             rows=70001, heads=6, qk_heads=2, dk=40, dv=71, lengths="ragged", joint=False,
             state=True),
        # One row behind the attention, head by head, with its gate: latency only.
        dict(name="gnorm_1_bf16", op="gnorm", over="row", train=False, dtype="bfloat16", n_seq=1,
             rows=1, groups=8, width=64, lengths="equal", affine=True, silu=False, gate=True,
             joint=False),
        # The same over the 64 x 30 s batch, in training.
        dict(name="gnorm_heads_train_bf16", op="gnorm", over="row", train=True,
             dtype="bfloat16", n_seq=64, rows=64 * 2998, groups=8, width=64, lengths="equal",
             affine=True, silu=False, gate=True, joint=True),
        # A first layer's norm over each 30-s clip, with its activation.
        dict(name="gnorm_clips_f16", op="gnorm", over="clip", train=False, dtype="float16",
             n_seq=64, rows=64 * 2998, groups=32, width=16, lengths="equal", affine=True,
             silu=True, gate=False, joint=False),
        # The same in training: forward and gradients.
        dict(name="gnorm_clips_train_bf16", op="gnorm", over="clip", train=True,
             dtype="bfloat16", n_seq=64, rows=64 * 2998, groups=32, width=16, lengths="equal",
             affine=True, silu=True, gate=False, joint=False),
        # Ragged clips with odd groups in training: nothing is aligned.
        dict(name="gnorm_ragged_train_f32", op="gnorm", over="clip", train=True,
             dtype="float32", n_seq=48, rows=70001, groups=3, width=107, lengths="ragged",
             affine=True, silu=True, gate=False, joint=False),
    ]


_MOST = 64 * 2998 * 512   # values of one operand in the largest listed cases


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rows(rng, case, most):
    rows = _log_uniform(rng, 1, min(521998, most))
    n_seq = _log_uniform(rng, 1, min(rows, 1024))
    lengths = rng.choice(["equal", "ragged"])
    case.update(n_seq=n_seq, rows=rows // n_seq * n_seq if lengths == "equal" else rows,
                lengths=lengths, joint=rng.random() < 0.4)


def draw(rng):
    op = rng.choice(["attn", "gnorm"])
    dtype = rng.choice(sorted(_DTYPES))
    case = dict(op=op, train=rng.random() < 0.5, dtype=dtype)
    most = _MOST // (2 if dtype == "float32" else 1)   # the largest cases hold 2-byte values
    if op == "attn":
        qk_heads = rng.choice([1, 2, 3, 4, 8])
        heads = qk_heads * rng.choice([1, 1, 1, 2, 3])
        dk, dv = _log_uniform(rng, 16, 128), _log_uniform(rng, 16, 128)
        if rng.random() < 0.6:
            dk, dv = (max(32, d // 32 * 32) for d in (dk, dv))
        case.update(heads=heads, qk_heads=qk_heads, dk=dk, dv=dv, state=rng.random() < 0.6)
        # as many values as the largest case, products and states too
        wide = heads * max(dk, dv) * (2 if max(dk, dv) > 64 and heads > qk_heads else 1)
        _draw_rows(rng, case, max(1, most // max(wide, 128)))
        case["n_seq"] = min(case["n_seq"], max(1, most // 2 // (heads * dk * dv)))
        if case["lengths"] == "equal":
            case["rows"] = case["rows"] // case["n_seq"] * case["n_seq"]
    else:
        groups, width = _log_uniform(rng, 1, 64), _log_uniform(rng, 8, 256)
        if rng.random() < 0.6:
            width = max(8, width // 8 * 8)
        if groups * width > 4096:
            groups = 4096 // width
        silu = rng.random() < 0.5
        case.update(over=rng.choice(["row", "clip"]), groups=groups, width=width,
                    affine=rng.random() < 0.8, silu=silu,
                    gate=rng.random() < (0.2 if silu else 0.6))
        _draw_rows(rng, case, max(1, most // (groups * width)))
    return case


def _lengths(case, seed):
    n, rows = case["n_seq"], case["rows"]
    if case["lengths"] == "equal":
        return np.full(n, rows // n, dtype=np.int64)
    # clips of log-uniform duration over a factor of about a thousand; short
    # totals leave some of them empty
    rng = np.random.default_rng(seed)
    w = np.exp(rng.uniform(0.0, math.log(1000.0), n))
    cut = np.floor(np.cumsum(w) / w.sum() * rows + 0.5).astype(np.int64)
    cut[-1] = rows
    return np.diff(np.concatenate([[0], cut]))


def work(case):
    rows, size = case["rows"], 4 if case["dtype"] == "float32" else 2
    if case["op"] == "attn":
        qk, v = rows * case["qk_heads"] * case["dk"], rows * case["heads"] * case["dv"]
        states = case["n_seq"] * case["heads"] * case["dk"] * case["dv"] * 4
        nbytes = (2 * qk + 2 * v) * size + states * (2 if case["state"] else 1)
        nbytes += 8 * (case["n_seq"] + 1) + 4 * case["heads"]
        flops = 4 * v * case["dk"]
        if case["train"]:   # do in, a gradient each of q, k and v out
            nbytes += (2 * qk + 2 * v) * size + states * (2 if case["state"] else 0)
            flops += 8 * v * case["dk"]
    else:
        c = case["groups"] * case["width"]
        n = rows * c
        operands = 3 if case["gate"] else 2
        if case["train"]:
            operands += 3 if case["gate"] else 2   # dy in, dx (and dgate) out
        nbytes = operands * n * size
        if case["affine"]:
            nbytes += 8 * c * (2 if case["train"] else 1)
        if case["over"] == "clip":
            nbytes += 8 * (case["n_seq"] + 1)
        flops = n * (8 + (5 if case["silu"] else 0) + (5 if case["gate"] else 0))
        if case["train"]:
            flops *= 3
    return {"bytes": float(nbytes), "flops": float(flops)}


# ------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda", 0)
    dt = _DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rows = case["rows"]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32) * scale

    def operands(widths, scales):
        # operands of one product: column slices of [rows, sum of widths], or apart
        if case["joint"]:
            p = torch.cat([normal(rows, w, scale=s) for w, s in zip(widths, scales)], 1).to(dt)
            return torch.split(p, widths, 1)
        return [normal(rows, w, scale=s).to(dt) for w, s in zip(widths, scales)]

    lens = _lengths(case, seed)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    st = dict(case=case, lens=lens, max_frames=int(lens.max()), off=torch.from_numpy(off).to(dev))
    if case["op"] == "attn":
        heads, dk, dv = case["heads"], case["dk"], case["dv"]
        qk, vw = case["qk_heads"] * dk, heads * dv
        st["q"], st["k"], st["v"] = operands([qk, qk, vw], [1.0, 1.0, 1.0])
        # memories of about two to two hundred rows over the heads
        st["log_decay"] = -torch.exp2(-8.0 * torch.arange(1, heads + 1, device=dev) / heads)
        st["scale"] = dk ** -0.5
        states = (len(lens), heads, dk, dv)
        st["state"] = normal(*states) if case["state"] else None
        st["state_out"] = torch.empty(states, dtype=torch.float32, device=dev)
        if case["train"]:
            st["do"] = normal(rows, vw).to(dt)
            st["dstate_out"] = normal(*states) if case["state"] else None
    else:
        c = case["groups"] * case["width"]
        parts = operands([c, c] if case["gate"] else [c], [1.0, 1.0])
        # levels and ranges that differ from channel to channel, as behind a product
        level, spread = normal(c), torch.exp(normal(c, scale=0.3))
        st["x"] = parts[0].mul_(spread.to(dt)).add_(level.to(dt))
        st["gate"] = parts[1] if case["gate"] else None
        st["w"] = 1.0 + normal(c, scale=0.1) if case["affine"] else None
        st["b"] = normal(c, scale=0.1) if case["affine"] else None
        if case["train"]:
            st["dy"] = normal(rows, c).to(dt)
    if own:
        import log_mel_spectrogram_amd as lm
        st["plan"] = lm.logmel_plan_create(dev.index)
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    if state["case"]["op"] == "attn":
        return _own_attn(state) if own else _plain_attn(state)
    return _own_gnorm(state) if own else _plain_gnorm(state)


def _own_attn(st):
    import log_mel_spectrogram_amd as lm
    case = st["case"]
    args = (st["q"], st["k"], st["v"], st["log_decay"], st["off"])
    more = dict(qk_heads=case["qk_heads"], scale=st["scale"], state=st["state"],
                max_frames=st["max_frames"])
    o = lm.logmel_linear_attention(st["plan"], *args, state_out=st["state_out"], **more)
    out = dict(o=o, state_out=st["state_out"])
    if case["train"]:
        dq, dk, dv, ds = lm.logmel_linear_attention_backward(
            st["plan"], st["do"], *args, dstate_out=st["dstate_out"], **more)
        out.update(dq=dq, dk=dk, dv=dv)
        if case["state"]:
            out["dstate"] = ds
    return out


def _own_gnorm(st):
    import log_mel_spectrogram_amd as lm
    case, x = st["case"], st["x"]
    more = dict(weight=st["w"], bias=st["b"], gate=st["gate"],
                activation="silu" if case["silu"] else None, eps=_EPS)
    stats = None
    if case["over"] == "clip":
        more.update(seq_offsets=st["off"], max_frames=st["max_frames"])
        if case["train"]:
            stats = torch.empty((case["n_seq"], case["groups"], 2), dtype=torch.float32,
                                device=x.device)
    y = lm.logmel_group_norm(st["plan"], x, case["groups"], stats=stats, **more)
    out = dict(y=y)
    if case["train"]:
        grads = lm.logmel_group_norm_backward(st["plan"], st["dy"], x, case["groups"],
                                              stats=stats, **more)
        out.update((k, v) for k, v in grads.items() if v is not None)
    return out


def _powers(g, n):
    """e^(g n) for each head, exponents in 64 bits: [heads, *n.shape], 0 where n < 0."""
    n = n.double()
    p = torch.exp(g.double().view(-1, *([1] * n.dim())) * n.clamp(min=0.0))
    return torch.where(n >= 0, p, 0.0).float()


def _chunks(lens, width, dev):
    """The sequences cut into chunks of at most `width` rows, none across two:
    each chunk's sequence, place within it, first row, rows, and rows of the
    sequence behind it."""
    per = -(-lens // width)
    seq = np.repeat(np.arange(len(lens)), per)
    at = np.arange(len(seq)) - np.repeat(np.cumsum(per) - per, per)
    first = (np.cumsum(lens) - lens)[seq] + at * width
    held = np.minimum(lens[seq] - at * width, width)
    after = lens[seq] - at * width - held
    return [torch.from_numpy(v).to(dev) for v in (seq, at, first, held, after)]


def _plain_attn(st):
    case, lens, g, scale = st["case"], st["lens"], st["log_decay"], st["scale"]
    heads, dk, dv = case["heads"], case["dk"], case["dv"]
    dt, dev, rows = st["q"].dtype, st["q"].device, case["rows"]
    width = min(128, st["max_frames"])
    i = torch.arange(width, device=dev)
    seq, at, first, held, after = _chunks(lens, width, dev)
    last = (after == 0).nonzero()[:, 0]
    fill = i < held[:, None]
    index = torch.where(fill, first[:, None] + i, 0)
    put = index[fill]

    def chunks(x, n, d):
        x = x.float().view(rows, n, d)[index] * fill[:, :, None, None]
        return x.permute(2, 0, 1, 3).repeat_interleave(heads // n, 0)   # [heads, chunks, width, d]

    def back(x, n):
        x = x.view(n, heads // n, *x.shape[1:]).sum(1).permute(1, 2, 0, 3)[fill]
        out = torch.empty((rows, x.shape[1] * x.shape[2]), dtype=dt, device=dev)
        out[put] = x.flatten(1).to(dt)
        return out

    q, k = chunks(st["q"], case["qk_heads"], dk), chunks(st["k"], case["qk_heads"], dk)
    v = chunks(st["v"], heads, dv)
    within = _powers(g, i[:, None] - i)[:, None]                        # decay from row j to row i
    enter = _powers(g, i + 1)[:, None, :, None]
    leave = _powers(g, held[:, None] - 1 - i)[..., None]
    same = seq[:, None] == seq
    hops = torch.where(same, (at[:, None] - at - 1) * width, -1)        # whole chunks between
    between = _powers(g, hops)
    begin = _powers(g, at * width)[..., None, None]
    init = st["state"] if st["state"] is not None else torch.zeros(
        (len(lens), heads, dk, dv), device=dev)
    own_part = (k * leave).transpose(2, 3) @ v                          # [heads, chunks, dk, dv]
    before = (between @ own_part.flatten(2)).view_as(own_part)
    before = before + begin * init[seq].transpose(0, 1)
    a = (q @ k.transpose(2, 3)) * within
    o = (a @ v + enter * (q @ before)) * scale
    state_out = init.clone()
    tail = _powers(g, held)[..., None, None][:, last] * before[:, last] + own_part[:, last]
    state_out[seq[last]] = tail.transpose(0, 1)
    out = dict(o=back(o, heads), state_out=state_out)
    if case["train"]:
        do = chunks(st["do"], heads, dv) * scale
        dbefore = (q * enter).transpose(2, 3) @ do
        dend = (between.transpose(1, 2) @ dbefore.flatten(2)).view_as(dbefore)
        if st["dstate_out"] is not None:
            behind = _powers(g, after)[..., None, None]
            dend = dend + behind * st["dstate_out"][seq].transpose(0, 1)
        da = (do @ v.transpose(2, 3)) * within
        out["dq"] = back(da @ k + enter * (do @ before.transpose(2, 3)), case["qk_heads"])
        out["dk"] = back(da.transpose(2, 3) @ q + leave * (v @ dend.transpose(2, 3)),
                         case["qk_heads"])
        out["dv"] = back(a.transpose(2, 3) @ do + leave * (k @ dend), heads)
        if case["state"]:
            ds = _powers(g, torch.from_numpy(lens).to(dev))[..., None, None].transpose(0, 1)
            ds = ds * st["dstate_out"]
            of = (torch.arange(len(lens), device=dev)[:, None] == seq).float()
            ds = ds + (of @ (begin * dbefore).flatten(2)).view(
                heads, -1, dk, dv).transpose(0, 1)
            out["dstate"] = ds
    return out


def _plain_gnorm(st):
    case, dt = st["case"], st["x"].dtype
    rows, groups, width = case["rows"], case["groups"], case["width"]
    x = st["x"].float().view(rows, groups, width)
    dev = x.device
    ones = torch.ones((groups, width), device=dev)
    w = st["w"].view(groups, width) if case["affine"] else ones
    b = st["b"].view(groups, width) if case["affine"] else torch.zeros_like(ones)
    clip = case["over"] == "clip"
    if clip:
        i = torch.arange(128, device=dev)
        seq, _, first, held, _ = _chunks(st["lens"], 128, dev)
        fill = i < held[:, None]
        index = torch.where(fill, first[:, None] + i, 0)
        n_rows = st["off"][1:] - st["off"][:-1]
        clips = torch.arange(len(n_rows), device=dev)
        member = (clips[:, None] == seq).double() / (n_rows.clamp(min=1) * width)[:, None]
        row_of = torch.repeat_interleave(clips, n_rows)

    def mean(t):
        # over a group's channels of a row, or of all rows of its clip; long sums in 64 bits
        if not clip:
            return t.mean(2, keepdim=True)
        s = (t.sum(2, dtype=torch.float64)[index] * fill[:, :, None]).sum(1)
        return (member @ s).float()[row_of][:, :, None]

    m = mean(x)
    r = torch.rsqrt(mean((x - m) ** 2) + _EPS)
    xh = (x - m) * r
    n = xh * w + b
    act, slope = n, torch.ones_like(n)
    if case["silu"]:
        s = 1.0 / (1.0 + torch.exp(-n))
        act, slope = n * s, s * (1.0 + n * (1.0 - s))
    y, gated = act, torch.ones_like(n)
    if case["gate"]:
        o = st["gate"].float().view(rows, groups, width)
        so = 1.0 / (1.0 + torch.exp(-o))
        gated = o * so
        y = act * gated
    out = dict(y=y.reshape(rows, -1).to(dt))
    if case["train"]:
        dy = st["dy"].float().view(rows, groups, width)
        dn = dy * gated * slope
        q = dn * w
        out["dx"] = (r * (q - mean(q) - xh * mean(q * xh))).reshape(rows, -1).to(dt)
        if case["gate"]:
            dg = dy * act * so * (1.0 + o * (1.0 - so))
            out["dgate"] = dg.reshape(rows, -1).to(dt)
        if case["affine"]:
            out["dweight"] = (dn * xh).sum(0, dtype=torch.float64).float().reshape(-1)
            out["dbias"] = dn.sum(0, dtype=torch.float64).float().reshape(-1)
    return out


# -------------------------------------------------------------------- exact

def exact(case, seed):
    st = prepare(case, seed)
    return _exact_attn(st) if case["op"] == "attn" else _exact_gnorm(st)


def _exact_attn(st):
    """Sequence after sequence in blocks of 512 rows, the state carried along
    and the state's gradient carried back, in fp64."""
    case, lens, scale = st["case"], st["lens"], st["scale"]
    heads, dk, dv, rows = case["heads"], case["dk"], case["dv"], case["rows"]
    dev = st["q"].device
    g = st["log_decay"].double()[:, None]

    def by_heads(x, d):
        x = x.double().view(rows, -1, d).transpose(0, 1)
        return x.repeat_interleave(heads // x.shape[0], 0)

    q, k, v = by_heads(st["q"], dk), by_heads(st["k"], dk), by_heads(st["v"], dv)
    o = torch.empty((heads, rows, dv), dtype=torch.float64, device=dev)
    out_state = torch.zeros((len(lens), heads, dk, dv), dtype=torch.float64, device=dev)
    train = case["train"]
    if train:
        do = by_heads(st["do"], dv)
        dq, dkk, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dstate = torch.zeros_like(out_state)
    steps = torch.arange(512, device=dev, dtype=torch.float64)
    gap = steps[:, None] - steps
    mask = torch.where(gap >= 0, torch.exp(g[:, :, None] * gap.clamp(min=0)), 0.0)
    begin = 0
    for j, length in enumerate(lens.tolist()):
        s = (st["state"][j].double() if st["state"] is not None else
             torch.zeros((heads, dk, dv), dtype=torch.float64, device=dev))
        kept = []
        for lo in range(begin, begin + length, 512):
            n = min(512, begin + length - lo)
            rng = slice(lo, lo + n)
            kept.append((rng, n, s))
            t = steps[:n]
            o[:, rng] = scale * (((q[:, rng] @ k[:, rng].transpose(1, 2)) * mask[:, :n, :n])
                                 @ v[:, rng] + torch.exp(g * (t + 1))[..., None] * (q[:, rng] @ s))
            s = torch.exp(g * n)[..., None] * s + (
                k[:, rng] * torch.exp(g * (n - 1 - t))[..., None]).transpose(1, 2) @ v[:, rng]
        out_state[j] = s
        begin += length
        if not train:
            continue
        ds = (st["dstate_out"][j].double() if st["dstate_out"] is not None else
              torch.zeros((heads, dk, dv), dtype=torch.float64, device=dev))
        for rng, n, s in reversed(kept):
            t = steps[:n]
            up, down = torch.exp(g * (t + 1))[..., None], torch.exp(g * (n - 1 - t))[..., None]
            a = (q[:, rng] @ k[:, rng].transpose(1, 2)) * mask[:, :n, :n]
            d = scale * (do[:, rng] @ v[:, rng].transpose(1, 2)) * mask[:, :n, :n]
            dq[:, rng] = d @ k[:, rng] + scale * up * (do[:, rng] @ s.transpose(1, 2))
            dkk[:, rng] = d.transpose(1, 2) @ q[:, rng] + down * (v[:, rng] @ ds.transpose(1, 2))
            dvv[:, rng] = scale * (a.transpose(1, 2) @ do[:, rng]) + down * (k[:, rng] @ ds)
            ds = torch.exp(g * n)[..., None] * ds + scale * (
                (q[:, rng] * up).transpose(1, 2) @ do[:, rng])
        dstate[j] = ds

    def flat(x, n):
        return x.view(n, heads // n, rows, -1).sum(1).transpose(0, 1).reshape(rows, -1)

    out = dict(o=flat(o, heads), state_out=out_state)
    if train:
        out.update(dq=flat(dq, case["qk_heads"]), dk=flat(dkk, case["qk_heads"]), dv=flat(dvv, heads))
        if case["state"]:
            out["dstate"] = dstate
    return out


def _exact_gnorm(st):
    case = st["case"]
    rows, groups, width = case["rows"], case["groups"], case["width"]
    names = dict(x="dx", gate="dgate", w="dweight", b="dbias")
    leaves = {key: st[key].double().requires_grad_(case["train"]) for key in names
              if st[key] is not None}
    x = leaves["x"].view(rows, groups, width)

    # the gradients are autograd's, in fp64, of the operator as it is defined
    def normed(t, dims):
        var, m = torch.var_mean(t, dims, correction=0, keepdim=True)
        return (t - m) * (var + _EPS).pow(-0.5)

    if case["over"] == "row":
        n = normed(x, (2,))
    else:
        n = torch.cat([normed(t, (0, 2)) for t in torch.split(x, st["lens"].tolist()) if len(t)])
    n = n.reshape(rows, -1)
    if case["affine"]:
        n = n * leaves["w"] + leaves["b"]
    if case["silu"]:
        n = n * torch.sigmoid(n)
    if case["gate"]:
        n = n * leaves["gate"] * torch.sigmoid(leaves["gate"])
    out = dict(y=n.detach())
    if case["train"]:
        n.backward(st["dy"].double())
        out.update((names[key], t.grad) for key, t in leaves.items())
    return out
