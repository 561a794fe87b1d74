"""Measured cases of the row operators: the gated scan over packed sequences
and the block norm, each forward and with its gradient.

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
_EPS = 1e-6


# -------------------------------------------------------------------- cases

def listed():
    return [
        # One frame of one stream: a recogniser's step between pushes, latency only.
        dict(name="scan_1x1_f32", op="scan", train=False, dtype="float32", n_seq=1, rows=1,
             channels=512, lengths="equal", joint=False, bias=True, state=True),
        # A push of 512 streams at the 80 ms clock: 8 frames each, state carried.
        dict(name="scan_512x8_bf16", op="scan", train=False, dtype="bfloat16", n_seq=512,
             rows=4096, channels=512, lengths="equal", joint=True, bias=True, state=True),
        # The 64 x 30 s batch of frames through one layer, value and gate slices of one product.
        dict(name="scan_64x2998_bf16", op="scan", train=False, dtype="bfloat16", n_seq=64,
             rows=64 * 2998, channels=512, lengths="equal", joint=True, bias=True, state=False),
        # The longest recording (87 min) on its own: one sequence, one row per frame.
        dict(name="scan_521998_f32", op="scan", train=False, dtype="float32", n_seq=1,
             rows=521998, channels=128, lengths="equal", joint=False, bias=True, state=True),
        # Training on the 64 x 30 s batch: forward and gradients.
        dict(name="scan_64x2998_train_bf16", op="scan", train=True, dtype="bfloat16", n_seq=64,
             rows=64 * 2998, channels=512, lengths="equal", joint=True, bias=True, state=False),
        # Training on ragged clips with an odd width: nothing is aligned.
        dict(name="scan_ragged_train_f16", op="scan", train=True, dtype="float16", n_seq=48,
             rows=70001, channels=257, lengths="ragged", joint=False, bias=True, state=True),
        # One row's norm, gate and residual: latency only.
        dict(name="norm_1_bf16", op="norm", train=False, dtype="bfloat16", rows=1, channels=512,
             block=True, gate=True, scale=True, pre=True, joint=False),
        # Log-mel rows of a push of 512 streams, normalised before the first product.
        dict(name="norm_4096x128_f16", op="norm", train=False, dtype="float16", rows=4096,
             channels=128, block=False, gate=False, scale=False, pre=True, joint=False),
        # End of a block on the 64 x 30 s batch, with the next block's norm.
        dict(name="norm_64x2998_bf16", op="norm", train=False, dtype="bfloat16", rows=64 * 2998,
             channels=512, block=True, gate=True, scale=True, pre=True, joint=True),
        # The same in training: forward and gradients.
        dict(name="norm_64x2998_train_bf16", op="norm", train=True, dtype="bfloat16",
             rows=64 * 2998, channels=512, block=True, gate=True, scale=True, pre=True,
             joint=True),
        # Wide fp32 rows of one 30-s clip in training.
        dict(name="norm_2998x4096_train_f32", op="norm", train=True, dtype="float32", rows=2998,
             channels=4096, block=True, gate=True, scale=True, pre=True, joint=False),
        # An odd width and row count in training.
        dict(name="norm_odd_train_f16", op="norm", train=True, dtype="float16", rows=30011,
             channels=321, block=True, gate=True, scale=False, pre=True, joint=False),
    ]


_MOST = 64 * 2998 * 512   # elements of one operand in the largest listed cases


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "norm"])
    train = rng.random() < 0.5
    dtype = rng.choice(sorted(_DTYPES))
    most = _MOST // (2 if dtype == "float32" else 1)   # the largest cases hold 2-byte values
    channels = _log_uniform(rng, 64, 4096)
    if rng.random() < 0.6:
        channels = max(64, channels // 64 * 64)
    rows = _log_uniform(rng, 1, min(600000, most // channels))
    case = dict(op=op, train=train, dtype=dtype, rows=rows, channels=channels,
                joint=rng.random() < 0.4)
    if op == "scan":
        n_seq = _log_uniform(rng, 1, min(rows, 1024))
        lengths = rng.choice(["equal", "ragged"])
        if lengths == "equal":
            case["rows"] = rows // n_seq * n_seq
        case.update(n_seq=n_seq, lengths=lengths, bias=rng.random() < 0.8,
                    state=rng.random() < 0.6)
    else:
        block = rng.random() < 0.75
        case.update(block=block, gate=block and rng.random() < 0.8,
                    scale=block and rng.random() < 0.7, pre=(not block) or rng.random() < 0.8)
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
    rows, c = case["rows"], case["channels"]
    size = 4 if case["dtype"] == "float32" else 2
    n = rows * c
    if case["op"] == "scan":
        side = case["n_seq"] * c * 4
        states = side * (2 if case["state"] else 1)
        nbytes = 3 * n * size + states + 8 * (case["n_seq"] + 1) + (4 * c if case["bias"] else 0)
        flops = 8 * n
        if case["train"]:
            nbytes += 3 * n * size + side * (2 if case["state"] else 1)
            nbytes += 4 * c if case["bias"] else 0
            flops += 16 * n
    else:
        reads, writes = 1, 0
        params = 0
        if case["block"]:
            reads, writes = 2, 1
            params += 1
            flops = 6 * n
        else:
            flops = 0
        if case["gate"]:
            reads += 1
            flops += 5 * n
        if case["scale"]:
            params += 1
        if case["pre"]:
            writes += 1
            params += 1
            flops += 4 * n
        if case["train"]:
            reads, writes = reads + writes, writes + reads   # a gradient per operand
            params *= 2
            flops *= 3
        nbytes = (reads + writes) * n * size + params * 4 * c
    return {"bytes": float(nbytes), "flops": float(flops)}


# ------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda", 0)
    dt = _DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rows, c = case["rows"], case["channels"]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32) * scale

    def slices(k):
        # k operands of one product: column slices of [rows, k c], or apart
        if case["joint"]:
            p = normal(rows, k * c).to(dt)
            return [p[:, i * c:(i + 1) * c] for i in range(k)]
        return [normal(rows, c).to(dt) for _ in range(k)]

    st = dict(case=case)
    if case["op"] == "scan":
        lens = _lengths(case, seed)
        off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        st["lens"] = lens
        st["max_frames"] = int(lens.max())
        st["off"] = torch.from_numpy(off).to(dev)
        st["x"], st["g"] = slices(2)
        # memories of about one to a hundred rows over the channels
        st["bias"] = (torch.rand(c, generator=gen, device=dev) * 5.0 - 0.5
                      if case["bias"] else None)
        st["state"] = normal(len(lens), c) if case["state"] else None
        st["state_out"] = torch.empty((len(lens), c), dtype=torch.float32, device=dev)
        if case["train"]:
            st["dh"] = normal(rows, c).to(dt)
            st["dstate_out"] = normal(len(lens), c) if case["state"] else None
    else:
        if case["block"]:
            parts = slices(2 if case["gate"] else 1)
            st["h"] = parts[0]
            st["o"] = parts[1] if case["gate"] else None
            st["w_post"] = 1.0 + normal(c, scale=0.1)
            st["res"] = normal(rows, c, scale=2.0).to(dt)
        else:
            st["h"] = st["o"] = st["w_post"] = None
            # log-mel rows: a level per row, a slope over the bands, the floor below
            level = normal(rows, 1, scale=3.0) - 6.0
            band = torch.linspace(2.0, -4.0, c, device=dev)
            st["res"] = torch.clamp(level + band + normal(rows, c, scale=1.5),
                                    min=math.log(1e-10)).to(dt)
        st["scale"] = (normal(c, scale=0.1) + 0.3) if case["scale"] else None
        st["w_pre"] = (1.0 + normal(c, scale=0.1)) if case["pre"] else None
        if case["train"]:
            st["dy"] = normal(rows, c).to(dt) if case["block"] else None
            st["dz"] = normal(rows, c).to(dt) if case["pre"] else None
    if own:
        import log_mel_spectrogram_amd as lm
        st["plan"] = lm.logmel_plan_create(dev.index)
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    if state["case"]["op"] == "scan":
        return _own_scan(state) if own else _plain_scan(state)
    return _own_norm(state) if own else _plain_norm(state)


def _own_scan(st):
    import log_mel_spectrogram_amd as lm
    case, x = st["case"], st["x"]
    ck = None
    if case["train"]:
        ck = torch.empty((lm.logmel_gated_scan_checkpoint_rows(case["rows"]), case["channels"]),
                         dtype=torch.float32, device=x.device)
    h = lm.logmel_gated_scan(st["plan"], x, st["g"], st["off"], bias=st["bias"],
                             state=st["state"], state_out=st["state_out"], checkpoints=ck,
                             max_frames=st["max_frames"])
    out = dict(h=h, state_out=st["state_out"])
    if case["train"]:
        dx, dg, db, ds = lm.logmel_gated_scan_backward(
            st["plan"], st["dh"], x, st["g"], st["off"], ck, bias=st["bias"], state=st["state"],
            dstate_out=st["dstate_out"], max_frames=st["max_frames"])
        out.update(dx=dx, dg=dg)
        if case["bias"]:
            out["db"] = db
        if case["state"]:
            out["dstate"] = ds
    return out


def _own_norm(st):
    import log_mel_spectrogram_amd as lm
    case = st["case"]
    parts = dict(h=st["h"], gate=st["o"], w_post=st["w_post"], scale=st["scale"],
                 w_pre=st["w_pre"], eps=_EPS)
    y, z = lm.logmel_block_norm(st["plan"], st["res"], want_y=case["block"], want_z=case["pre"],
                                **parts)
    out = {}
    if case["block"]:
        out["y"] = y
    if case["pre"]:
        out["z"] = z
    if case["train"]:
        grads = lm.logmel_block_norm_backward(st["plan"], st["res"], dy=st["dy"], dz=st["dz"],
                                              **parts)
        out.update((k, v) for k, v in grads.items() if v is not None)
    return out


def _starts(lens, rows, dev):
    """Rows that begin and rows that end a sequence, and those sequences."""
    full = np.flatnonzero(lens)
    ends = np.cumsum(lens)[full]
    first = torch.from_numpy((ends - lens[full]).astype(np.int64)).to(dev)
    last = torch.from_numpy((ends - 1).astype(np.int64)).to(dev)
    return torch.from_numpy(full.astype(np.int64)).to(dev), first, last


def _doubling(a, b, reach):
    """h_t = a_t h_{t-1} + b_t by doubling: a is 0 where a sequence begins."""
    d = 1
    while d < reach:
        b = torch.cat([b[:d], b[d:] + a[d:] * b[:-d]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _plain_scan(st):
    case, x, lens = st["case"], st["x"].float(), st["lens"]
    dt, dev = st["x"].dtype, x.device
    g = st["g"].float()
    if st["bias"] is not None:
        g = g + st["bias"]
    a, u = 1.0 / (1.0 + torch.exp(-g)), 1.0 / (1.0 + torch.exp(g))
    seq, first, last = _starts(lens, case["rows"], dev)
    h0 = st["state"] if st["state"] is not None else torch.zeros(
        (len(lens), case["channels"]), device=dev)
    reach = st["max_frames"]
    b = u * x
    b[first] = b[first] + a[first] * h0[seq]
    carry = a.clone()
    carry[first] = 0.0
    h = _doubling(carry, b, reach)
    state_out = h0.clone()
    state_out[seq] = h[last]
    out = dict(h=h.to(dt), state_out=state_out)
    if case["train"]:
        prev = torch.roll(h, 1, 0)
        prev[first] = h0[seq]
        d = st["dh"].float()
        if st["dstate_out"] is not None:
            d[last] = d[last] + st["dstate_out"][seq]
        back = torch.roll(a, -1, 0)
        back[last] = 0.0
        grad = _doubling(back.flip(0), d.flip(0), reach).flip(0)
        dg = a * u * (prev - x) * grad
        out.update(dx=(u * grad).to(dt), dg=dg.to(dt))
        if case["bias"]:
            out["db"] = dg.sum(0, dtype=torch.float64).float()
        if case["state"]:
            ds = st["dstate_out"].clone()
            ds[seq] = a[first] * grad[first]
            out["dstate"] = ds
    return out


def _plain_norm(st):
    case, dt = st["case"], st["res"].dtype
    res = st["res"].float()
    c = case["channels"]
    if case["block"]:
        h = st["h"].float()
        r1 = torch.rsqrt((h * h).sum(1, keepdim=True) / c + _EPS)
        n = h * r1 * st["w_post"]
        if case["gate"]:
            o = st["o"].float()
            sg = 1.0 / (1.0 + torch.exp(-o))
            act = o * sg
        else:
            act = torch.ones_like(h)
        s = st["scale"] if case["scale"] else torch.ones(c, device=res.device)
        t = n * act
        y = res + s * t
    else:
        y = res
    out = {}
    if case["block"]:
        out["y"] = y.to(dt)
    if case["pre"]:
        r2 = torch.rsqrt((y * y).sum(1, keepdim=True) / c + _EPS)
        out["z"] = (y * r2 * st["w_pre"]).to(dt)
    if case["train"]:
        if case["pre"]:
            dz = st["dz"].float()
            q = dz * st["w_pre"]
            grad = r2 * q - y * (r2 * r2 * r2) * ((q * y).sum(1, keepdim=True) / c)
            dw_pre = (dz * y * r2).sum(0, dtype=torch.float64).float()
        else:
            grad, dw_pre = torch.zeros_like(y), None
        if st["dy"] is not None:
            grad = grad + st["dy"].float()
        out["dres"] = grad.to(dt)
        if case["block"]:
            gs = grad * s
            q = gs * act
            if case["gate"]:
                out["dgate"] = (gs * n * sg * (1.0 + o * (1.0 - sg))).to(dt)
            if case["scale"]:
                out["dscale"] = (grad * t).sum(0, dtype=torch.float64).float()
            out["dw_post"] = (q * h * r1).sum(0, dtype=torch.float64).float()
            q = q * st["w_post"]
            out["dh"] = (r1 * q - h * (r1 * r1 * r1) * ((q * h).sum(1, keepdim=True) / c)).to(dt)
        if case["pre"]:
            out["dw_pre"] = dw_pre
    return _ordered(out)


_ORDER = ["y", "z", "dres", "dh", "dgate", "dw_post", "dscale", "dw_pre"]


def _ordered(out):
    return {k: out[k] for k in _ORDER if k in out}


# -------------------------------------------------------------------- exact

def _exact_recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t over the rows, from 0, in fp64: blocks of rows
    side by side, then their ends in turn, then each block from its start."""
    rows, c = a.shape
    width = max(1, int(math.isqrt(rows)))
    blocks = -(-rows // width)
    pad = blocks * width - rows
    a = torch.nn.functional.pad(a, (0, 0, 0, pad)).view(blocks, width, c)
    b = torch.nn.functional.pad(b, (0, 0, 0, pad)).view(blocks, width, c)
    prod = torch.ones((blocks, c), dtype=a.dtype, device=a.device)
    end = torch.zeros_like(prod)
    for t in range(width):
        end = a[:, t] * end + b[:, t]
        prod = prod * a[:, t]
    enter = torch.zeros_like(prod)
    for k in range(1, blocks):
        enter[k] = prod[k - 1] * enter[k - 1] + end[k - 1]
    h = torch.empty_like(b)
    for t in range(width):
        enter = a[:, t] * enter + b[:, t]
        h[:, t] = enter
    return h.reshape(blocks * width, c)[:rows]


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_scan(st) if case["op"] == "scan" else _exact_norm(st)


def _exact_scan(st):
    case = st["case"]
    lens, rows, c = st["lens"], case["rows"], case["channels"]
    x, g = st["x"].double(), st["g"].double()
    dev = x.device
    if st["bias"] is not None:
        g = g + st["bias"].double()
    forget, take = torch.sigmoid(g), torch.sigmoid(-g)
    start = st["state"].double() if st["state"] is not None else torch.zeros(
        (len(lens), c), dtype=torch.float64, device=dev)
    # one more row in front of each sequence holds its first state
    where = torch.from_numpy(np.repeat(np.arange(1, len(lens) + 1), lens)).to(dev)
    at = torch.arange(rows, device=dev) + where
    heads = torch.from_numpy(np.concatenate([[0], np.cumsum(lens + 1)[:-1]]).astype(np.int64))
    heads = heads.to(dev)
    total = rows + len(lens)
    big_a = torch.zeros((total, c), dtype=torch.float64, device=dev)
    big_b = torch.zeros_like(big_a)
    big_a[at], big_b[at] = forget, take * x
    big_b[heads] = start
    big_h = _exact_recurrence(big_a, big_b)
    h, before = big_h[at], big_h[at - 1]
    tails = heads + torch.from_numpy(lens).to(dev)
    out = dict(h=h, state_out=big_h[tails])
    if case["train"]:
        big_d = torch.zeros((total, c), dtype=torch.float64, device=dev)
        big_d[at] = st["dh"].double()
        if st["dstate_out"] is not None:
            big_d[tails] += st["dstate_out"].double()
        # row t takes a_{t+1} D_{t+1}; the row after a sequence is a head, with a = 0
        after = torch.cat([big_a[1:], torch.zeros((1, c), dtype=torch.float64, device=dev)])
        big_d = _exact_recurrence(after.flip(0), big_d.flip(0)).flip(0)
        grad = big_d[at]
        dg = grad * (before - x) * forget * take
        out.update(dx=grad * take, dg=dg)
        if case["bias"]:
            out["db"] = dg.sum(0)
        if case["state"]:
            out["dstate"] = big_d[heads]
    return out


def _exact_norm(st):
    case = st["case"]
    c = case["channels"]
    leaves = {}

    def leaf(key):
        v = st[key]
        return None if v is None else leaves.setdefault(key, v.double().requires_grad_(True))

    # the gradients are autograd's, in fp64, of the operator as it is defined
    y = leaf("res")
    if case["block"]:
        h = leaf("h")
        t = h * (h.square().mean(1, keepdim=True) + _EPS).pow(-0.5) * leaf("w_post")
        if case["gate"]:
            t = t * leaf("o") * torch.sigmoid(leaf("o"))
        if case["scale"]:
            t = t * leaf("scale")
        y = y + t
    out, tops, grads = {}, [], []
    if case["block"]:
        out["y"] = y
    if case["pre"]:
        out["z"] = y * (y.square().mean(1, keepdim=True) + _EPS).pow(-0.5) * leaf("w_pre")
    if case["train"]:
        if st["dy"] is not None:
            tops.append(y)
            grads.append(st["dy"].double())
        if st["dz"] is not None:
            tops.append(out["z"])
            grads.append(st["dz"].double())
        torch.autograd.backward(tops, grads)
        names = dict(res="dres", h="dh", o="dgate", w_post="dw_post", scale="dscale",
                     w_pre="dw_pre")
        out.update((names[k], v.grad) for k, v in leaves.items())
    return _ordered({k: v.detach() for k, v in out.items()})
