"""Linear attention on the GPU, with its gradient, against the fp64 form of
attn_ref.py, whose bounds follow from the number of roundings."""

import numpy as np
import pytest

from tests import attn_ref
from tests.test_gpu_rows import DTYPES, Rows, check, env, host, say  # noqa: F401

pytestmark = pytest.mark.gpu


def untouched(torch, t):
    """Values around a row operand's own, as Rows made them."""
    base = t._base if t._base is not None else t
    whole = base.flatten().clone()
    at = torch.as_strided(torch.arange(whole.numel(), device=t.device), t.shape, t.stride(),
                          t.storage_offset())
    whole[at.reshape(-1)] = 7.0
    return bool((whole == 7.0).all())


def decays(heads, kind):
    if kind == "steps":      # memories of two to two hundred rows
        return -np.exp2(-8.0 * np.arange(1, heads + 1) / heads)
    return np.array([0.0, -np.inf, -3.0, -1e-4, -40.0, -1e30] * heads)[:heads]   # extremes


def attn_case(env, dtype, lens, heads=2, qk=2, dk=64, dv=64, layout="dense", state=True, behind=0,
              max_frames=0, seed=0, kind="steps", scale=None, train=True, in_place=False):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    rows, n, last = int(off[-1]) + behind, len(lens), int(off[-1])
    mq = Rows(torch, dtype, rows, qk * dk, layout, seed)
    mv = Rows(torch, dtype, rows, heads * dv, layout, seed + 1000)
    q, k, v, do = mq.normal(), mq.normal(), mv.normal(), mv.normal()
    rng = mq.rng
    scale = dk ** -0.5 if scale is None else scale

    def f32(*shape):
        return torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(dev)

    g = torch.from_numpy(decays(heads, kind).astype(np.float32)).to(dev)
    s0 = f32(n, heads, dk, dv) if state else None
    dso = f32(n, heads, dk, dv) if state else None
    off_d = torch.from_numpy(off).to(dev)
    o, dq, dkk, dvv = mv.empty(), mq.empty(), mq.empty(), mv.empty()
    so = s0.clone() if in_place else torch.full((n, heads, dk, dv), 7.0, device=dev)
    more = dict(qk_heads=qk, scale=scale, max_frames=max_frames)
    lm.logmel_linear_attention(plan, q, k, v, g, off_d, state=so if in_place else s0, out=o,
                               state_out=so, **more)
    got = dict(o=o, state_out=so)
    if train:
        _, _, _, ds = lm.logmel_linear_attention_backward(
            plan, do, q, k, v, g, off_d, state=s0, dstate_out=dso, dq=dq, dk=dkk, dv=dvv, **more)
        got.update(dq=dq, dk=dkk, dv=dvv)
        if state:
            got["dstate"] = ds
    torch.cuda.synchronize()
    val, tol = attn_ref.attention(
        host(q), host(k), host(v), host(g), off, qk, scale, None if s0 is None else host(s0),
        host(do) if train else None, None if dso is None else host(dso), dtype=dtype)
    for name, t in got.items():
        if name in ("o", "dq", "dk", "dv"):
            check(t[:last], val[name][:last], tol[name][:last], name)
            assert (t[last:] == 7.0).all(), name
            if layout != "dense":
                assert untouched(torch, t), name
        else:
            check(t, val[name], tol[name], name)


SEQS = {
    "one": [1],
    "empty_around": [0, 1, 0, 0, 5, 0],
    "ones": [1] * 70,
    "edges": [31, 1, 32, 33, 0, 64, 63, 65, 127, 128, 129, 3],
    "ragged": [300, 2, 0, 233, 41],
    "long": [1500],
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seqs", sorted(SEQS))
def test_attention_lengths(env, dtype, seqs):
    lens = SEQS[seqs]
    for max_frames in (0, max(lens)):
        say(f"attention {dtype} {seqs} max_frames {max_frames}")
        attn_case(env, dtype, lens, behind=5, max_frames=max_frames)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["dense", "slice", "odd"])
@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 130 - 2), (128, 2), (40, 71), (64, 32), (33, 65),
                                   (128, 128), (16, 48)])
def test_attention_widths(env, dtype, layout, dk, dv):
    for max_frames in (0, 11):
        say(f"attention {dtype} {layout} {dk} x {dv} max_frames {max_frames}")
        lens = [150, 0, 77] if max_frames == 0 else [11, 0, 9, 1]
        attn_case(env, dtype, lens, dk=dk, dv=dv, layout=layout, behind=2, seed=dk,
                  state=layout != "slice", max_frames=max_frames)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,qk", [(1, 1), (3, 1), (6, 2), (5, 5), (8, 4)])
def test_attention_heads(env, dtype, heads, qk):
    say(f"attention {dtype} {heads} heads, {qk} of q and k")
    attn_case(env, dtype, [90, 3, 0, 70], heads=heads, qk=qk, dk=24, dv=40, behind=3, seed=heads)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[1, 0, 7], [200, 5, 0, 130]])
def test_attention_extreme_decays(env, dtype, lens):
    """Nothing kept, everything kept, and decays whose powers underflow."""
    say(f"attention extremes {dtype} {lens}")
    attn_case(env, dtype, lens, heads=6, qk=6, dk=32, dv=32, kind="extremes", seed=3)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[1, 0, 8, 3], [700, 0, 40]])
def test_attention_state_in_place(env, dtype, lens):
    for max_frames in (0, max(lens)):
        say(f"attention in place {dtype} {lens} {max_frames}")
        attn_case(env, dtype, lens, train=False, in_place=True, max_frames=max_frames, seed=4)


@pytest.mark.parametrize("scale", [0.0, -2.5])
def test_attention_scales(env, scale):
    say(f"attention scale {scale}")
    attn_case(env, "float32", [70, 3], scale=scale, seed=5)


@pytest.mark.parametrize("max_frames", [1, 20, 1 << 40])
def test_attention_wrong_hint_changes_no_result(env, max_frames):
    say(f"attention hint {max_frames}")
    for n in (1, 30):
        attn_case(env, "bfloat16", [170, 3, 0, 65] * n, dk=32, dv=32, max_frames=max_frames,
                  seed=6)


def test_attention_no_sequences_and_no_rows(env):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say("attention of nothing")
    q = torch.full((4, 16), 3.0, device=dev)
    g = torch.zeros(2, device=dev)
    o = torch.full((4, 16), 7.0, device=dev)
    lm.logmel_linear_attention(plan, q, q, q, g, torch.zeros(1, dtype=torch.int64, device=dev),
                               out=o)
    assert (o == 7.0).all()
    e = q[:0]
    s = torch.randn((3, 2, 8, 8), device=dev)
    so, ds = torch.empty_like(s), None
    off = torch.zeros(4, dtype=torch.int64, device=dev)
    lm.logmel_linear_attention(plan, e, e, e, g, off, state=s, state_out=so)
    _, _, _, ds = lm.logmel_linear_attention_backward(plan, e, e, e, e, g, off, state=s,
                                                      dstate_out=s)
    assert torch.equal(so, s) and torch.equal(ds, s)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("max_frames", [0, 100])
def test_attention_not_finite_stays_behind(env, dtype, max_frames):
    """A NaN or infinity in q reaches its row and head; one in k or v its
    sequence and head from its row on: earlier rows keep every bit."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say(f"attention not finite {dtype} {max_frames}")
    dt = getattr(torch, dtype)
    rows, heads, d = 300, 3, 32
    gen = torch.Generator(device=dev).manual_seed(7)
    q, k, v = (torch.randn((rows, heads * d), generator=gen, device=dev).to(dt) for _ in range(3))
    off = torch.tensor([0, 100, 200, 300], device=dev)
    g = torch.tensor([-0.1, -0.01, -1.0], device=dev)

    def call():
        return lm.logmel_linear_attention(plan, q, k, v, g, off, max_frames=max_frames)

    o = call().clone()
    for bad in (float("nan"), float("inf"), -float("inf")):
        for x, row, head, whole in ((q, 130, 1, False), (k, 137, 0, True), (v, 190, 2, True),
                                    (v, 100, 1, True), (k, 163, 1, True)):
            keep = x[row, head * d + 5].clone()
            x[row, head * d + 5] = bad
            b = call()
            x[row, head * d + 5] = keep
            same = torch.ones_like(o, dtype=torch.bool)
            same[row:200 if whole else row + 1, head * d:(head + 1) * d] = False
            assert torch.equal(b[same], o[same]), (bad, row, head)
            at = b[row, head * d:(head + 1) * d]
            assert not torch.isfinite(at).all(), (bad, row, head)
            if whole:
                assert not torch.isfinite(b[199, head * d:(head + 1) * d]).all()
    assert torch.equal(call(), o)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_attention_pushes_equal_the_whole(env, dtype):
    """Streams fed row by row, then in pushes, with the state carried in place:
    the rows of the whole sequences, within the bounds of both."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say(f"attention pushes {dtype}")
    n, total, heads, dk, dv = 5, 50, 2, 24, 40
    rng = np.random.default_rng(8)
    dt = getattr(torch, dtype)
    q, k = (torch.from_numpy(rng.normal(size=(n, total, heads * dk))).to(dt) for _ in range(2))
    v = torch.from_numpy(rng.normal(size=(n, total, heads * dv))).to(dt)
    g = -np.array([0.3, 0.02])
    gd = torch.from_numpy(g.astype(np.float32)).to(dev)
    state = torch.zeros((n, heads, dk, dv), device=dev)
    got = []
    at = 0
    for push in [1, 1, 1, 8, 8, 1, 30]:
        rows = [x[:, at:at + push].reshape(n * push, -1).to(dev) for x in (q, k, v)]
        off = torch.arange(n + 1, device=dev) * push
        o = lm.logmel_linear_attention(plan, *rows, gd, off, state=state, state_out=state,
                                       max_frames=push)
        got.append(o.view(n, push, -1))
        at += push
    flat = [x.reshape(n * total, -1) for x in (q, k, v)]
    val, tol = attn_ref.attention(*(host(x) for x in flat), g.astype(np.float32),
                                  np.arange(n + 1) * total, heads, 1.0, dtype=dtype)
    check(torch.cat(got, 1).reshape(n * total, -1), val["o"], tol["o"], "o")
    check(state, val["state_out"], tol["state_out"], "state")


@pytest.mark.parametrize("dtype", ["float32", "float16"])
@pytest.mark.parametrize("lens,max_frames", [([3, 8, 1], 8), ([200, 70, 0, 130], 0)])
def test_attention_same_bits_other_stream_and_graph(env, dtype, lens, max_frames):
    """The same call gives the same bits, on another stream and replayed from
    a graph with the program's own work between the replays."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say(f"attention graph {dtype} {lens}")
    dt = getattr(torch, dtype)
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device=dev)
    rows, heads, dk, dv = int(sum(lens)), 4, 40, 72
    gen = torch.Generator(device=dev).manual_seed(9)
    q, k = (torch.randn((rows, 2 * dk), generator=gen, device=dev).to(dt) for _ in range(2))
    v, do = (torch.randn((rows, heads * dv), generator=gen, device=dev).to(dt) for _ in range(2))
    g = -torch.rand(heads, generator=gen, device=dev)
    s0 = torch.randn((len(lens), heads, dk, dv), generator=gen, device=dev)

    def call(stream=None):
        so = torch.empty_like(s0)
        more = dict(qk_heads=2, state=s0, max_frames=max_frames, stream=stream)
        o = lm.logmel_linear_attention(plan, q, k, v, g, off, state_out=so, **more)
        return [o, so, *lm.logmel_linear_attention_backward(plan, do, q, k, v, g, off,
                                                            dstate_out=s0, **more)]

    first = [t.clone() for t in call()]
    assert all(torch.equal(a, b) for a, b in zip(first, call()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    with torch.cuda.graph(graph2):
        held2 = call()
    for _ in range(3):
        for t in held + held2:
            t.fill_(3.0)
        graph.replay()
        graph2.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, held))
        assert all(torch.equal(a, b) for a, b in zip(first, held2))
        assert all(torch.equal(a, b) for a, b in zip(first, call()))
    v.mul_(2.0)
    graph.replay()
    again = call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, again))


def test_attention_many_sequences(env):
    """Tens of thousands of short sequences, with and without the hint."""
    lens = np.random.default_rng(10).integers(0, 4, size=20000).tolist()
    for max_frames in (0, 3):
        say(f"attention 20,000 sequences max_frames {max_frames}")
        attn_case(env, "bfloat16", lens, heads=1, qk=1, dk=8, dv=8, max_frames=max_frames,
                  behind=1, seed=11)


def test_attention_offsets_past_32_bits(env):
    """Rows whose elements lie past 2^31, against the last rows by themselves."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say("attention past 2^31 elements")
    rows, wide, d = 70_000, 32_768, 32
    big = torch.zeros((rows, wide), dtype=torch.bfloat16, device=dev)
    gen = torch.Generator(device=dev).manual_seed(12)
    q, k, v = big[:, :d], big[:, wide - d:], big[:, 64:64 + d]
    small = [torch.randn((300, d), generator=gen, device=dev).to(torch.bfloat16) for _ in range(4)]
    for x, s in zip((q, k, v), small):
        x[-300:] = s
    out = big[:, 1024:1024 + d]
    g = torch.tensor([-0.05], device=dev)
    off, off_s = (torch.tensor([0, n], device=dev) for n in (rows, 300))
    lm.logmel_linear_attention(plan, q, k, v, g, off, out=out)
    val, tol = attn_ref.attention(*(host(s) for s in small[:3]), host(g), np.array([0, 300]), 1,
                                  1.0, dtype="bfloat16")
    check(out[-300:], val["o"], tol["o"], "o")
    assert (out[:-300] == 0).all()
    do = big[:, 2048:2048 + d]
    do[-300:] = small[3]
    dq, dk, dv, _ = lm.logmel_linear_attention_backward(plan, do, q, k, v, g, off)
    val, tol = attn_ref.attention(*(host(s) for s in small[:3]), host(g), np.array([0, 300]), 1,
                                  1.0, do=host(small[3]), dtype="bfloat16")
    for name, t in dict(dq=dq, dk=dk, dv=dv).items():
        check(t[-300:], val[name], tol[name], name)


def test_attention_refusals_of_the_binding(env):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say("attention refusals")
    q, g = torch.zeros((4, 16), device=dev), torch.zeros(2, device=dev)
    off = torch.tensor([0, 4], device=dev)

    def call(**kw):
        d = dict(q=q, k=q, v=q, log_decay=g, seq_offsets=off)
        d.update(kw)
        more = {k: d.pop(k) for k in list(d) if k not in ("q", "k", "v", "log_decay",
                                                          "seq_offsets")}
        return lm.logmel_linear_attention(plan, d["q"], d["k"], d["v"], d["log_decay"],
                                          d["seq_offsets"], **more)

    call()
    for kw in (dict(k=q[:3]), dict(k=q[:, :8]), dict(v=q[:3]), dict(v=q[:, :15]),
               dict(q=q[:, ::2]), dict(log_decay=g[:0]), dict(log_decay=g.view(1, 2)),
               dict(log_decay=g.cpu()), dict(qk_heads=3), dict(qk_heads=0),
               dict(state=torch.zeros((1, 2, 8, 9), device=dev)),
               dict(out=q), dict(seq_offsets=off.int()), dict(log_decay=g.double()),
               dict(k=q.half()), dict(v=q.half()), dict(scale=float("nan")),
               dict(log_decay=torch.zeros(2, device=dev, requires_grad=True)),
               dict(v=torch.zeros((4, 16), device=dev, requires_grad=True))):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call(**kw)


def chain(a, b, c, off, g, scale):
    """o_i = scale a_i S_i of one head row by row in fp64, with its bound: the
    formula over absolute values A, 8 + 2 DK + 64 + 6 roundings for the sums and
    pieces, and 6 + 2 |g| for each of a term's i - j + 1 steps, whose sum over the
    terms is that of the state R_i = lambda R_{i-1} + |S|_i."""
    u, lam = 2.0 ** -24, np.exp(g)
    out, tol, last = np.zeros_like(c), np.zeros_like(c), []
    for lo, hi in zip(off[:-1], off[1:]):
        s = np.zeros((a.shape[1], c.shape[1]))
        p, r = s.copy(), s.copy()
        for t in range(lo, hi):
            x = np.outer(b[t], c[t])
            s = lam * s + x
            p = lam * p + np.abs(x)
            r = lam * r + p
            out[t] = scale * (a[t] @ s)
            m = np.abs(a[t])
            tol[t] = scale * u * ((78 + 2 * a.shape[1]) * (m @ p) + (6 + 2 * abs(g)) * (m @ r))
        last.append(s)
    return out, tol + u * np.abs(out), np.stack(last)


def test_more_places_between_parts_than_one_pass_takes(env):
    """One head and few long sequences: several hundred parts."""
    lm, plan, torch = env
    off = np.array([0, 41000, 41000, 70001], np.int64)
    rng = np.random.default_rng(5)
    q, k, v, do = (rng.normal(size=(70001, 8)).astype(np.float32) for _ in range(4))
    g = np.float32(-2.0 ** -9)
    scale = 0.25
    dev = torch.device("cuda", 0)
    tq, tk, tv, td, tg, to = (torch.from_numpy(np.asarray(x)).to(dev)
                              for x in (q, k, v, do, g.reshape(1), off))
    o = torch.empty_like(tv)
    end = torch.empty(3, 1, 8, 8, device=dev)
    lm.logmel_linear_attention(plan, tq, tk, tv, tg, to, scale=scale, out=o, state_out=end)
    _, _, dv, _ = lm.logmel_linear_attention_backward(plan, td, tq, tk, tv, tg, to, scale=scale)
    f = [x.astype(np.float64) for x in (q, k, v, do)]
    want, tol, last = chain(*f[:3], off, float(g), scale)
    got = o.cpu().numpy()
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol)
    assert (end[1] == 0).all()
    # 512 steps of memory, 6 + 2 |g| and less than 2 more roundings for each
    np.testing.assert_allclose(end[:, 0].cpu().numpy(), last, rtol=0, atol=float(
        2.0 ** -24 * 8 * 512 * np.abs(last).max()))
    want, tol, _ = chain(f[1][::-1], f[0][::-1], f[3][::-1], 70001 - off[::-1], float(g), scale)
    got = dv.cpu().numpy()[::-1]
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv", [(32, 64), (64, 128)])
def test_attention_first_chunk_marks_of_every_wavefront(env, dtype, dk, dv):
    """A value that is not finite in a workgroup's very first chunk, in the
    columns that each wavefront brings in turn: the rows before it keep every
    bit. Each sequence is a workgroup's and has one such value."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say(f"attention first chunk {dtype} {dk} x {dv}")
    dt = getattr(torch, dtype)
    n, length = 512, 40
    gen = torch.Generator(device=dev).manual_seed(21)
    q, k = (torch.randn((n * length, dk), generator=gen, device=dev).to(dt) for _ in range(2))
    v = torch.randn((n * length, dv), generator=gen, device=dev).to(dt)
    off = torch.arange(n + 1, device=dev) * length
    g = torch.tensor([-0.1], device=dev)

    def call():
        return lm.logmel_linear_attention(plan, q, k, v, g, off, max_frames=length)

    whole = call()
    seq = torch.arange(n, device=dev)
    at = 1 + seq % (length - 1)                     # the row in its sequence
    row = seq * length + at
    before = (torch.arange(length, device=dev) < at[:, None]).reshape(-1)
    for x, wide in ((k, dk), (v, dv)):
        col = (seq * 5) % wide                      # every column, in every block of rows
        keep = x[row, col].clone()
        x[row, col] = float("nan")
        got = call()
        x[row, col] = keep
        assert torch.equal(got[before], whole[before])
        behind = got[~before] if x is k else got[torch.arange(n * length, device=dev)[~before],
                                                 col.repeat_interleave(length)[~before]]
        assert torch.isnan(behind).all()
    assert torch.equal(call(), whole)


LARGEST = float(np.finfo(np.float32).max)
NEAR = [(k, "float32") for k in ("q", "k", "v", "do", "score")]
NEAR += [(k, d) for k in ("state", "dstate_out") for d in DTYPES if (k, d) != ("dstate_out", "float16")]


@pytest.mark.parametrize("lens,max_frames", [([11, 0, 9], 11), ([150, 0, 77], 150),
                                             ([1300, 0, 900], 0)])
@pytest.mark.parametrize("dk,dv", [(32, 48), (72, 80)])
@pytest.mark.parametrize("kind,dtype", NEAR)
def test_attention_values_near_the_largest(env, kind, dtype, dk, dv, lens, max_frames):
    """fp32's largest values, and its lowest as masks have it, are values like
    others: in a row operand, in a score, and in a state of rows of any type.
    The rest is small, so that results are finite, and rows before a large one
    keep every bit."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say(f"attention near the largest {kind} {dtype} {dk} x {dv} {lens}")
    dt = getattr(torch, dtype)
    heads, rows, n = 2, sum(lens), len(lens)
    rng = np.random.default_rng(22)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)

    def small(*shape):
        return torch.from_numpy(rng.normal(size=shape) / 64).to(dev)

    t = dict(q=small(rows, heads * dk), k=small(rows, heads * dk), v=small(rows, heads * dv),
             do=small(rows, heads * dv))
    t = {name: x.to(dt) for name, x in t.items()}
    state, dso = (small(n, heads, dk, dv).float() for _ in range(2))
    g = torch.tensor([0.0, -0.05], device=dev)
    # a 2-byte result of such a state is finite where the scale makes it so
    scale = 1.0 if dtype == "float32" else 2.0 ** -120
    args = dict(qk_heads=heads, scale=scale, max_frames=max_frames)
    off_d = torch.from_numpy(off).to(dev)

    def call():
        so = torch.empty_like(state)
        o = lm.logmel_linear_attention(plan, t["q"], t["k"], t["v"], g, off_d, state=state,
                                       state_out=so, **args)
        dq, dkk, dvv, ds = lm.logmel_linear_attention_backward(
            plan, t["do"], t["q"], t["k"], t["v"], g, off_d, state=state, dstate_out=dso, **args)
        return dict(o=o, state_out=so, dq=dq, dk=dkk, dv=dvv, dstate=ds)

    first = call()
    at = [lens[0] - 6, rows - 3]   # a row of each sequence, others before and behind it
    if kind in ("state", "dstate_out"):
        x = state if kind == "state" else dso
        x[..., ::2] = -LARGEST
        x[..., 1::2] = LARGEST
    elif kind == "score":
        t["q"][at], t["k"][:, 5] = 0.0, 1.0
        t["q"][at, 5] = -LARGEST
    else:
        t[kind][at, : t[kind].shape[1] // 2] = -LARGEST
        t[kind][at, -1] = LARGEST
    got = call()
    val, tol = attn_ref.attention(*(host(t[x]) for x in ("q", "k", "v")), host(g), off, heads,
                                  scale, host(state), host(t["do"]), host(dso), dtype=dtype)
    # fp32 sums may overflow on the way, in any order, where the terms' absolute
    # values add up to more than fp32 has (of the scores, those of 1300 rows do)
    most, _ = attn_ref.attention(*(np.abs(host(t[x])) for x in ("q", "k", "v")), host(g), off,
                                 heads, scale, np.abs(host(state)), np.abs(host(t["do"])),
                                 np.abs(host(dso)), dtype=dtype)
    for name, x in got.items():
        with np.errstate(over="ignore"):
            fits = np.isfinite(most[name].astype(np.float32))
        assert fits.mean() > 0.5, name
        check(x[torch.from_numpy(fits).to(dev)], val[name][fits], tol[name][fits], name)
    if kind == "v":
        for lo, hi in ((0, at[0]), (lens[0], at[1])):
            assert torch.equal(got["o"][lo:hi], first["o"][lo:hi])


def test_attention_takes_a_module_s_parameters(env):
    """Every operand may be a torch.nn.Parameter where no graph is recorded,
    the decays too; where one is, it is refused as other tensors are."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say("attention of parameters")
    gen = torch.Generator(device=dev).manual_seed(23)
    x = torch.randn((9, 16), generator=gen, device=dev)
    g = torch.tensor([-0.1, -0.2], device=dev)
    s = torch.randn((2, 2, 8, 8), generator=gen, device=dev)
    off = torch.tensor([0, 5, 9], device=dev)
    px, pg, ps = (torch.nn.Parameter(t.clone()) for t in (x, g, s))
    o = lm.logmel_linear_attention(plan, x, x, x, g, off, state=s)
    with torch.no_grad():
        assert torch.equal(lm.logmel_linear_attention(plan, px, px, px, pg, off, state=ps), o)
        grads = lm.logmel_linear_attention_backward(plan, x, px, px, px, pg, off, state=ps)
    for a, b in zip(grads, lm.logmel_linear_attention_backward(plan, x, x, x, x, g, off, state=s)):
        assert torch.equal(a, b)
    with pytest.raises(RuntimeError):
        lm.logmel_linear_attention(plan, x, x, x, pg, off)


# lengths that are split by parts at each of the widths below: 1603 rows are 7 parts
# of bf16 rows and 13 of others
SPLIT = [900, 0, 700, 3]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,qk", [(6, 2), (3, 3)])
@pytest.mark.parametrize("dk,dv", [(40, 71), (71, 40), (128, 128), (16, 64), (64, 16), (128, 33)])
def test_attention_parts_of_every_shape(env, dtype, heads, qk, dk, dv):
    """Parts with shared heads (whose sums lie before the states in the
    workspace), of unequal widths (dv reads the states that dk formed), and of
    either number of wavefronts."""
    say(f"attention parts {dtype} {heads} heads, {qk} of q and k, {dk} x {dv}")
    attn_case(env, dtype, SPLIT, heads=heads, qk=qk, dk=dk, dv=dv, behind=5, seed=24,
              layout="odd" if dk == 40 else "dense", state=dk != 16)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_parts_state_in_place(env, dtype):
    say(f"attention parts in place {dtype}")
    attn_case(env, dtype, SPLIT, heads=6, qk=2, dk=40, dv=71, train=False, in_place=True, seed=25)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_not_finite_across_parts(env, dtype):
    """In the first, a middle and the last part of a sequence: earlier rows,
    other sequences and other heads keep every bit, and the states between the
    parts carry it to the last row. In the gradient as the formulas have it: of
    do to dk and dv of its row and earlier ones and dq of its row, of k to dq of
    its row and later ones and dv of its row, of v to dq and dk so."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say(f"attention not finite across parts {dtype}")
    dt = getattr(torch, dtype)
    lens, heads, d, e = [500, 1700, 300], 2, 32, 72
    rows, lo, hi = sum(lens), 500, 2200
    gen = torch.Generator(device=dev).manual_seed(26)
    q, k = (torch.randn((rows, heads * d), generator=gen, device=dev).to(dt) for _ in range(2))
    v, do = (torch.randn((rows, heads * e), generator=gen, device=dev).to(dt) for _ in range(2))
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device=dev)
    g = torch.tensor([-0.001, -0.002], device=dev)

    def call():
        o = lm.logmel_linear_attention(plan, q, k, v, g, off)
        grads = lm.logmel_linear_attention_backward(plan, do, q, k, v, g, off)
        return dict(zip(("o", "dq", "dk", "dv"), (o, *grads)))

    first = call()
    wide = dict(o=e, dq=d, dk=d, dv=e)
    # of each operand the rows of each result that it reaches, from its own
    later, earlier, own, none = (0, hi), (lo, 1), (0, 1), None
    reach = dict(q=dict(o=own, dq=none, dk=earlier, dv=earlier),
                 k=dict(o=later, dq=later, dk=none, dv=own),
                 v=dict(o=later, dq=later, dk=own, dv=none),
                 do=dict(o=none, dq=own, dk=earlier, dv=earlier))
    for name, x in dict(q=q, k=k, v=v, do=do).items():
        for row, head in ((lo + 3, 0), (lo + 850, 1), (hi - 2, 0)):
            col = head * (x.shape[1] // heads) + 7
            for bad in (float("nan"), float("inf")):
                keep = x[row, col].clone()
                x[row, col] = bad
                got = call()
                x[row, col] = keep
                for key, to in reach[name].items():
                    same = torch.ones_like(first[key], dtype=torch.bool)
                    cols = slice(head * wide[key], (head + 1) * wide[key])
                    if to is not none:
                        a, b = {later: (row, hi), earlier: (lo, row + 1), own: (row, row + 1)}[to]
                        same[a:b, cols] = False
                        for far in (a, b - 1):
                            assert not torch.isfinite(got[key][far, cols]).all(), (name, key, row)
                    assert torch.equal(got[key][same], first[key][same]), (name, key, row, bad)
    again = call()
    assert all(torch.equal(again[key], first[key]) for key in first)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,max_frames", [([8, 0, 3], 8), ([150, 90], 150), ([1300, 700], 0)])
def test_attention_state_not_finite_stays_in_its_column(env, dtype, lens, max_frames):
    """A NaN or infinity in an initial state reaches its column of the outputs
    and of the state behind them, in its sequence and head."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say(f"attention state not finite {dtype} {lens}")
    dt = getattr(torch, dtype)
    heads, d, e, n = 2, 32, 48, len(lens)
    gen = torch.Generator(device=dev).manual_seed(27)
    q, k = (torch.randn((sum(lens), heads * d), generator=gen, device=dev).to(dt)
            for _ in range(2))
    v = torch.randn((sum(lens), heads * e), generator=gen, device=dev).to(dt)
    s = torch.randn((n, heads, d, e), generator=gen, device=dev)
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device=dev)
    g = torch.tensor([-0.001, 0.0], device=dev)

    def call():
        so = torch.empty_like(s)
        o = lm.logmel_linear_attention(plan, q, k, v, g, off, state=s, state_out=so,
                                       max_frames=max_frames)
        return o, so

    first = call()
    for bad in (float("nan"), float("inf")):
        s[0, 1, 5, 40] = bad
        o, so = call()
        s[0, 1, 5, 40] = 1.0
        same, same_s = (torch.ones_like(t, dtype=torch.bool) for t in first)
        same[:lens[0], e + 40] = False
        same_s[0, 1, :, 40] = False
        assert torch.equal(o[same], first[0][same]) and torch.equal(so[same_s], first[1][same_s])
        assert not torch.isfinite(o[lens[0] - 1, e + 40]) and not torch.isfinite(so[0, 1, 5, 40])


@pytest.mark.parametrize("length,max_frames", [(17, 17), (4, 4)])
def test_attention_more_sequences_than_a_launch_has_workgroups(env, length, max_frames):
    """Workgroups that take several sequences: the first, the last and others
    between against the fp64 form, the states too."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    heads, d = 4, 8
    n = 300_000 if length > 16 else 1_100_000     # items past 2^20 and 2^22
    say(f"attention of {n} sequences x {length}")
    gen = torch.Generator(device=dev).manual_seed(28)
    q, k, v = (torch.randn((n * length, heads * d), generator=gen, device=dev).to(torch.bfloat16)
               for _ in range(3))
    s = torch.randn((n, heads, d, d), generator=gen, device=dev)
    so = torch.empty_like(s)
    g = torch.tensor([-0.1, -0.5, 0.0, -2.0], device=dev)
    off = torch.arange(n + 1, device=dev) * length
    o = lm.logmel_linear_attention(plan, q, k, v, g, off, state=s, state_out=so,
                                   max_frames=max_frames)
    for at in (0, n // 2 - 1, (1 << 20) // heads - 1, (1 << 20) // heads, n - 2):
        rows = slice(at * length, (at + 2) * length)
        val, tol = attn_ref.attention(*(host(x[rows]) for x in (q, k, v)), host(g),
                                      np.arange(3) * length, heads, 1.0, host(s[at:at + 2]),
                                      dtype="bfloat16")
        check(o[rows], val["o"], tol["o"], "o")
        check(so[at:at + 2], val["state_out"], tol["state_out"], "state_out")
