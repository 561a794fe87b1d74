"""The group norm on the GPU, with its gradient, against the fp64 form of
attn_ref.py, whose bounds follow from the number of roundings; and a layer of
both operators along streams."""

import numpy as np
import pytest

from tests import attn_ref
from tests.test_gpu_attention import untouched
from tests.test_gpu_rows import DTYPES, Rows, check, env, host, say  # noqa: F401

pytestmark = pytest.mark.gpu


def norm_case(env, dtype, groups, width, lens=None, rows=None, layout="dense", affine=True,
              silu=False, gate=False, behind=0, max_frames=0, seed=0, level=0.0, spread=1.0,
              eps=1e-5):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    c = groups * width
    off = None
    if lens is not None:
        off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        rows = int(off[-1]) + behind
    last = rows if off is None else int(off[-1])
    mk = Rows(torch, dtype, rows, c, layout, seed)
    x = mk.of(mk.rng.normal(size=(rows, c)) * spread + level * mk.rng.normal(size=c))
    o = mk.normal() if gate else None
    dy = mk.normal()

    def f32(lo):
        return torch.from_numpy((mk.rng.normal(size=c) + lo).astype(np.float32)).to(dev)

    w, b = (f32(1.0), f32(0.0)) if affine else (None, None)
    y, dx = mk.empty(), mk.empty()
    dg = mk.empty() if gate else None
    more = dict(weight=w, bias=b, gate=o, activation="silu" if silu else None, eps=eps)
    stats = None
    if off is not None:
        more.update(seq_offsets=torch.from_numpy(off).to(dev), max_frames=max_frames)
        stats = torch.full((len(lens), groups, 2), 7.0, device=dev)
    lm.logmel_group_norm(plan, x, groups, out=y, stats=stats, **more)
    grads = lm.logmel_group_norm_backward(plan, dy, x, groups, stats=stats, dx=dx, dgate=dg,
                                          **more)
    torch.cuda.synchronize()
    arg = [None if t is None else host(t) for t in (w, b, o)]
    val, tol = attn_ref.group_norm(host(x), groups, *arg, silu=silu, off=off, eps=eps,
                                   dy=host(dy), dtype=dtype)
    got = dict(y=y, **{k: t for k, t in grads.items() if t is not None})
    for name, t in got.items():
        if name in ("y", "dx", "dgate"):
            check(t[:last], val[name][:last], tol[name][:last], name)
            assert (t[last:] == 7.0).all(), name
            if layout != "dense":
                assert untouched(torch, t), name
        else:
            check(t, val[name], tol[name], name)
    assert set(got) == set(val)


PARTS = [dict(), dict(silu=True), dict(gate=True), dict(silu=True, gate=True, affine=False),
         dict(affine=False)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("parts", range(len(PARTS)))
def test_group_norm_parts(env, dtype, parts):
    for lens in (None, [40, 0, 1, 130, 7]):
        say(f"group norm {dtype} parts {parts} over {lens}")
        norm_case(env, dtype, 4, 24, lens=lens, rows=77, behind=3, seed=parts, **PARTS[parts])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["dense", "slice", "odd"])
@pytest.mark.parametrize("groups,width", [(1, 1), (1, 2), (5, 1), (3, 3), (8, 64), (2, 7),
                                          (3, 107), (32, 16), (1, 257), (64, 128), (1, 8192),
                                          (2, 1500), (16, 40)])
def test_group_norm_widths(env, dtype, layout, groups, width):
    for lens in (None, [33, 0, 70]):
        say(f"group norm {dtype} {layout} {groups} x {width} over {lens}")
        norm_case(env, dtype, groups, width, lens=lens, rows=21, layout=layout, behind=2,
                  seed=width, silu=True, gate=width % 2 == 0)


SEQS = {
    "one": [1],
    "empty_around": [0, 1, 0, 0, 5, 0],
    "ones": [1] * 130,
    "edges": [127, 1, 128, 129, 0, 256, 3],
    "long": [4000],
    "ragged": [700, 2, 0, 1333, 41],
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seqs", sorted(SEQS))
def test_group_norm_lengths(env, dtype, seqs):
    lens = SEQS[seqs]
    for max_frames in (0, 1, max(lens)):
        say(f"group norm {dtype} {seqs} max_frames {max_frames}")
        norm_case(env, dtype, 3, 20, lens=lens, behind=5, silu=True, max_frames=max_frames)


@pytest.mark.parametrize("lens", [None, [900, 60, 3]])
def test_group_norm_levels_far_above_the_spread(env, lens):
    """Means a thousand times the spread: the variance is that of what is left
    (fp32; 2-byte rows have rounded it away before)."""
    say(f"group norm levels {lens}")
    norm_case(env, "float32", 2, 1, lens=lens, rows=50, level=1e3, spread=1.0, eps=1e-3)
    norm_case(env, "float32", 4, 16, lens=lens, rows=50, level=30.0, spread=0.01, eps=1e-5)


def test_group_norm_constant_rows_and_eps(env):
    """Rows of one value have a variance of 0: y is the bias, and dx is
    finite."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say("group norm of constant rows")
    x = torch.full((10, 64), -3.25, dtype=torch.bfloat16, device=dev)
    b = torch.randn(64, device=dev)
    for off in (None, torch.tensor([0, 4, 10], device=dev)):
        st = None if off is None else torch.empty((2, 4, 2), device=dev)
        y = lm.logmel_group_norm(plan, x, 4, bias=b, seq_offsets=off, stats=st)
        assert torch.equal(y, b.to(torch.bfloat16).expand(10, 64))
        g = lm.logmel_group_norm_backward(plan, x, x, 4, stats=st, bias=b, seq_offsets=off)
        assert torch.isfinite(g["dx"]).all()
        assert torch.equal(g["dbias"], torch.full((64,), -32.5, device=dev))


def test_group_norm_not_finite_stays_in_its_mean(env):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    for dtype in DTYPES:
        say(f"group norm not finite {dtype}")
        x = torch.randn((60, 48), device=dev).to(getattr(torch, dtype))
        off = torch.tensor([0, 20, 45, 60], device=dev)
        for o in (None, off):
            y = lm.logmel_group_norm(plan, x, 3, seq_offsets=o)
            for bad in (float("nan"), float("inf")):
                z = x.clone()
                z[30, 20] = bad
                b = lm.logmel_group_norm(plan, z, 3, seq_offsets=o)
                same = torch.ones_like(x, dtype=torch.bool)
                same[slice(30, 31) if o is None else slice(20, 45), 16:32] = False
                assert torch.equal(b[same], y[same])
                assert not torch.isfinite(b[30, 20])


def test_group_norm_nothing(env):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say("group norm of nothing")
    x = torch.randn((4, 16), device=dev)
    w = torch.ones(16, device=dev)
    y = torch.full_like(x, 7.0)
    none = torch.zeros(1, dtype=torch.int64, device=dev)
    st = torch.empty((0, 2, 2), device=dev)
    lm.logmel_group_norm(plan, x, 2, weight=w, seq_offsets=none, out=y, stats=st)
    assert (y == 7.0).all()
    g = lm.logmel_group_norm_backward(plan, x, x, 2, weight=w, seq_offsets=none, stats=st, dx=y)
    assert (y == 7.0).all() and (g["dweight"] == 0).all()
    g = lm.logmel_group_norm_backward(plan, x[:0], x[:0], 2, weight=w, bias=w)
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()
    # sequences of no rows at all
    off = torch.zeros(4, dtype=torch.int64, device=dev)
    st = torch.empty((3, 2, 2), device=dev)
    lm.logmel_group_norm(plan, x, 2, seq_offsets=off, out=y, stats=st)
    assert (y == 7.0).all()
    g = lm.logmel_group_norm_backward(plan, x, x, 2, weight=w, seq_offsets=off, stats=st, dx=y)
    assert (y == 7.0).all() and (g["dweight"] == 0).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("over", ["row", "clip"])
def test_group_norm_same_bits_other_stream_and_graph(env, dtype, over):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say(f"group norm graph {dtype} {over}")
    x, o, dy = (torch.randn((1500, 96), device=dev).to(getattr(torch, dtype)) for _ in range(3))
    w, b = torch.randn(96, device=dev), torch.randn(96, device=dev)
    off = torch.tensor([0, 700, 705, 1400], device=dev) if over == "clip" else None

    def call(stream=None):
        more = dict(weight=w, bias=b, gate=o, activation="silu", seq_offsets=off, stream=stream)
        st = None if off is None else torch.empty((3, 4, 2), device=dev)
        y = torch.zeros_like(x)
        dx, dg = torch.zeros_like(x), torch.zeros_like(x)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        lm.logmel_group_norm(plan, x, 4, out=y, stats=st, **more)
        g = lm.logmel_group_norm_backward(plan, dy, x, 4, stats=st, dx=dx, dgate=dg, **more)
        return [y, *g.values()]

    first = [t.clone() for t in call()]
    assert all(torch.equal(a, c) for a, c in zip(first, call()))
    side = torch.cuda.Stream()
    other = call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for _ in range(3):
        for t in held:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(first, held))
        assert all(torch.equal(a, c) for a, c in zip(first, call()))


@pytest.mark.parametrize("over", ["row", "clip"])
def test_group_norm_offsets_past_32_bits(env, over):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say(f"group norm past 2^31 elements, {over}")
    rows, wide, c = 70_000, 32_768, 64
    big = torch.ones((rows, wide), dtype=torch.bfloat16, device=dev)
    x, y, dy, dx = (big[:, i * 512 + 8:i * 512 + 8 + c] for i in range(4))
    mk = np.random.default_rng(13)
    parts = [torch.from_numpy(mk.normal(size=(500, c))).to(torch.bfloat16).to(dev)
             for _ in range(2)]
    x[-500:], dy[-500:] = parts
    off = np.array([0, rows - 500, rows])
    more, st = {}, None
    if over == "clip":
        st = torch.empty((2, 4, 2), device=dev)
        more = dict(seq_offsets=torch.from_numpy(off).to(dev))
    lm.logmel_group_norm(plan, x, 4, out=y, stats=st, **more)
    lm.logmel_group_norm_backward(plan, dy, x, 4, stats=st, dx=dx, **more)
    val, tol = attn_ref.group_norm(host(parts[0]), 4, off=None if over == "row" else
                                   np.array([0, 500]), dy=host(parts[1]), dtype="bfloat16")
    check(y[-500:], val["y"], tol["y"], "y")
    check(dx[-500:], val["dx"], tol["dx"], "dx")
    assert (y[:-500] == 0).all()


def test_group_norm_refusals_of_the_binding(env):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say("group norm refusals")
    x = torch.zeros((4, 16), device=dev)
    off = torch.tensor([0, 4], device=dev)
    st = torch.zeros((1, 2, 2), device=dev)
    lm.logmel_group_norm(plan, x, 2, seq_offsets=off, stats=st)
    for kw in (dict(groups=3), dict(groups=0), dict(activation="gelu"), dict(weight=x[0, :8]),
               dict(gate=x[:3]), dict(gate=x.half()), dict(stats=st), dict(out=x), dict(eps=-1.0),
               dict(max_frames=3), dict(seq_offsets=off, stats=st[:, :1]),
               dict(bias=torch.zeros(16, device=dev, requires_grad=True))):
        d = dict(groups=2)
        d.update(kw)
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            lm.logmel_group_norm(plan, x, **d)
    with pytest.raises(lm.LogmelError):
        lm.logmel_group_norm_backward(plan, x, x, 2, seq_offsets=off)


def test_layer_along_streams(env):
    """Log-mel rows of streams through a layer of both operators, push by push
    with the states carried in place, against the same layer over the whole
    recordings in fp64: the norm of each row, one product to q, k, v and gate,
    linear attention, the norm of each head with the gate."""
    import logmel_synth as S
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say("layer along streams")
    n, heads, d = 3, 2, 16
    clips = [S.speech_like(60 + j, 12800, "cuda") for j in range(n)]
    x, fo = lm.log_mel(plan, torch.cat(clips), np.arange(n + 1, dtype=np.int64) * 12800)
    frames = int(fo[1])
    rng = np.random.default_rng(14)
    w = torch.from_numpy(rng.normal(size=(128, 4 * heads * d)).astype(np.float32) / 11.3).to(dev)
    g = torch.tensor([-0.2, -0.02], device=dev)
    c = heads * d

    def layer(rows, off, state, state_out, max_frames):
        z = lm.logmel_group_norm(plan, rows, 1)
        p = z @ w
        q, k, v, gate = (p[:, i * c:(i + 1) * c] for i in range(4))
        o = lm.logmel_linear_attention(plan, q, k, v, g, off, scale=d ** -0.5, state=state,
                                       state_out=state_out, max_frames=max_frames)
        return lm.logmel_group_norm(plan, o, heads, gate=gate), p, o

    off = torch.from_numpy(fo).to(dev)
    whole, p, o = layer(x, off, None, None, frames)
    # the operators' parts of the layer in fp64, from the same product
    q, k, v, gate = (host(p[:, i * c:(i + 1) * c]) for i in range(4))
    val, tol = attn_ref.attention(q, k, v, host(g), fo, heads, d ** -0.5)
    check(o, val["o"], tol["o"], "o")
    val, tol = attn_ref.group_norm(host(o), heads, gate=gate)
    check(whole, val["y"], tol["y"], "y")
    # push by push: the product's own rounding differs by the rows it is called
    # on, the norms divide by a spread that it may be large against
    state = torch.zeros((n, heads, d, d), device=dev)
    got, at = [], 0
    per = x.view(n, frames, 128)
    while at < frames:
        push = min(8, frames - at)
        rows = per[:, at:at + push].reshape(n * push, 128).contiguous()
        y, _, _ = layer(rows, torch.arange(n + 1, device=dev) * push, state, state, push)
        got.append(y.view(n, push, c))
        at += push
    got = torch.cat(got, 1).reshape(n * frames, c)
    # 128-term products of values to 4 (the norm) and 1/3: sums to about 4, off
    # by up to 128 roundings of 2^-24 times 20; then as above, 2^-10 in all
    assert (got - whole).abs().max().item() <= 2.0 ** -10 * whole.abs().max().item()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("groups,width", [(1, 4096), (2, 257), (1, 8192)])
def test_group_norm_wide_groups_of_many_sequences(env, dtype, groups, width):
    say(f"group norm wide, many sequences {dtype} {groups} x {width}")
    norm_case(env, dtype, groups, width, lens=[1, 0, 2] * 100, behind=2, silu=True, seed=31)


def test_group_norm_parameter_sums_do_not_grow_with_sequences(env):
    """Half a million sequences of one row, of a group too wide to be summed in
    registers: parts of 512 sequences. Every row is the same, so a parameter's
    sum is the count times one value; its parts are rounded once (2^-24), as the
    result is, and dn xh once before (dn itself is dy)."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say("group norm parameter sums of 2^19 sequences")
    rows, width = 1 << 19, 257
    x = torch.ones((rows, width), device=dev)
    x[:, ::2] = -1.0
    dy = torch.full((rows, width), 1.0 + 0.4 * 2.0 ** -16, device=dev)
    off = torch.arange(rows + 1, device=dev)
    w, b = torch.ones(width, device=dev), torch.zeros(width, device=dev)
    more = dict(weight=w, bias=b, seq_offsets=off, max_frames=1)
    st = torch.empty((rows, 1, 2), device=dev)
    y = lm.logmel_group_norm(plan, x, 1, stats=st, **more)
    assert (y == y[0]).all()                      # xh, as weight is 1 and bias 0
    g = lm.logmel_group_norm_backward(plan, dy, x, 1, stats=st, **more)
    u = 2.0 ** -24
    want = host(dy[0]) * rows
    assert (np.abs(host(g["dbias"]) - want) <= 2 * u * want).all()
    want = host(dy[0]) * host(y[0]) * rows
    assert (np.abs(host(g["dweight"]) - want) <= 3 * u * np.abs(want)).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("over", ["row", "clip"])
def test_group_norm_squares_that_overflow(env, dtype, over):
    """A group whose squares pass fp32 is normed to 0: y is that of a constant
    group; other groups keep every bit. Where the sums pass it too, NaN."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say(f"group norm of squares that overflow {dtype} {over}")
    gen = torch.Generator(device=dev).manual_seed(32)
    x = torch.randn((40, 64), generator=gen, device=dev).to(getattr(torch, dtype))
    b = torch.randn(64, generator=gen, device=dev)
    off = torch.tensor([0, 25, 40], device=dev) if over == "clip" else None

    def call(t):
        return lm.logmel_group_norm(plan, t, 4, bias=b, activation="silu", seq_offsets=off)

    y, flat = call(x), call(torch.full_like(x, 2.0))
    big = x.clone()
    big[:, 16:32] *= 1e25
    got = call(big)
    assert torch.equal(got[:, 16:32], flat[:, 16:32])
    big[:, 16:32] = 3e38
    assert torch.isnan(call(big)[:, 16:32]).all()
    for lo, hi in ((0, 16), (32, 64)):
        assert torch.equal(got[:, lo:hi], y[:, lo:hi])


def test_group_norm_more_sequences_than_a_launch_has_wavefronts(env):
    """Half a million sequences of two rows and 16 groups: those across parts
    are joined by wavefronts that take several."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say("group norm of 2^19 sequences x 16 groups")
    n, groups, width = 1 << 19, 16, 4
    gen = torch.Generator(device=dev).manual_seed(33)
    x, dy = (torch.randn((2 * n - 1, groups * width), generator=gen, device=dev) for _ in range(2))
    off = torch.arange(n + 1, device=dev) * 2 - 1
    off[0] = 0                                      # parts begin inside sequences
    st = torch.empty((n, groups, 2), device=dev)
    y = lm.logmel_group_norm(plan, x, groups, seq_offsets=off, stats=st, max_frames=2)
    g = lm.logmel_group_norm_backward(plan, dy, x, groups, seq_offsets=off, stats=st, max_frames=2)
    for at in (1, 2 * (n // 3) - 1, 2 * n - 1 - 4000):
        rows = slice(at, at + 4000)
        val, tol = attn_ref.group_norm(host(x[rows]), groups, off=np.arange(2001) * 2,
                                       dy=host(dy[rows]))
        check(y[rows], val["y"], tol["y"], "y")
        check(g["dx"][rows], val["dx"], tol["dx"], "dx")
