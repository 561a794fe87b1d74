"""The row operators on the GPU: the gated scan and the block norm, with their
gradients, against the fp64 forms of rows_ref.py, whose bounds follow from the
number of roundings."""

import sys

import numpy as np
import pytest

import logmel_synth as S
from tests import rows_ref

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "float16", "bfloat16"]


def say(msg):
    print(f"[gpu-case] {msg}", flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from tests.libload import load_binding
    lm = load_binding()
    plan = lm.logmel_plan_create(0)
    return lm, plan, torch


def host(t):
    return t.double().cpu().numpy()


def check(got, val, tol, what):
    got = host(got)
    assert got.shape == val.shape, what
    bad = ~(np.abs(got - val) <= tol)
    if bad.any():
        i = tuple(int(k) for k in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: "
                             f"{got[i]} for {val[i]}, bound {tol[i]}")


class Rows:
    """Row operands of one call in the wanted layout, spare values around."""

    def __init__(self, torch, dtype, rows, channels, layout, seed):
        self.torch, self.rows, self.c = torch, rows, channels
        self.dtype = getattr(torch, dtype)
        self.layout = layout
        self.rng = np.random.default_rng(seed)

    def of(self, array):
        t = self.empty()
        t.copy_(self.torch.from_numpy(np.ascontiguousarray(array)).to(t.device))
        return t

    def empty(self):
        torch, r, c = self.torch, self.rows, self.c
        dev = torch.device("cuda", 0)
        if self.layout == "dense":
            return torch.full((r, c), 7.0, dtype=self.dtype, device=dev)
        if self.layout == "slice":      # columns of a wider product, aligned
            return torch.full((r, 3 * c + 16), 7.0, dtype=self.dtype, device=dev)[:, 8:8 + c]
        # odd stride, odd start: no alignment beyond the element's
        return torch.full((r * (c + 3) + 1,), 7.0, dtype=self.dtype, device=dev)[1:].view(
            r, c + 3)[:, :c]

    def normal(self, scale=1.0):
        return self.of(self.rng.normal(size=(self.rows, self.c)) * scale)


SEQS = {
    "one": [1],
    "empty_around": [0, 1, 0, 0, 5, 0],
    "ones": [1] * 130,
    "edges": [127, 1, 128, 129, 0, 256, 3],
    "ragged": [700, 2, 0, 333, 41],
    "long": [4000],
}


def scan_case(env, dtype, channels, lens, layout, bias, state, behind=0, max_frames=0, seed=0,
              gate_scale=2.0):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    rows, n = int(off[-1]) + behind, len(lens)
    mk = Rows(torch, dtype, rows, channels, layout, seed)
    x, g, dh = mk.normal(), mk.normal(gate_scale), mk.normal()
    rng = mk.rng

    def f32(*shape, lo=0.0):
        return torch.from_numpy(rng.normal(size=shape).astype(np.float32) + np.float32(lo)).to(dev)

    b = f32(channels, lo=1.0) if bias else None
    h0 = f32(n, channels) if state else None
    dso = f32(n, channels) if state else None
    off_d = torch.from_numpy(off).to(dev)
    h, dx, dg = mk.empty(), mk.empty(), mk.empty()
    so = torch.full((n, channels), 7.0, device=dev)
    ck = torch.full((lm.logmel_gated_scan_checkpoint_rows(rows), channels), float("nan"),
                    device=dev)
    lm.logmel_gated_scan(plan, x, g, off_d, bias=b, state=h0, out=h, state_out=so, checkpoints=ck,
                         max_frames=max_frames)
    _, _, db, ds = lm.logmel_gated_scan_backward(plan, dh, x, g, off_d, ck, bias=b, state=h0,
                                                 dstate_out=dso, dx=dx, dgate=dg,
                                                 max_frames=max_frames)
    torch.cuda.synchronize()
    arg = [None if t is None else host(t) for t in (b, h0)]
    val, tol = rows_ref.scan(host(x), host(g), off, *arg, dh=host(dh),
                             dstate_out=None if dso is None else host(dso), dtype=dtype)
    last = int(off[-1])
    got = dict(h=h, state_out=so, dx=dx, dgate=dg)
    if bias:
        got["dbias"] = db
    if state:
        got["dstate"] = ds
    for k, t in got.items():
        if k in ("h", "dx", "dgate"):
            check(t[:last], val[k][:last], tol[k][:last], k)
            # rows behind the last sequence and values between the rows stay
            assert (t[last:] == 7.0).all(), k
        else:
            check(t, val[k], tol[k], k)
    if layout != "dense":
        for k in ("h", "dx", "dgate"):
            base = got[k]._base if got[k]._base is not None else got[k]
            whole = base.flatten().clone()
            at = torch.as_strided(torch.arange(whole.numel(), device=dev), got[k].shape,
                                  got[k].stride(), got[k].storage_offset())
            whole[at.reshape(-1)] = 7.0
            assert (whole == 7.0).all(), k
    return val


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seqs", sorted(SEQS))
def test_scan_lengths(env, dtype, seqs):
    lens = SEQS[seqs]
    for max_frames in (0, max(lens)):
        say(f"scan {dtype} {seqs} max_frames {max_frames}")
        scan_case(env, dtype, 66, lens, "dense", True, True, behind=5, max_frames=max_frames)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["dense", "slice", "odd"])
@pytest.mark.parametrize("channels", [1, 2, 3, 64, 127, 128, 257])
def test_scan_widths(env, dtype, layout, channels):
    say(f"scan {dtype} {layout} {channels} channels")
    scan_case(env, dtype, channels, [300, 0, 77], layout, channels % 2 == 1, layout != "slice",
              behind=2, seed=channels)


@pytest.mark.parametrize("seqs", ["long", "ragged"])
def test_scan_wide_and_split(env, seqs):
    say(f"scan wide {seqs}")
    scan_case(env, "bfloat16", 640, SEQS[seqs] + [150, 900], "slice", True, True, behind=130,
              seed=11)


@pytest.mark.parametrize("dtype", DTYPES)
def test_scan_very_wide_rows(env, dtype):
    say(f"scan {dtype} 70,001 channels")
    scan_case(env, dtype, 70001, [3, 0, 2], "odd", True, True, behind=1, seed=13)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_scan_tens_of_thousands_of_sequences(env, dtype):
    lens = np.random.default_rng(14).integers(0, 4, size=30000).tolist()
    for max_frames in (0, 3):
        say(f"scan {dtype} 30,000 sequences max_frames {max_frames}")
        scan_case(env, dtype, 3, lens, "dense", True, True, behind=1, max_frames=max_frames,
                  seed=15)


@pytest.mark.parametrize("max_frames", [1, 200, 1 << 40])
def test_scan_wrong_hint_changes_no_result(env, max_frames):
    """max_frames below and far above the longest sequence: another split, the
    same recurrence."""
    say(f"scan max_frames {max_frames}")
    for n in (1, 40):
        scan_case(env, "float16", 130, [700, 3, 0, 129] * n, "slice", True, True,
                  max_frames=max_frames, seed=16)


def test_scan_long_sequence_many_parts(env):
    say("scan 60000 rows x 4")
    scan_case(env, "float32", 4, [60000, 17], "dense", True, True, seed=12, gate_scale=1.0)


def test_scan_gate_extremes(env):
    """Gates at both infinities, at the type's lowest and largest values and
    far out hold the state or take the row, with finite gradients; a NaN and
    an infinity stay in their sequence and channel."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    for dtype in DTYPES:
        say(f"scan extremes {dtype}")
        dt = getattr(torch, dtype)
        inf = float("inf")
        top = float(torch.finfo(dt).max)
        col = torch.tensor([inf, -inf, top, -top, 30.0, -30.0, 100.0, -100.0, 0.0, inf, inf, -inf])
        rows = 3 * len(col)
        g = torch.cat([col, col.flip(0), col]).unsqueeze(1).repeat(1, 64).to(dt).to(dev)
        rng = np.random.default_rng(5)
        x = torch.from_numpy(rng.normal(size=(rows, 64))).to(dt).to(dev)
        dh = torch.from_numpy(rng.normal(size=(rows, 64))).to(dt).to(dev)
        off = np.array([0, 12, 24, 36])
        off_d = torch.from_numpy(off).to(dev)
        ck = torch.zeros((1, 64), device=dev)
        h = lm.logmel_gated_scan(plan, x, g, off_d, checkpoints=ck)
        dx, dg, _, _ = lm.logmel_gated_scan_backward(plan, dh, x, g, off_d, ck)
        hg = host(g)
        val, tol = rows_ref.scan(host(x), np.clip(hg, -1e4, 1e4), off, dh=host(dh), dtype=dtype)
        # beyond |gate| 60 a and u are 0 and 1 to far below the smallest step
        # here; the bound's |gate| factor is that of the products that remain
        _, tol = rows_ref.scan(host(x), np.clip(hg, -60, 60), off, dh=host(dh), dtype=dtype)
        for k, t in dict(h=h, dx=dx, dgate=dg).items():
            check(t, val[k], tol[k] + 1e-20, k)
        x[3, 5] = float("nan")
        x[14, 7] = inf
        h2 = lm.logmel_gated_scan(plan, x, g, off_d)
        same = torch.ones((rows, 64), dtype=torch.bool)
        same[3:12, 5] = False
        same[14:24, 7] = False
        same = same.to(dev)
        assert torch.equal(h2[same], h[same])
        assert torch.isnan(h2[3:12, 5]).all()
        assert not torch.isfinite(h2[15, 7])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [8, 300, 4000])
def test_scan_closes_behind_the_largest_values(env, dtype, rows):
    """A row near the type's largest and lowest values, taken whole, and a gate
    at the lowest value behind it: nothing of the large state is left."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say(f"scan closes {dtype} {rows} rows")
    dt = getattr(torch, dtype)
    top = float(torch.finfo(dt).max)
    rng = np.random.default_rng(rows)
    x = torch.from_numpy(rng.normal(size=(rows, 64))).to(dt).to(dev)
    g = torch.from_numpy(rng.normal(size=(rows, 64))).to(dt).to(dev)
    first = rows // 2   # of the rows from the closing one on
    x[first - 1, 0::2], x[first - 1, 1::2] = top / 4, -top / 4
    g[first - 1 : first + 1] = -top
    state_out = torch.empty((1, 64), device=dev)
    off_d = torch.tensor([0, rows], device=dev)
    h = lm.logmel_gated_scan(plan, x, g, off_d, state_out=state_out)
    assert torch.isfinite(h[first - 1]).all() and (h[first - 1].abs() > top / 5).all()
    # from there on it is the recurrence of a sequence that starts there
    val, tol = rows_ref.scan(host(x)[first:], np.maximum(host(g)[first:], -60.0),
                             np.array([0, rows - first]), dtype=dtype)
    check(h[first:], val["h"], tol["h"] + 1e-20, "h")
    check(state_out, val["state_out"], tol["state_out"] + 1e-20, "state_out")


def test_scan_pushes_carry_the_state(env):
    """Streams fed a few rows at a time with the state updated in place give
    the rows of the whole sequences (streams that get nothing included)."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    rng = np.random.default_rng(6)
    n, c, total = 37, 96, 40
    x = rng.normal(size=(n, total, c)).astype(np.float32)
    g = rng.normal(size=(n, total, c)).astype(np.float32)
    state = torch.zeros((n, c), device=dev)
    done = np.zeros(n, dtype=int)
    parts = [[] for _ in range(n)]
    while done.min() < total:
        take = np.minimum(rng.integers(0, 10, n), total - done)
        off = np.concatenate([[0], np.cumsum(take)]).astype(np.int64)
        cat = [np.concatenate([v[j, done[j]:done[j] + take[j]] for j in range(n)]) for v in (x, g)]
        xd, gd = (torch.from_numpy(v).to(dev) for v in cat)
        h = lm.logmel_gated_scan(plan, xd, gd, torch.from_numpy(off).to(dev), state=state,
                                 state_out=state)
        for j in range(n):
            parts[j].append(host(h[off[j]:off[j + 1]]))
        done += take
    off = np.arange(n + 1) * total
    val, tol = rows_ref.scan(x.reshape(-1, c), g.reshape(-1, c), off)
    got = np.concatenate([np.concatenate(p) for p in parts])
    # each row is also rounded to fp32 nowhere but in the state: same bounds
    assert (np.abs(got - val["h"]) <= tol["h"]).all()
    check(state, val["state_out"], tol["state_out"], "state")


def test_scan_state_in_place_over_many_parts(env):
    """state_out = state where a sequence spans parts of the split."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    lens = [0, 9000, 3, 0, 7000, 1, 0]
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    off_d = torch.from_numpy(off).to(dev)
    gen = torch.Generator(device=dev).manual_seed(1)
    x, g = (torch.randn((int(off[-1]), 130), generator=gen, device=dev) for _ in range(2))
    state = torch.randn((len(lens), 130), generator=gen, device=dev)
    for mf in (0, 9000, 1):
        say(f"in place, max_frames {mf}")
        apart = torch.empty_like(state)
        h = lm.logmel_gated_scan(plan, x, g, off_d, state=state, state_out=apart, max_frames=mf)
        kept = state.clone()
        h2 = lm.logmel_gated_scan(plan, x, g, off_d, state=kept, state_out=kept, max_frames=mf)
        assert torch.equal(h, h2) and torch.equal(apart, kept)
        again = lm.logmel_gated_scan(plan, x, g, off_d, state=state, max_frames=mf)
        assert torch.equal(h, again)


@pytest.mark.parametrize("channels", [3, 65, 129, 257])
def test_scan_state_in_place_odd_widths(env, channels):
    """In place at widths where the last lanes, or the last workgroup, could
    share a channel with others: one row to a few per sequence, and sequences
    long enough for a workgroup each."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    for n, rows in ((700, 1), (333, 9), (200, 200)):
        say(f"in place, {n} sequences of {rows} x {channels}")
        off = torch.arange(n + 1, device=dev) * rows
        gen = torch.Generator(device=dev).manual_seed(channels)
        x, g = (torch.randn((n * rows, channels), generator=gen, device=dev).half()
                for _ in range(2))
        state = torch.randn((n, channels), generator=gen, device=dev)
        apart = torch.empty_like(state)
        h = lm.logmel_gated_scan(plan, x, g, off, state=state, state_out=apart, max_frames=rows)
        for _ in range(3):
            kept = state.clone()
            h2 = lm.logmel_gated_scan(plan, x, g, off, state=kept, state_out=kept,
                                      max_frames=rows)
            assert torch.equal(h, h2) and torch.equal(apart, kept)


def test_scan_gradient_repeats_bit_for_bit(env):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    off = torch.tensor([0, 5000, 5001, 20000], device=dev)
    gen = torch.Generator(device=dev).manual_seed(2)
    x, g, dh = (torch.randn((20000, 257), generator=gen, device=dev).half() for _ in range(3))
    bias = torch.randn(257, generator=gen, device=dev)
    ck = torch.empty((lm.logmel_gated_scan_checkpoint_rows(20000), 257), device=dev)
    lm.logmel_gated_scan(plan, x, g, off, bias=bias, checkpoints=ck)
    first = lm.logmel_gated_scan_backward(plan, dh, x, g, off, ck, bias=bias)
    for _ in range(5):
        again = lm.logmel_gated_scan_backward(plan, dh, x, g, off, ck, bias=bias)
        assert all(torch.equal(a, b) for a, b in zip(first[:3], again[:3]))


def test_scan_offsets_past_2_31(env):
    """Row starts past 2^31 elements, in a column slice of a wide buffer."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    rows, width, c = 70000, 36000, 65
    say(f"{rows} rows {width} apart")
    wide = torch.empty((rows, width), dtype=torch.float16, device=dev)
    rng = np.random.default_rng(8)
    col = {}
    for i, k in enumerate(("x", "g", "dh", "h", "dx", "dg")):
        col[k] = wide[:, 1000 + 100 * i:1000 + 100 * i + c]
    gen = torch.Generator(device=dev).manual_seed(3)
    dense = {k: torch.randn((rows, c), generator=gen, device=dev).half() for k in ("x", "g", "dh")}
    for k, v in dense.items():
        col[k].copy_(v)
    off = torch.tensor([0, 69000, rows], device=dev)
    ck = torch.empty((lm.logmel_gated_scan_checkpoint_rows(rows), c), device=dev)
    lm.logmel_gated_scan(plan, col["x"], col["g"], off, out=col["h"], checkpoints=ck)
    lm.logmel_gated_scan_backward(plan, col["dh"], col["x"], col["g"], off, ck, dx=col["dx"],
                                  dgate=col["dg"])
    h = lm.logmel_gated_scan(plan, dense["x"], dense["g"], off, checkpoints=ck)
    dx, dg, _, _ = lm.logmel_gated_scan_backward(plan, dense["dh"], dense["x"], dense["g"], off,
                                                 ck)
    for a, b in ((col["h"], h), (col["dx"], dx), (col["dg"], dg)):
        assert torch.equal(a, b)
    y, z = lm.logmel_block_norm(plan, col["x"], h=col["h"], gate=col["g"], y=col["dx"],
                                z=col["dg"])
    y2, z2 = lm.logmel_block_norm(plan, dense["x"], h=h, gate=dense["g"])
    assert torch.equal(y, y2) and torch.equal(z, z2)
    del wide
    torch.cuda.empty_cache()


# -------------------------------------------------------------------- norm

def norm_case(env, dtype, rows, channels, layout, block=True, gate=True, params=True, dy=True,
              dz=True, eps=1e-6, seed=0, scale=1.0):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    mk = Rows(torch, dtype, rows, channels, layout, seed)

    def f32(mean):
        v = mk.rng.normal(size=channels) * 0.3 + mean
        return torch.from_numpy(v.astype(np.float32)).to(dev)

    res = mk.normal(scale)
    p = dict(h=mk.normal(scale) if block else None, gate=mk.normal(2.0) if block and gate else None,
             w_post=f32(1.0) if block and params else None,
             scale=f32(0.5) if block and params else None, w_pre=f32(1.0) if params else None)
    up = dict(dy=mk.normal() if dy else None, dz=mk.normal() if dz else None)
    y, z = lm.logmel_block_norm(plan, res, eps=eps, y=mk.empty() if block else None, z=mk.empty(),
                                **p)
    got = lm.logmel_block_norm_backward(plan, res, eps=eps, dres=mk.empty(),
                                        dh=mk.empty() if block else None,
                                        dgate=mk.empty() if p["gate"] is not None else None,
                                        **p, **up)
    torch.cuda.synchronize()
    val, tol = rows_ref.norm(host(res), eps=eps, grad=True, dtype=dtype,
                             **{k: None if t is None else host(t) for k, t in {**p, **up}.items()})
    got = {k: t for k, t in {**got, "y": y, "z": z}.items() if t is not None}
    for k, t in got.items():
        check(t, val[k], tol[k], k)
    want = {"z", "dres"} | ({"y", "dh"} if block else set())
    if p["gate"] is not None:
        want.add("dgate")
    if params:
        want |= ({"dw_post", "dscale"} if block else set()) | ({"dw_pre"} if dz else set())
    assert set(got) == want


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["dense", "slice", "odd"])
@pytest.mark.parametrize("channels", [1, 2, 7, 64, 128, 321, 512, 1000, 1024, 2050])
def test_norm_widths(env, dtype, layout, channels):
    say(f"norm {dtype} {layout} {channels} channels")
    norm_case(env, dtype, 37, channels, layout, seed=channels)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("channels", [4096, 5001, 8191, 8192])
def test_norm_wide(env, dtype, channels):
    say(f"norm {dtype} {channels} channels")
    norm_case(env, dtype, 5, channels, "odd" if channels % 2 else "dense", seed=1)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 63, 1025, 9001])
def test_norm_rows(env, rows):
    say(f"norm {rows} rows")
    norm_case(env, "bfloat16", rows, 128, "slice", seed=rows)
    norm_case(env, "float32", rows, 65, "odd", seed=rows)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("block,gate,params,dy,dz", [
    (False, False, True, False, True), (False, False, False, True, True),
    (True, False, False, True, True), (True, True, False, True, False),
    (True, False, True, False, True), (True, True, True, False, True),
    (False, False, True, True, False)])
def test_norm_parts(env, dtype, block, gate, params, dy, dz):
    for channels in (96, 700):
        say(f"norm {dtype} {channels} block {block} gate {gate} params {params} dy {dy} dz {dz}")
        norm_case(env, dtype, 50, channels, "dense", block, gate, params, dy, dz, seed=2)


def test_norm_extremes(env):
    """Rows of zeros, tiny and large rows (their squares inside fp32), and a
    NaN row beside others; gates far out."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    for dtype in DTYPES:
        for scale in (1e-3, 3e4 if dtype == "float16" else 1e9):
            say(f"norm {dtype} scale {scale}")
            mk = Rows(torch, dtype, 9, 200, "dense", 3)
            res, h = mk.normal(), mk.normal(scale if dtype != "float16" else min(scale, 8000.0))
            h[4] = 0.0
            res[4] = 0.0
            y, z = lm.logmel_block_norm(plan, res, h=h)
            val, tol = rows_ref.norm(host(res), h=host(h), dtype=dtype)
            check(y, val["y"], tol["y"], "y")
            check(z, val["z"], tol["z"], "z")
            h2, res2 = h.clone(), res.clone()
            h2[2, 7] = float("nan")
            res2[6, 1] = float("inf")
            y2, z2 = lm.logmel_block_norm(plan, res2, h=h2)
            keep = [0, 1, 3, 4, 5, 7, 8]
            assert torch.equal(y2[keep], y[keep]) and torch.equal(z2[keep], z[keep])
            assert torch.isnan(y2[2]).all() and torch.isnan(z2[2]).all()
            g = h.clone()
            g[:, 0::4], g[:, 1::4] = float("-inf"), -float(torch.finfo(g.dtype).max)
            g[:, 2::4], g[:, 3::4] = 50.0, -50.0
            y3, _ = lm.logmel_block_norm(plan, res, h=mk.normal(), gate=g)
            # silu(-inf) is -inf * 0: not a number, as the formula; elsewhere finite
            assert torch.isfinite(y3[:, 1::4]).all() and torch.isfinite(y3[:, 2::4]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_without_eps(env, dtype):
    """eps 0, and rows that leave the last workgroup partly empty: the lanes
    without a row add nothing to the parameters' sums."""
    for channels in (64, 200, 700):
        for rows in (1, 5, 33):
            say(f"norm without eps {dtype} {rows} x {channels}")
            norm_case(env, dtype, rows, channels, "dense", eps=0.0, seed=rows)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_gates_far_out(env, dtype):
    """A gate at the type's lowest value, or far below 0, closes its channel:
    y is res there and the gradients of h and of the gate are 0; the others
    come out as without it. silu is below 1e-36 from -100 on down."""
    lm, plan, torch = env
    say(f"norm gates far out {dtype}")
    mk = Rows(torch, dtype, 40, 96, "dense", 4)
    res, h, gate, dy = mk.normal(), mk.normal(), mk.normal(2.0), mk.normal()
    low = float(torch.finfo(gate.dtype).min)
    gate[:, 3::4], gate[:, 1::4] = low, -100.0 if dtype != "float32" else -1e30
    gate[7] = low
    y, _ = lm.logmel_block_norm(plan, res, h=h, gate=gate)
    got = lm.logmel_block_norm_backward(plan, res, h=h, gate=gate, dy=dy)
    mid = host(gate).astype(np.float64)
    val, tol = rows_ref.norm(host(res), h=host(h), gate=np.maximum(mid, -100.0), dy=host(dy),
                             grad=True, dtype=dtype)
    for k, t in dict(y=y, **got).items():
        if t is not None:
            check(t, val[k], tol[k], k)
    for cols in (slice(3, None, 4), slice(1, None, 4)):
        assert torch.equal(y[:, cols], res[:, cols])
        assert np.abs(host(got["dgate"])[:, cols]).max() < 1e-30


def test_norm_gradient_repeats_bit_for_bit(env):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev).manual_seed(4)
    t = [torch.randn((6007, 300), generator=gen, device=dev).bfloat16() for _ in range(5)]
    w = [torch.randn(300, generator=gen, device=dev) for _ in range(3)]
    kw = dict(h=t[1], gate=t[2], w_post=w[0], scale=w[1], w_pre=w[2], dy=t[3], dz=t[4])
    first = lm.logmel_block_norm_backward(plan, t[0], **kw)
    for _ in range(5):
        again = lm.logmel_block_norm_backward(plan, t[0], **kw)
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_empty_calls(env):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    x = torch.empty((0, 8), device=dev)
    off = torch.zeros(4, dtype=torch.int64, device=dev)
    state = torch.randn((3, 8), device=dev)
    so = torch.zeros_like(state)
    bias = torch.ones(8, device=dev)
    ck = torch.empty((0, 8), device=dev)
    h = lm.logmel_gated_scan(plan, x, x, off, bias=bias, state=state, state_out=so, checkpoints=ck)
    assert h.shape == (0, 8) and torch.equal(so, state)
    up = torch.randn_like(state)
    dx, dg, db, ds = lm.logmel_gated_scan_backward(plan, x, x, x, off, ck, bias=bias, state=state,
                                                   dstate_out=up)
    assert dx.shape == (0, 8) and torch.equal(ds, up) and (db == 0).all()
    # rows, but no sequence
    y = torch.full((5, 8), 7.0, device=dev)
    none = torch.zeros(1, dtype=torch.int64, device=dev)
    ck = torch.empty((1, 8), device=dev)
    lm.logmel_gated_scan(plan, torch.ones_like(y), torch.ones_like(y), none, out=y)
    _, _, db, _ = lm.logmel_gated_scan_backward(plan, torch.ones_like(y), torch.ones_like(y),
                                                torch.ones_like(y), none, ck, bias=bias)
    assert (y == 7.0).all() and (db == 0).all()
    w = torch.ones(8, device=dev)
    _, z = lm.logmel_block_norm(plan, x, w_pre=w)
    g = lm.logmel_block_norm_backward(plan, x, w_pre=w, dz=x)
    assert z.shape == (0, 8) and (g["dw_pre"] == 0).all()


# ----------------------------------------------------- together, as they run

def _block(lm, plan, torch, rows, off, weights, state, state_out, max_frames, ck=None,
           stream=None):
    """One block over rows [rows, 128]: norm, products, scan, norm with gate
    and residual (the products are torch's)."""
    w_in, b, w_pre, w_post, scale, w_next = weights
    _, z = lm.logmel_block_norm(plan, rows, w_pre=w_pre, stream=stream)
    p = z @ w_in
    x, g, o = p[:, :128], p[:, 128:256], p[:, 256:]
    h = lm.logmel_gated_scan(plan, x, g, off, bias=b, state=state, state_out=state_out,
                             checkpoints=ck, max_frames=max_frames, stream=stream)
    y, z2 = lm.logmel_block_norm(plan, rows, h=h, gate=o, w_post=w_post, scale=scale,
                                 w_pre=w_next, stream=stream)
    return dict(z=z, x=x, g=g, o=o, h=h, y=y, z2=z2)


def _weights(torch, dtype, seed=0):
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device=dev)   # noqa: E731
    return ((r(128, 384) * 128 ** -0.5).to(dtype), r(128) + 1.0, 1.0 + 0.1 * r(128),
            1.0 + 0.1 * r(128), 0.3 + 0.1 * r(128), 1.0 + 0.1 * r(128))


def test_block_over_log_mel_rows(env):
    """Audio to log-mel rows to one block, in the library's own layout: each
    operator against its fp64 form on the inputs it was given, and the
    gradients back to the rows."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    lens = np.array([8000, 399, 31234, 400])
    audio, so = S.pack(lens, lambda i, v: S.speech_like(70 + i, int(lens[i]), "cuda", out=v),
                       "cuda")
    rows, fo = lm.log_mel(plan, audio, so)
    off = torch.from_numpy(fo).to(dev)
    w = _weights(torch, torch.float32)
    state = torch.randn((4, 128), device=dev)
    so_ = torch.empty_like(state)
    ck = torch.empty((lm.logmel_gated_scan_checkpoint_rows(len(rows)), 128), device=dev)
    t = _block(lm, plan, torch, rows, off, w, state, so_, int(np.diff(fo).max()), ck)
    val, tol = rows_ref.norm(host(rows), w_pre=host(w[2]))
    check(t["z"], val["z"], tol["z"], "z")
    val, tol = rows_ref.scan(host(t["x"]), host(t["g"]), fo, host(w[1]), host(state))
    check(t["h"], val["h"], tol["h"], "h")
    check(so_, val["state_out"], tol["state_out"], "state_out")
    dy, dz = torch.randn_like(rows), torch.randn_like(rows)
    kw = dict(h=t["h"], gate=t["o"], w_post=w[3], scale=w[4], w_pre=w[5])
    val, tol = rows_ref.norm(host(rows), grad=True, dy=host(dy), dz=host(dz),
                             **{k: host(v) for k, v in kw.items()})
    check(t["y"], val["y"], tol["y"], "y")
    check(t["z2"], val["z"], tol["z"], "z2")
    gr = lm.logmel_block_norm_backward(plan, rows, dy=dy, dz=dz, **kw)
    for k, v in gr.items():
        check(v, val[k], tol[k], k)
    dx, dg, db, ds = lm.logmel_gated_scan_backward(plan, gr["dh"], t["x"], t["g"], off, ck,
                                                   bias=w[1], state=state)
    val, tol = rows_ref.scan(host(t["x"]), host(t["g"]), fo, host(w[1]), host(state),
                             dh=host(gr["dh"]))
    for k, v in dict(dx=dx, dgate=dg, dbias=db, dstate=ds).items():
        check(v, val[k], tol[k], k)
    dz0 = torch.cat([dx, dg, gr["dgate"]], 1) @ w[0].t()
    first = lm.logmel_block_norm_backward(plan, rows, w_pre=w[2], dz=dz0)
    val, tol = rows_ref.norm(host(rows), w_pre=host(w[2]), dz=host(dz0), grad=True)
    check(first["dres"], val["dres"], tol["dres"], "dres")
    check(first["dw_pre"], val["dw_pre"], tol["dw_pre"], "dw_pre")


def test_block_over_stream_pushes(env):
    """512-frame streams in pushes of 80 ms: log-mel frames of each push, one
    block with its state carried, against the offline frames' block."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    n, pushes = 9, 6
    audio = torch.stack([S.speech_like(80 + j, 1280 * pushes, dev) for j in range(n)])
    w = _weights(torch, torch.float32, 1)
    s = lm.logmel_stream_create(plan, n, 1280)
    state = torch.zeros((n, 128), device=dev)
    parts = [[] for _ in range(n)]
    scans = [[] for _ in range(n)]
    for k in range(pushes):
        new = audio[:, 1280 * k:1280 * (k + 1)].contiguous().reshape(-1)
        rows, fo = lm.logmel_stream_push(s, new, [1280] * n)
        t = _block(lm, plan, torch, rows, torch.from_numpy(np.array(fo)).to(dev), w, state, state,
                   int(np.diff(fo).max()))
        for j in range(n):
            parts[j].append(rows[fo[j]:fo[j + 1]])
            scans[j].append(torch.stack([t[q][fo[j]:fo[j + 1]] for q in ("x", "g", "h")]))
    s.close()
    off_rows, fo = lm.log_mel(plan, audio.reshape(-1), np.arange(n + 1) * 1280 * pushes)
    assert torch.equal(off_rows, torch.cat([torch.cat(p) for p in parts]))
    for j in range(n):
        x, g, h = (host(v) for v in torch.cat(scans[j], 1))
        val, tol = rows_ref.scan(x, g, [0, len(x)], host(w[1]))
        assert (np.abs(h - val["h"]) <= tol["h"]).all()
        assert (np.abs(host(state[j]) - val["state_out"][0]) <= tol["state_out"][0]).all()


def test_block_in_a_graph(env):
    """Captured once (forward and gradients, long enough for several parts)
    and replayed with other inputs; each replay equals the eager calls, which
    run in between; a second graph alive beside it."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    off = torch.tensor([0, 3000, 3000, 3500, 9000], device=dev)
    w = _weights(torch, torch.bfloat16, 2)
    gen = torch.Generator(device=dev).manual_seed(9)
    rows, p, up = (torch.zeros((9000, k), dtype=torch.bfloat16, device=dev)
                   for k in (128, 384, 128))
    state = torch.zeros((4, 128), device=dev)

    def fill():
        for t in (rows, p, up):
            t.copy_(torch.randn(t.shape, generator=gen, device=dev))
        state.copy_(torch.randn(state.shape, generator=gen, device=dev))

    def calls():
        x, g, o = p[:, :128], p[:, 128:256], p[:, 256:]
        ck = torch.empty((lm.logmel_gated_scan_checkpoint_rows(9000), 128), device=dev)
        so = torch.empty_like(state)
        h = lm.logmel_gated_scan(plan, x, g, off, bias=w[1], state=state, state_out=so,
                                 checkpoints=ck)
        kw = dict(h=h, gate=o, w_post=w[3], scale=w[4], w_pre=w[5])
        y, z = lm.logmel_block_norm(plan, rows, **kw)
        gr = lm.logmel_block_norm_backward(plan, rows, dy=up, dz=up, **kw)
        back = lm.logmel_gated_scan_backward(plan, gr["dh"], x, g, off, ck, bias=w[1], state=state,
                                             dstate_out=so)
        return [h, so, y, z, *gr.values(), *back]

    fill()
    calls()
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        say(f"capture {i}")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = calls()
        graphs.append((graph, out))
    for rep in range(4):
        fill()
        want = [t.clone() for t in calls()]
        for i, (graph, out) in enumerate(graphs):
            say(f"replay {rep} of graph {i}")
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams_at_once(env):
    """The same calls on two HIP streams at once and on the default stream
    alone give the same bits."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    off = torch.tensor([0, 20000, 20000, 50000], device=dev)
    gen = torch.Generator(device=dev).manual_seed(10)
    ops = [[torch.randn((50000, 128), generator=gen, device=dev).half() for _ in range(3)]
           for _ in range(2)]
    ck_rows = lm.logmel_gated_scan_checkpoint_rows(50000)

    def calls(t, stream):
        x, g, d = t
        ck = torch.empty((ck_rows, 128), device=dev)
        h = lm.logmel_gated_scan(plan, x, g, off, checkpoints=ck, stream=stream)
        y, z = lm.logmel_block_norm(plan, x, h=h, gate=g, stream=stream)
        gr = lm.logmel_block_norm_backward(plan, x, h=h, gate=g, dy=d, dz=d, stream=stream)
        dx, dg, _, _ = lm.logmel_gated_scan_backward(plan, gr["dh"], x, g, off, ck, stream=stream)
        return [h, y, z, gr["dres"], gr["dh"], gr["dgate"], dx, dg], ck

    want = [calls(t, None)[0] for t in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in ops]
    for rep in range(3):
        say(f"both streams, {rep}")
        got = [calls(t, s) for t, s in zip(ops, streams)]
        torch.cuda.synchronize()
        for (outs, _), ref in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_validate_refuses_offsets(env, monkeypatch):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    monkeypatch.setenv("LOGMEL_VALIDATE", "1")
    x = torch.randn((10, 8), device=dev)
    ck = torch.zeros((1, 8), device=dev)
    for off, mf in (([1, 10], 0), ([0, 6, 5, 10], 0), ([0, 11], 0), ([0, 4, 10], 5)):
        off_d = torch.tensor(off, device=dev)
        out = torch.full_like(x, 7.0)
        with pytest.raises(lm.LogmelError) as e:
            lm.logmel_gated_scan(plan, x, x, off_d, out=out, max_frames=mf)
        assert e.value.status == lm.LOGMEL_ERR_INVALID_ARGUMENT
        with pytest.raises(lm.LogmelError):
            lm.logmel_gated_scan_backward(plan, x, x, x, off_d, ck, dx=out, max_frames=mf)
        torch.cuda.synchronize()
        assert (out == 7.0).all()
    lm.logmel_gated_scan(plan, x, x, torch.tensor([0, 4, 9], device=dev), max_frames=5)


def test_binding_refuses(env):
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    x = torch.zeros((4, 8), device=dev)
    off = torch.tensor([0, 4], device=dev)
    with pytest.raises(ValueError):
        lm.logmel_gated_scan(plan, x, x[:, :7], off)
    with pytest.raises(ValueError):
        lm.logmel_gated_scan(plan, x.t().contiguous().t(), x, off)
    with pytest.raises(ValueError):
        lm.logmel_gated_scan(plan, x[:1].expand(4, 8), x, off)
    with pytest.raises(TypeError):
        lm.logmel_gated_scan(plan, x, x.half(), off)
    with pytest.raises(TypeError):
        lm.logmel_gated_scan(plan, x, x, off.int())
    with pytest.raises(TypeError):
        lm.logmel_gated_scan(plan, x, x, off.cpu())
    with pytest.raises(ValueError):
        lm.logmel_gated_scan(plan, x, x, off, state=torch.zeros((2, 8), device=dev))
    with pytest.raises(ValueError):
        lm.logmel_gated_scan(plan, x, x, off, checkpoints=torch.zeros((2, 8), device=dev))
    with pytest.raises(lm.LogmelError):
        lm.logmel_gated_scan(plan, x, torch.zeros_like(x), off, out=x)
    with pytest.raises(lm.LogmelError):
        lm.logmel_block_norm(plan, x, gate=torch.zeros_like(x), want_y=False)
    with pytest.raises(lm.LogmelError):
        lm.logmel_block_norm(plan, x, want_z=False)
    with pytest.raises(lm.LogmelError):
        lm.logmel_block_norm_backward(plan, x)
    with pytest.raises(TypeError):
        lm.logmel_block_norm(plan, x, w_pre=torch.ones(8, device=dev).half())


def test_rows_past_2_31(env):
    """More than 2^31 rows of one channel: states by the closed form of a
    constant gate (a = 1/2, x = 1: h_t = 1 - 2^-(t+1) from a sequence's first
    row), gradients by that of a constant dh, and the norm of one channel."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    first = 2 ** 31 + 77
    rows = first + 1001
    say(f"{rows} rows x 1")
    off = torch.tensor([0, first, rows], device=dev)
    x = torch.ones((rows, 1), dtype=torch.float16, device=dev)
    g = torch.zeros((rows, 1), dtype=torch.float16, device=dev)
    ck = torch.empty((lm.logmel_gated_scan_checkpoint_rows(rows), 1), device=dev)
    so = torch.empty((2, 1), device=dev)
    h = lm.logmel_gated_scan(plan, x, g, off, state_out=so, checkpoints=ck)
    # exact: every h is a multiple of 2^-11 or rounds to 1
    t = torch.arange(40, device=dev).double()
    want = (1.0 - 0.5 ** (t + 1)).half().unsqueeze(1)
    for start in (0, first):
        assert torch.equal(h[start:start + 40], want)
    assert (h[40:first] == 1.0).all() and (h[first + 40:] == 1.0).all()
    assert torch.equal(so, torch.ones_like(so))
    say("gradient")
    dx, dg, _, _ = lm.logmel_gated_scan_backward(plan, x, x, g, off, ck)
    # D_t = 2 - 2^-(last - t): dx = D / 2; dg = (h_{t-1} - 1) D / 4
    for start, end in ((0, first), (first, rows)):
        assert torch.equal(dx[end - 40:end].flip(0), want)
        assert (dx[start:end - 40] == 1.0).all()
        head = (-(0.5 ** t) * 2.0 / 4.0).half().unsqueeze(1)
        assert torch.allclose(dg[start:start + 20], head[:20], rtol=2.0 ** -10, atol=0.0)
    del dx, dg, ck
    say("norm")
    _, z = lm.logmel_block_norm(plan, x, eps=0.0)
    assert (z == 1.0).all()
    del h, z, x, g
    torch.cuda.empty_cache()
