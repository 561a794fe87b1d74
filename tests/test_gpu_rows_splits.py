"""The row operators on the GPU where the work is split otherwise than in small
calls: a workgroup per sequence, gradients included, norms whose resident
workgroups walk several rows, and what NaN and infinities reach in the
gradients."""

import numpy as np
import pytest

from tests import rows_ref
from tests.test_gpu_rows import DTYPES, Rows, check, env, host, norm_case, say   # noqa: F401

pytestmark = pytest.mark.gpu


def lengths(n, seed):
    """n sequences of few different lengths, empty ones, single rows and whole
    tiles of 128 among them; the longest twice the mean at most."""
    p = [0.03, 0.03, 0.1, 0.24, 0.3, 0.3]
    out = np.random.default_rng(seed).choice([0, 1, 129, 256, 513, 700], size=n, p=p)
    out[n // 2], out[n // 3] = 0, 1
    return out


def by_length(x, g, lens, off, bias, state, dh, dstate_out, dtype):
    """rows_ref.scan with the sequences of one length side by side as channels
    of one sequence."""
    n, c = len(lens), x.shape[1]
    rows = ("h", "dx", "dgate")
    per_seq = ("state_out", "dstate")
    val = {k: np.zeros(x.shape) for k in rows}
    val.update({k: np.zeros((n, c)) for k in per_seq}, dbias=np.zeros(c))
    tol = {k: v.copy() for k, v in val.items()}
    total = np.zeros(c)
    for length in np.unique(lens):
        seqs = np.flatnonzero(lens == length)
        at = off[seqs][:, None] + np.arange(length)      # [sequences][rows]

        def side(a):
            return a[at].transpose(1, 0, 2).reshape(length, len(seqs) * c)

        v, t = rows_ref.scan(side(x), side(g), [0, length], np.tile(bias, len(seqs)),
                             state[seqs].reshape(1, -1), side(dh),
                             dstate_out[seqs].reshape(1, -1), dtype)
        for k in rows:
            for out, got in ((val, v), (tol, t)):
                out[k][at] = got[k].reshape(length, len(seqs), c).transpose(1, 0, 2)
        for k in per_seq:
            for out, got in ((val, v), (tol, t)):
                out[k][seqs] = got[k].reshape(len(seqs), c)
        # a sequence's bound counts a rounding a row, of which the 16 rows
        # summed in fp32 have no more; sequences are joined in fp64
        val["dbias"] += v["dbias"].reshape(-1, c).sum(0)
        tol["dbias"] += t["dbias"].reshape(-1, c).sum(0)
        total += np.abs(v["dgate"]).sum(0).reshape(-1, c).sum(0)
    # sums of fewer than 16 rows, and the result, are rounded too
    tol["dbias"] += 16 * rows_ref.U * total
    return val, tol


# Widths of one channel per lane (64, and 129 and 130 forward), of two (512;
# 193 with a ragged slab) and, in the gradient, of two with the row's last
# channel in a slab of its own (257, 385).
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,channels", [(170, 64), (85, 129), (85, 130), (128, 193), (64, 257),
                                        (64, 385), (64, 512)])
def test_scan_by_sequences(env, dtype, n, channels):
    """Enough long sequences that each has a workgroup to itself (two slabs and
    more: several), in both directions."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say(f"scan by sequences {dtype} {n} x {channels}")
    lens = lengths(n, n)
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    rows = int(off[-1]) + 3
    mk = Rows(torch, dtype, rows, channels, "slice" if channels % 2 else "dense", channels)
    x, g, dh, h, dx, dg = mk.normal(), mk.normal(2.0), mk.normal(), mk.empty(), mk.empty(), \
        mk.empty()

    def f32(*shape):
        return torch.from_numpy(mk.rng.normal(size=shape).astype(np.float32)).to(dev)

    bias, state, dso = f32(channels) + 1.0, f32(n, channels), f32(n, channels)
    so, off_d = torch.empty_like(state), torch.from_numpy(off).to(dev)
    ck = torch.full((lm.logmel_gated_scan_checkpoint_rows(rows), channels), float("nan"),
                    device=dev)
    mf = int(lens.max())
    # the split this test is for: forward without workspace (one lane each
    # would take 140 us for the longest), the gradient with a bias sum of
    # doubles per sequence and nothing else
    inp = lm._scan_input(plan, x, g, off_d, bias, state, mf)
    assert lm._gated_scan_workspace(plan.handle, inp, 0) == 0
    assert lm._gated_scan_workspace(plan.handle, inp, 1) == n * channels * 8
    lm.logmel_gated_scan(plan, x, g, off_d, bias=bias, state=state, out=h, state_out=so,
                         checkpoints=ck, max_frames=mf)
    _, _, db, ds = lm.logmel_gated_scan_backward(plan, dh, x, g, off_d, ck, bias=bias, state=state,
                                                 dstate_out=dso, dx=dx, dgate=dg, max_frames=mf)
    val, tol = by_length(host(x), host(g), lens, off, host(bias), host(state), host(dh), host(dso),
                         dtype)
    last = int(off[-1])
    for k, t in dict(h=h, dx=dx, dgate=dg).items():
        check(t[:last], val[k][:last], tol[k][:last], k)
        assert (t[last:] == 7.0).all(), k
    for k, t in dict(state_out=so, dbias=db, dstate=ds).items():
        check(t, val[k], tol[k], k)


# Rows of two to four times what the resident workgroups hold at once, for
# rows of part of a wavefront, of one, and of several that meet in LDS.
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,channels", [(45001, 128), (30011, 321), (12001, 512), (6001, 1000),
                                           (2003, 4096), (901, 8192)])
def test_norm_many_rows(env, dtype, rows, channels):
    say(f"norm {dtype} {rows} x {channels}")
    norm_case(env, dtype, rows, channels, "odd" if channels % 2 else "dense", seed=rows)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("channels", [6, 128, 321, 1000, 2050, 4100, 8192])
def test_norm_parameter_sums_of_many_rows_a_lane(env, dtype, channels):
    """34 rows and more for each resident lane, summed 16 at a time. A term is
    the product of three values, of which the inverse root is off by the 28
    roundings of rows_ref; the sums add 9, and one each for the workgroup's
    part and the result."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    # a row takes 16 to 1024 lanes of 4 (2-byte rows: 8) values, four
    # wavefronts of them are resident per SIMD
    lanes = 16
    while lanes * (4 if dtype == "float32" else 8) < channels and lanes < 1024:
        lanes *= 2
    rows = 34 * (4 * 4 * 64 * 256 // lanes) + 5
    say(f"norm sums {dtype} {rows} x {channels}")
    gen = torch.Generator(device=dev).manual_seed(channels)
    v, up = (torch.randn((rows, channels), generator=gen, device=dev).to(getattr(torch, dtype))
             for _ in range(2))
    one = torch.ones(channels, device=dev)
    p = v.double()
    p *= up.double() / (p.square().mean(1, keepdim=True) + 1e-6).sqrt()
    want, bound = p.sum(0), (28 + 3 + 9 + 2) * rows_ref.U * p.abs().sum(0)
    del p
    got = lm.logmel_block_norm_backward(plan, v, w_pre=one, dz=up)["dw_pre"]
    assert ((got.double() - want).abs() <= bound).all()
    got = lm.logmel_block_norm_backward(plan, v, h=v, scale=one, w_post=one, dy=up)
    for k in ("dscale", "dw_post"):
        assert ((got[k].double() - want).abs() <= bound).all(), k


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("channels", [7, 200, 1000])
def test_norm_gradient_of_small_and_large_rows(env, dtype, channels):
    """Rows whose squares are near fp32's smallest and largest normal numbers
    (fp16: near the type's)."""
    for scale in (1e-3, 4e3) if dtype == "float16" else (1e-18, 1e16):
        say(f"norm gradient {dtype} {channels} rows near {scale}")
        norm_case(env, dtype, 23, channels, "dense", eps=0.0, seed=8, scale=scale)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("block,gate,params,dy,dz", [
    (False, False, True, False, True), (False, False, False, True, False),
    (True, False, True, True, False), (True, True, False, True, True),
    (True, True, True, True, False), (True, True, True, True, True)])
def test_norm_parts_of_rows_below_16_bytes(env, dtype, block, gate, params, dy, dz):
    """Rows of one value per lane, with several rows per lane."""
    for channels in (1, 3, 5, 7, 8):
        say(f"norm {dtype} {channels} block {block} gate {gate} params {params} dy {dy} dz {dz}")
        norm_case(env, dtype, 20001 if channels == 3 else 65, channels, "odd", block, gate, params,
                  dy, dz, seed=channels)


def test_norm_gradients_in_a_graph(env):
    """With and without dz, of the narrowest and the widest rows (whose sums
    take most of a compute unit's LDS), captured together and replayed with
    other inputs between eager calls."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev).manual_seed(12)
    sets = [[torch.zeros(rows, c, dtype=dt, device=dev) for _ in range(5)]
            for rows, c, dt in ((50000, 3, torch.float32), (700, 8192, torch.float32),
                                (5000, 8192, torch.bfloat16))]

    def fill():
        for ops in sets:
            for t in ops:
                t.copy_(torch.randn(t.shape, generator=gen, device=dev))

    def calls():
        out = []
        for res, h, gate, dy, dz in sets:
            w = torch.ones(res.shape[1], device=dev)
            kw = dict(h=h, gate=gate, w_post=w, scale=w)
            for up in (dict(w_pre=w, dy=dy, dz=dz), dict(dy=dy)):
                out += [t for t in lm.logmel_block_norm_backward(plan, res, **kw, **up).values()
                        if t is not None]
        return out

    fill()
    calls()
    torch.cuda.synchronize()
    say("capture")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    for rep in range(4):
        say(f"replay {rep}")
        fill()
        want = calls()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


# Sequences, channels and hint of a call in parts, and of one by sequences.
REACH = {"parts": ([300, 0, 5000, 70, 2500], 40, 0),
         "sequences": (lengths(85, 85).tolist(), 130, 700)}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("split", sorted(REACH))
@pytest.mark.parametrize("where", ["x", "gate", "dh"])
def test_scan_gradient_keeps_non_finite_values_in_place(env, dtype, split, where):
    """A NaN and an infinity reach the rows of their own sequence and channel
    that depend on them, and nothing else changes by a bit: x and gate the
    later rows' h, dh and gate the earlier rows' gradients."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say(f"non-finite {where} {split} {dtype}")
    lens, channels, mf = REACH[split]
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    n, rows = len(lens), int(off[-1])
    mk = Rows(torch, dtype, rows, channels, "dense", 9)
    ops = dict(x=mk.normal(), gate=mk.normal(2.0), dh=mk.normal())
    off_d = torch.from_numpy(off).to(dev)
    state = torch.randn((n, channels), device=dev)
    bias = torch.randn(channels, device=dev)

    def calls(x, gate, dh):
        ck = torch.empty((lm.logmel_gated_scan_checkpoint_rows(rows), channels), device=dev)
        h = lm.logmel_gated_scan(plan, x, gate, off_d, bias=bias, state=state, checkpoints=ck,
                                 max_frames=mf)
        inp = lm._scan_input(plan, x, gate, off_d, bias, state, mf)
        need = lm._gated_scan_workspace(plan.handle, inp, 1)
        assert (need == n * channels * 8) == (split == "sequences")
        dx, dg, db, ds = lm.logmel_gated_scan_backward(plan, dh, x, gate, off_d, ck, bias=bias,
                                                       state=state, max_frames=mf)
        return dict(h=h, dx=dx, dgate=dg, dbias=db, dstate=ds)

    clean = calls(**ops)
    long = [j for j in range(n) if lens[j] > 250]
    spots = [(long[0], 0, 0), (long[1], 200, 3), (long[-1], lens[long[-1]] - 1, 5),
             (long[-1], 130, channels - 1)]
    hit = ops[where].clone()
    reach = {k: torch.zeros((rows, channels), dtype=torch.bool) for k in ("h", "dx", "dgate")}
    reach.update(dbias=torch.zeros(channels, dtype=torch.bool),
                 dstate=torch.zeros((n, channels), dtype=torch.bool))
    for i, (j, t, c) in enumerate(spots):
        s, e = int(off[j]), int(off[j + 1])
        # a gate at infinity is an ordinary gate
        hit[s + t, c] = float("nan") if where == "gate" or i % 2 else float("inf")
        later, earlier = slice(s + t, e), slice(s, s + t + 1)
        if where != "dh":
            reach["h"][later, c] = reach["dgate"][later, c] = True
        if where != "x":
            reach["dx"][earlier, c] = reach["dgate"][earlier, c] = True
            reach["dstate"][j, c] = True
        reach["dbias"][c] = True
    got = calls(**{**ops, where: hit})
    for k, t in got.items():
        same = ~reach[k].to(dev)
        assert torch.equal(t[same], clean[k][same]), k
        # (where a product with 0 could give 0, NaN: none, the gates are near 0)
        assert not torch.isfinite(t[~same]).any(), k
