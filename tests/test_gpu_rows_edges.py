"""The row operators on the GPU at their edges: values and calls beside the
sizes and layouts of test_gpu_rows.py."""

import numpy as np
import pytest

from tests import rows_ref
from tests.test_gpu_rows import DTYPES, Rows, check, env, host, say   # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 8, 300, 4000])
def test_scan_closed_gate_leaves_nothing_of_a_large_state(env, dtype, rows):
    """States are fp32 whatever the rows' type: a gate at the type's lowest
    value closes behind a state near fp32's largest, in the gradient too, and
    of an infinite one leaves 0 times infinity."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    say(f"scan closes behind a large state {dtype} {rows} rows")
    dt = getattr(torch, dtype)
    rng = np.random.default_rng(rows)
    x, g, dh = (torch.from_numpy(rng.normal(size=(rows + 1, 64))).to(dt).to(dev)
                for _ in range(3))
    g[0] = g[rows] = float(torch.finfo(dt).min)
    off = np.array([0, rows, rows + 1])
    off_d = torch.from_numpy(off).to(dev)
    state = torch.full((2, 64), 3e38, device=dev)
    state[:, 1::2] = -3e38
    dso = torch.zeros((2, 64), device=dev)
    dso[1] = 3e38
    state_out = torch.empty_like(state)
    ck = torch.empty((lm.logmel_gated_scan_checkpoint_rows(rows + 1), 64), device=dev)
    h = lm.logmel_gated_scan(plan, x, g, off_d, state=state, state_out=state_out, checkpoints=ck)
    dx, dg, _, ds = lm.logmel_gated_scan_backward(plan, dh, x, g, off_d, ck, state=state,
                                                  dstate_out=dso)
    # the recurrence from a state of 0; what a gate beyond -60 leaves of its
    # rows is below 1e-20
    val, tol = rows_ref.scan(host(x), np.maximum(host(g), -60.0), off, dh=host(dh), dtype=dtype)
    check(h, val["h"], tol["h"] + 1e-20, "h")
    check(state_out, val["state_out"], tol["state_out"] + 1e-20, "state_out")
    check(dx[:rows], val["dx"][:rows], tol["dx"][:rows] + 1e-20, "dx")
    check(dg, np.where(np.isin(np.arange(rows + 1), (0, rows))[:, None], 0.0, val["dgate"]),
          tol["dgate"] + 1e-20, "dgate")
    assert (ds == 0.0).all()
    h = lm.logmel_gated_scan(plan, x, g, off_d, state=torch.full_like(state, float("inf")))
    assert torch.isnan(h).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("block,gate", [(False, False), (True, False), (True, True)])
def test_norm_gradient_without_dz_is_independent_of_y(env, dtype, block, gate):
    """Without dz, y's gradient is dy as it is, and no output depends on res
    or w_pre: infinities and NaN there change nothing."""
    lm, plan, torch = env
    for channels in (5, 96, 700, 2050):
        say(f"norm gradient of dy alone {dtype} block {block} gate {gate} {channels}")
        mk = Rows(torch, dtype, 70, channels, "odd", 6)
        res, dy = mk.normal(), mk.normal()
        kw = dict(dy=dy)
        if block:
            kw.update(h=mk.normal(), w_post=torch.full((channels,), 1.25, device=res.device),
                      scale=torch.full((channels,), 0.5, device=res.device))
        if gate:
            kw.update(gate=mk.normal(2.0))
        want = lm.logmel_block_norm_backward(plan, res, **kw)
        assert torch.equal(want["dres"], dy)
        res2 = res.clone()
        res2[3, 1], res2[9, 0], res2[66, channels - 1] = float("inf"), float("nan"), -float("inf")
        w_pre = torch.full((channels,), float("inf"), device=res.device)
        got = lm.logmel_block_norm_backward(plan, res2, w_pre=w_pre, **kw)
        for k, t in want.items():
            assert (got[k] is None) if t is None else torch.equal(got[k], t), k


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("scale", [1e-20, 3e-21])
def test_norm_of_rows_with_subnormal_mean_square(env, dtype, scale):
    """eps 0 and rows whose squares are subnormal: their mean square has fewer
    digits, and the norm and its gradient as many."""
    lm, plan, torch = env
    for channels in (64, 321, 2050):
        say(f"norm of rows near {scale} {dtype} {channels}")
        mk = Rows(torch, dtype, 33, channels, "dense", 7)
        res, h, gate = mk.normal(scale), mk.normal(scale), mk.normal(2.0)
        dz, up = mk.normal(), mk.normal()
        y, z = lm.logmel_block_norm(plan, res, eps=0.0)
        assert y is None
        got = lm.logmel_block_norm_backward(plan, res, eps=0.0, dz=dz)
        val, tol = rows_ref.norm(host(res), eps=0.0, dz=host(dz), grad=True, dtype=dtype)
        # each of at most 2 channels + 2 roundings of the mean square is half
        # a subnormal step, 2^-150; the root halves what that is of it, and
        # the gradient has the root three times (and the mean of dz y, whose
        # terms are near 1)
        def lost(rows):
            ms = (host(rows) ** 2).mean(1, keepdims=True)
            return (2 * channels + 2) * 2.0 ** -150 / channels / ms + 2.0 ** -150 / ms

        e = lost(res)
        check(z, val["z"], tol["z"] + e * np.abs(val["z"]), "z")
        r2 = 1.0 / np.sqrt((host(res) ** 2).mean(1, keepdims=True))
        parts = np.abs(r2 * host(dz)) + np.abs(host(res)) * r2 ** 3 * np.abs(
            (host(dz) * host(res)).mean(1, keepdims=True))
        check(got["dres"], val["dres"], tol["dres"] + 3 * e * parts, "dres")
        # a block's h of that size: t is of the size of 1 whatever h's is
        one = mk.normal()
        y, z = lm.logmel_block_norm(plan, one, h=h, gate=gate, eps=0.0)
        val, tol = rows_ref.norm(host(one), h=host(h), gate=host(gate), eps=0.0, dtype=dtype)
        e = lost(h)
        t = np.abs(val["y"] - host(one))
        check(y, val["y"], tol["y"] + e * t, "y")
        assert torch.isfinite(z).all()
        got = lm.logmel_block_norm_backward(plan, one, h=h, gate=gate, eps=0.0, dy=up)
        val, tol = rows_ref.norm(host(one), h=host(h), gate=host(gate), eps=0.0, dy=host(up),
                                 grad=True, dtype=dtype)
        check(got["dgate"], val["dgate"], tol["dgate"] + e * np.abs(val["dgate"]), "dgate")
        o = host(gate)
        q = np.abs(host(up) * o * rows_ref.sigmoid(o))
        r1 = 1.0 / np.sqrt((host(h) ** 2).mean(1, keepdims=True))
        parts = r1 * q + np.abs(host(h)) * r1 ** 3 * (q * np.abs(host(h))).mean(1, keepdims=True)
        check(got["dh"], val["dh"], tol["dh"] + 3 * e * parts, "dh")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_norm_parameter_sums_over_millions_of_rows(env, dtype):
    """The gradients of the parameters over 2^22 rows of equal values, whose
    sums in fp32 drift by one rounding a row. Rows of ones have a mean square
    of 1 and give dy and dz themselves as terms; a sum of up to 16 of them in
    fp32 is off by at most half of 16 roundings and some, (16 + 2) / 2 2^-24,
    the part of a workgroup and the result by one each."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    rows, channels = 2 ** 22, 64 if dtype == "float32" else 128
    say(f"norm sums {dtype} {rows} x {channels}")
    ones = torch.ones((rows, channels), dtype=getattr(torch, dtype), device=dev)
    # 0.7 and 1.1 in fp32; in bf16 the parameter carries the digits
    up = torch.full_like(ones, 0.7)
    w = torch.full((channels,), 1.0, device=dev)
    got = lm.logmel_block_norm_backward(plan, ones, w_pre=w, eps=0.0, dz=up)
    want = rows * float(up[0, 0])
    bound = (9 + 2) * 2.0 ** -24 * want
    assert (got["dw_pre"].double() - want).abs().max() <= bound
    del got
    # t = 1 + 2^-12: a term of fp32 digits out of 2-byte rows needs the gate,
    # whose silu is the same in every row; the sum of one row tells it
    gate = torch.full_like(ones, 1.5)
    kw = dict(w_post=w, scale=w, eps=0.0)
    one = lm.logmel_block_norm_backward(plan, ones[:1], h=ones[:1], gate=gate[:1], dy=up[:1], **kw)
    got = lm.logmel_block_norm_backward(plan, ones, h=ones, gate=gate, dy=up, **kw)
    for k in ("dw_post", "dscale"):
        term = one[k].double()
        assert ((got[k].double() - rows * term).abs() <= (9 + 3) * 2.0 ** -24 * rows * term).all()


def test_binding_refuses_to_lose_a_graph(env):
    """The calls record nothing for torch's autograd: an operand that asks for
    a gradient while graphs are recorded is refused, and runs where they are
    not."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    x, g, dh = (torch.randn((6, 8), device=dev) for _ in range(3))
    w = torch.nn.Parameter(torch.randn(8, device=dev))
    leaf = x.clone().requires_grad_()
    off = torch.tensor([0, 6], device=dev)
    ck = torch.empty((1, 8), device=dev)
    state = torch.zeros((1, 8), device=dev)

    def calls(x, g, dh, w, state):
        yield lambda: lm.logmel_gated_scan(plan, x, g, off, bias=w, state=state, checkpoints=ck)
        yield lambda: lm.logmel_gated_scan_backward(plan, dh, x, g, off, ck, bias=w, state=state)[0]
        yield lambda: lm.logmel_block_norm(plan, x, h=g, w_pre=w)[1]
        yield lambda: lm.logmel_block_norm_backward(plan, x, h=g, w_pre=w, dz=dh)["dh"]

    plain = [c() for c in calls(x, g, dh, w.detach(), state)]
    for args in ((leaf, g, dh, w.detach(), state), (x, leaf, dh, w.detach(), state),
                 (x, g, dh, w, state)):
        for c in calls(*args):
            with pytest.raises(RuntimeError, match="autograd"):
                c()
        with torch.no_grad():
            got = [c() for c in calls(*args)]
        if args[0] is x and args[1] is g:
            assert all(torch.equal(a, b) for a, b in zip(got, plain))
    with pytest.raises(RuntimeError, match="autograd"):
        lm.logmel_gated_scan(plan, x, g, off, out=torch.empty_like(x).requires_grad_())
    with pytest.raises(RuntimeError, match="autograd"):
        lm.logmel_gated_scan(plan, x, g, off, state=state.clone().requires_grad_())
    with pytest.raises(RuntimeError, match="autograd"):
        lm.logmel_block_norm_backward(plan, x, dz=leaf)

    class Scan(torch.autograd.Function):
        """The two calls as one differentiable function: no graph is recorded
        inside it."""

        @staticmethod
        def forward(ctx, x, g, b):
            ck = torch.empty((1, 8), device=dev)
            ctx.save_for_backward(x, g, b, ck)
            return lm.logmel_gated_scan(plan, x, g, off, bias=b, checkpoints=ck)

        @staticmethod
        def backward(ctx, dh):
            x, g, b, ck = ctx.saved_tensors
            return lm.logmel_gated_scan_backward(plan, dh, x, g, off, ck, bias=b)[:3]

    Scan.apply(leaf, g, w).backward(dh)
    want = lm.logmel_gated_scan_backward(plan, dh, x, g, off, ck, bias=w.detach())
    assert torch.equal(leaf.grad, want[0]) and torch.equal(w.grad, want[2])


def test_scan_gradient_of_the_state_without_a_state(env):
    """want_dstate asks for the initial state's gradient where the state is
    left out (0), or leaves it out where there is one."""
    lm, plan, torch = env
    dev = torch.device("cuda", 0)
    off = torch.tensor([0, 300, 300, 411], device=dev)
    x, g, dh = (torch.randn((411, 66), device=dev) for _ in range(3))
    zero = torch.zeros((3, 66), device=dev)
    ck = torch.empty((4, 66), device=dev)
    lm.logmel_gated_scan(plan, x, g, off, checkpoints=ck)
    call = lm.logmel_gated_scan_backward
    want = call(plan, dh, x, g, off, ck, state=zero)
    got = call(plan, dh, x, g, off, ck, want_dstate=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(got[3], want[3])
    _, tol = rows_ref.scan(host(x), host(g), host(off).astype(int), dh=host(dh))
    val, _ = rows_ref.scan(host(x), host(g), host(off).astype(int), dh=host(dh))
    check(got[3], val["dstate"], tol["dstate"], "dstate")
    assert call(plan, dh, x, g, off, ck)[3] is None
    assert call(plan, dh, x, g, off, ck, state=zero, want_dstate=False)[3] is None
