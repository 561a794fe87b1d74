"""The row operators without a GPU: the fp64 forms they are tested against
(closed forms, differences), and the calls that are refused on the host before
any launch."""

import ctypes

import numpy as np
import pytest

from tests import rows_ref
from tests.libload import load_binding


@pytest.fixture(scope="module")
def lm():
    lm = load_binding()
    assert ctypes.sizeof(lm.logmel_config) == 48   # the fake plan's first field
    return lm


# ------------------------------------------------------------ the fp64 forms

def test_scan_form_constant_gate():
    # a constant, x = 1: h_t = 1 - a^(t + 1)
    g = np.full((50, 1), 1.25)
    val, _ = rows_ref.scan(np.ones((50, 1)), g, [0, 50])
    a = 1.0 / (1.0 + np.exp(-1.25))
    assert np.allclose(val["h"][:, 0], 1.0 - a ** np.arange(1, 51), atol=1e-14)


def test_scan_form_gradient_by_differences():
    rng = np.random.default_rng(3)
    off = np.array([0, 7, 7, 8, 20])
    rows, c, n = 20, 3, 4
    p = dict(x=rng.normal(size=(rows, c)), g=rng.normal(size=(rows, c)) * 2,
             bias=rng.normal(size=c), state=rng.normal(size=(n, c)))
    dh, ds = rng.normal(size=(rows, c)), rng.normal(size=(n, c))

    def loss():
        v, _ = rows_ref.scan(p["x"], p["g"], off, p["bias"], p["state"])
        return (v["h"] * dh).sum() + (v["state_out"] * ds).sum()

    val, _ = rows_ref.scan(p["x"], p["g"], off, p["bias"], p["state"], dh, ds)
    names = dict(x="dx", g="dgate", bias="dbias", state="dstate")
    for key, name in names.items():
        _differences(p[key], loss, val[name])


def test_norm_form_gradient_by_differences():
    rng = np.random.default_rng(4)
    rows, c = 3, 5
    p = dict(res=rng.normal(size=(rows, c)), h=rng.normal(size=(rows, c)),
             gate=rng.normal(size=(rows, c)), w_post=rng.normal(size=c),
             scale=rng.normal(size=c), w_pre=rng.normal(size=c))
    dy, dz = rng.normal(size=(rows, c)), rng.normal(size=(rows, c))

    def loss():
        v, _ = rows_ref.norm(eps=1e-3, **p)
        return (v["y"] * dy).sum() + (v["z"] * dz).sum()

    val, _ = rows_ref.norm(eps=1e-3, dy=dy, dz=dz, grad=True, **p)
    names = dict(res="dres", h="dh", gate="dgate", w_post="dw_post", scale="dscale",
                 w_pre="dw_pre")
    for key, name in names.items():
        _differences(p[key], loss, val[name])


def _differences(array, loss, grad):
    step = 1e-5   # truncation ~ step^2, rounding ~ 1e-16 * loss / step
    for i in np.ndindex(array.shape):
        keep = array[i]
        array[i] = keep + step
        up = loss()
        array[i] = keep - step
        down = loss()
        array[i] = keep
        assert abs((up - down) / (2 * step) - grad[i]) <= 1e-7 * (1 + np.abs(grad).max())


# ------------------------------------------------------------ refused calls

# A plan for the checks, which come before anything that uses the device: its
# memory reads as a plan on device 0 of 256 compute units. Never passed to a
# call that is accepted.
class _FakePlan(ctypes.Structure):
    _fields_ = [("cfg", ctypes.c_char * 48), ("tables", ctypes.c_void_p),
                ("resident_waves", ctypes.c_int)]


FAKE_PLAN = _FakePlan(resident_waves=4 * 256)
FAKE = ctypes.c_void_p(ctypes.addressof(FAKE_PLAN))


def _scan_in(lm, **kw):
    d = dict(type=lm.LOGMEL_F32, rows=10, channels=8, n_seq=2, d_seq_offsets=0x1000, max_frames=0,
             d_x=0x100000, x_stride=8, d_gate=0x110000, gate_stride=8, d_bias=None, d_state=None)
    d.update(kw)
    return lm.logmel_scan_input(**d)


def _scan(lm, inp, h=0x200000, hs=8, so=None, ck=None, ws=0x400000, wsb=1 << 30):
    return lm._gated_scan(FAKE, inp, h, hs, so, ck, ws, wsb, None)


_BAD = dict(
    rows=dict(rows=-1), channels=dict(channels=0), n_seq=dict(n_seq=-1),
    offsets_null=dict(d_seq_offsets=None), offsets_odd=dict(d_seq_offsets=0x1004),
    max_frames=dict(max_frames=-1), x_null=dict(d_x=None), x_odd=dict(d_x=0x100002),
    x_stride=dict(x_stride=7), gate_null=dict(d_gate=None), gate_stride=dict(gate_stride=0),
    bias_odd=dict(d_bias=0x1001), state_odd=dict(d_state=0x1002))


@pytest.mark.parametrize("name", sorted(_BAD))
def test_scan_refuses_bad_inputs(lm, name):
    inp = _scan_in(lm, **_BAD[name])
    assert _scan(lm, inp) == lm.LOGMEL_ERR_INVALID_ARGUMENT
    grad = lm.logmel_scan_grad(0x300000, 8, None, 0x310000, 8, 0x320000, 8, None, None)
    assert lm._gated_scan_backward(FAKE, inp, 0x500000, grad, 0x400000, 1 << 30,
                                   None) == lm.LOGMEL_ERR_INVALID_ARGUMENT
    assert lm._gated_scan_workspace(FAKE, inp, 0) == -1


def test_scan_refuses_types_and_lengths(lm):
    assert _scan(lm, _scan_in(lm, type=lm.LOGMEL_I16)) == lm.LOGMEL_ERR_UNSUPPORTED
    assert _scan(lm, _scan_in(lm, type=9)) == lm.LOGMEL_ERR_UNSUPPORTED
    big = 1 << 61
    assert _scan(lm, _scan_in(lm, rows=1 << 40, x_stride=big)) == lm.LOGMEL_ERR_INPUT_TOO_LONG
    assert _scan(lm, _scan_in(lm, channels=1 << 61, x_stride=1 << 61, gate_stride=1 << 61)) == \
        lm.LOGMEL_ERR_INPUT_TOO_LONG
    assert _scan(lm, _scan_in(lm, n_seq=1 << 60)) == lm.LOGMEL_ERR_INPUT_TOO_LONG
    assert _scan(lm, _scan_in(lm, n_seq=1 << 58, d_state=0x1000000000000)) == \
        lm.LOGMEL_ERR_INPUT_TOO_LONG


def test_scan_splits_within_a_launch(lm):
    """Ever more sequences of 1000 rows of two channels: one workgroup each
    holds up to 2^22 of them (2^32 threads are too many for a launch), more
    are worked in parts, whose sums of a bias's gradient take less room."""
    for log2, most in ((20, None), (22, None), (23, 1 << 20), (24, 1 << 20)):
        n = 1 << log2
        inp = _scan_in(lm, type=lm.LOGMEL_F16, rows=1000 * n, channels=2, n_seq=n, x_stride=2,
                       gate_stride=2, max_frames=1000, d_bias=0x800000,
                       d_x=0x100000000000, d_gate=0x200000000000)
        need = lm._gated_scan_workspace(FAKE, inp, 1)
        assert need == 16 * n if most is None else 0 < need < most
    wide = lm.SCAN_MAX_CHANNELS
    inp = _scan_in(lm, rows=1, channels=wide, x_stride=wide, gate_stride=wide,
                   d_x=0x100000000000, d_gate=0x200000000000)
    assert lm._gated_scan_workspace(FAKE, inp, 1) >= 0
    inp = _scan_in(lm, rows=1, channels=wide + 1, x_stride=wide + 1, gate_stride=wide + 1,
                   d_x=0x100000000000, d_gate=0x200000000000)
    assert _scan(lm, inp) == lm.LOGMEL_ERR_INPUT_TOO_LONG
    assert lm._gated_scan_workspace(FAKE, inp, 1) == -1


def test_scan_refuses_bad_outputs(lm):
    bad = lm.LOGMEL_ERR_INVALID_ARGUMENT
    assert _scan(lm, _scan_in(lm), h=None) == bad
    assert _scan(lm, _scan_in(lm), h=0x200002) == bad
    assert _scan(lm, _scan_in(lm), hs=7) == bad
    assert lm._gated_scan(None, _scan_in(lm), 0x200000, 8, None, None, None, 0, None) == bad
    assert lm._gated_scan(FAKE, None, 0x200000, 8, None, None, None, 0, None) == bad


def test_scan_refuses_overlap(lm):
    bad = lm.LOGMEL_ERR_INVALID_ARGUMENT
    x = 0x100000
    assert _scan(lm, _scan_in(lm), h=x) == bad                    # h is x
    assert _scan(lm, _scan_in(lm), h=x + 16) == bad
    assert _scan(lm, _scan_in(lm), h=0x110000 - 8 * 10 * 4 + 4) == bad   # its last value in gate
    # slices of one product: x in columns 0..7, h would take 4..11 of 16
    wide = _scan_in(lm, x_stride=16)
    assert _scan(lm, wide, h=x + 16, hs=16) == bad
    assert _scan(lm, _scan_in(lm), so=0x200000 + 32) == bad       # state_out in h
    st = _scan_in(lm, d_state=0x600000)
    assert _scan(lm, st, so=0x600000 + 4) == bad                  # neither the state nor apart
    assert _scan(lm, _scan_in(lm), ck=0x200000) == bad            # checkpoints in h
    assert _scan(lm, _scan_in(lm, d_seq_offsets=0x200008)) == bad   # offsets in h
    assert _scan(lm, _scan_in(lm, d_bias=0x200000)) == bad
    g = (0x300000, 8, None, 0x300000, 8, 0x320000, 8, None, None)   # dx is dh
    assert lm._gated_scan_backward(FAKE, _scan_in(lm), 0x500000,
                                   lm.logmel_scan_grad(*g), 0x400000, 1 << 30, None) == bad
    g = (0x300000, 8, None, 0x310000, 8, 0x310010, 8, None, None)   # dgate in dx
    assert lm._gated_scan_backward(FAKE, _scan_in(lm), 0x500000,
                                   lm.logmel_scan_grad(*g), 0x400000, 1 << 30, None) == bad


def test_scan_backward_refuses(lm):
    bad = lm.LOGMEL_ERR_INVALID_ARGUMENT
    fine = dict(d_dh=0x300000, dh_stride=8, d_dx=0x340000, dx_stride=8, d_dgate=0x380000,
                dgate_stride=8)

    def call(ck=0x500000, ws=0x800000, wsb=1 << 30, **kw):
        # rows enough for several work items, whose sums of a bias's gradient
        # (and of the parts they are) need workspace
        inp = _scan_in(lm, rows=5000, d_bias=0x700000, d_x=0x1000000, d_gate=0x1100000)
        return lm._gated_scan_backward(FAKE, inp, ck,
                                       lm.logmel_scan_grad(**{**fine, **kw}), ws, wsb, None)

    assert call(ck=None) == bad
    assert call(ck=0x500002) == bad
    assert call(d_dh=None) == bad and call(d_dx=None) == bad and call(d_dgate=None) == bad
    assert call(dx_stride=7) == bad
    assert call(ws=None) == bad
    assert call(wsb=4) == bad
    assert call(ws=0x800004) == bad
    assert call(ws=0x340000) == bad     # workspace in dx
    # the gradient of a bias that is not there
    grad = lm.logmel_scan_grad(**fine, d_dbias=0x710000)
    for n_seq in (0, 2):
        assert lm._gated_scan_backward(FAKE, _scan_in(lm, n_seq=n_seq), 0x500000, grad, 0x400000,
                                       1 << 30, None) == bad


def _norm_in(lm, **kw):
    d = dict(type=lm.LOGMEL_F32, rows=10, channels=8, d_res=0x100000, res_stride=8, d_h=0x110000,
             h_stride=8, d_gate=None, gate_stride=0, d_w_post=None, d_scale=None, d_w_pre=None,
             eps=1e-6)
    d.update(kw)
    return lm.logmel_norm_input(**d)


def _norm(lm, inp, y=0x200000, ys=8, z=0x210000, zs=8):
    return lm._block_norm(FAKE, inp, y, ys, z, zs, None)


def test_norm_refuses(lm):
    bad = lm.LOGMEL_ERR_INVALID_ARGUMENT
    for kw in (dict(rows=-1), dict(channels=0), dict(d_res=None), dict(res_stride=7),
               dict(h_stride=7), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(d_h=None, d_gate=0x120000, gate_stride=8), dict(d_h=None, d_scale=0x130000),
               dict(d_h=None, d_w_post=0x130000), dict(d_w_pre=0x130002), dict(d_res=0x100001)):
        assert _norm(lm, _norm_in(lm, **kw)) == bad, kw
    assert _norm(lm, _norm_in(lm, type=lm.LOGMEL_I16)) == lm.LOGMEL_ERR_UNSUPPORTED
    wide = lm.NORM_MAX_CHANNELS + 1
    assert _norm(lm, _norm_in(lm, channels=wide, res_stride=wide, h_stride=wide)) == \
        lm.LOGMEL_ERR_UNSUPPORTED
    assert _norm(lm, _norm_in(lm, rows=1 << 40, res_stride=1 << 61)) == \
        lm.LOGMEL_ERR_INPUT_TOO_LONG
    assert _norm(lm, _norm_in(lm), y=None, z=None) == bad
    assert _norm(lm, _norm_in(lm, d_h=None)) == bad                 # y without h
    assert _norm(lm, _norm_in(lm), y=0x100000) == bad               # y is res
    assert _norm(lm, _norm_in(lm), z=0x200010) == bad               # z in y
    assert _norm(lm, _norm_in(lm), ys=4) == bad
    assert _norm(lm, _norm_in(lm, d_w_pre=0x200020)) == bad
    assert lm._block_norm(None, _norm_in(lm), 0x200000, 8, None, 0, None) == bad


def test_norm_backward_refuses(lm):
    bad = lm.LOGMEL_ERR_INVALID_ARGUMENT
    fine = dict(d_dy=0x300000, dy_stride=8, d_dz=0x310000, dz_stride=8, d_dres=0x320000,
                dres_stride=8, d_dh=0x330000, dh_stride=8)

    def call(inp=None, ws=0x400000, wsb=1 << 30, **kw):
        return lm._block_norm_backward(FAKE, inp or _norm_in(lm),
                                       lm.logmel_norm_grad(**{**fine, **kw}), ws, wsb, None)

    assert call(d_dy=None, d_dz=None) == bad
    assert call(d_dres=None) == bad and call(d_dh=None) == bad
    assert call(d_dgate=0x340000, dgate_stride=8) == bad            # no gate
    gated = _norm_in(lm, d_gate=0x120000, gate_stride=8)
    assert call(inp=gated) == bad                                   # its gradient is missing
    plain = _norm_in(lm, d_h=None)
    assert call(inp=plain) == bad                                   # dh without h
    assert call(inp=plain, d_dh=None, d_dscale=0x350000) == bad
    assert call(d_dz=None, d_dw_pre=0x350000) == bad
    assert call(d_dres=0x300000) == bad                             # dres is dy
    assert call(d_dh=0x320010) == bad
    assert call(ws=0x320000) == bad


def test_checkpoint_rows(lm):
    f = lm.logmel_gated_scan_checkpoint_rows
    assert [f(r) for r in (-1, 0, 1, 128, 129, 256, 2 ** 40 + 1)] == \
        [-1, 0, 1, 1, 2, 2, 2 ** 33 + 1]


def test_binding_refuses_host_tensors(lm):
    import torch

    class P:
        handle, device = None, 0

    x = torch.zeros(4, 8)
    off = torch.tensor([0, 4])
    with pytest.raises(TypeError):
        lm.logmel_gated_scan(P(), x, x, off)
    with pytest.raises(TypeError):
        lm.logmel_gated_scan(P(), x.double(), x.double(), off)
    with pytest.raises(TypeError):
        lm.logmel_block_norm(P(), x)
    with pytest.raises(TypeError):
        lm.logmel_block_norm_backward(P(), x.to(torch.int16), dz=x)
