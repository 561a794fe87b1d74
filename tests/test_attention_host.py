"""Linear attention and the group norm without a GPU: the fp64 forms they are
tested against (recurrence, closed forms, differences), and the calls that are
refused on the host before any launch."""

import ctypes

import numpy as np
import pytest

from tests import attn_ref
from tests.libload import load_binding
from tests.test_rows_host import FAKE, _differences


@pytest.fixture(scope="module")
def lm():
    return load_binding()


# ------------------------------------------------------------ the fp64 forms

def test_attention_form_is_the_recurrence():
    rng = np.random.default_rng(1)
    off, heads, qk, dk, dv, scale = np.array([0, 5, 5, 6, 20]), 4, 2, 3, 5, 0.7
    q, k = rng.normal(size=(20, qk * dk)), rng.normal(size=(20, qk * dk))
    v, g = rng.normal(size=(20, heads * dv)), -np.array([0.0, 0.01, 1.0, np.inf])
    s0 = rng.normal(size=(4, heads, dk, dv))
    val, _ = attn_ref.attention(q, k, v, g, off, qk, scale, s0)
    for j in range(4):
        s = s0[j].copy()
        for t in range(off[j], off[j + 1]):
            for h in range(heads):
                hq = h // 2
                s[h] = np.exp(g[h]) * s[h] + np.outer(k[t, hq * dk:(hq + 1) * dk],
                                                      v[t, h * dv:(h + 1) * dv])
                o = scale * q[t, hq * dk:(hq + 1) * dk] @ s[h]
                assert np.allclose(val["o"][t, h * dv:(h + 1) * dv], o, atol=1e-12)
        assert np.allclose(val["state_out"][j], s, atol=1e-12)


def test_attention_form_gradient_by_differences():
    rng = np.random.default_rng(2)
    off, heads, qk, dk, dv, scale = np.array([0, 4, 4, 5, 9]), 2, 1, 3, 2, 0.7
    p = dict(q=rng.normal(size=(9, qk * dk)), k=rng.normal(size=(9, qk * dk)),
             v=rng.normal(size=(9, heads * dv)), state=rng.normal(size=(4, heads, dk, dv)))
    g = -np.array([0.05, 0.8])
    do, dso = rng.normal(size=(9, heads * dv)), rng.normal(size=(4, heads, dk, dv))

    def loss():
        v, _ = attn_ref.attention(p["q"], p["k"], p["v"], g, off, qk, scale, p["state"])
        return (v["o"] * do).sum() + (v["state_out"] * dso).sum()

    val, _ = attn_ref.attention(p["q"], p["k"], p["v"], g, off, qk, scale, p["state"], do, dso)
    for key, name in dict(q="dq", k="dk", v="dv", state="dstate").items():
        _differences(p[key], loss, val[name])


def test_group_form_is_the_norm():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(7, 12)) * 3 + 5
    val, _ = attn_ref.group_norm(x, 3, eps=0.0)
    y = val["y"].reshape(7, 3, 4)
    assert np.allclose(y.mean(2), 0.0, atol=1e-12) and np.allclose(y.var(2), 1.0)
    val, _ = attn_ref.group_norm(x, 3, off=np.array([0, 2, 2, 6]), eps=0.0)
    y = val["y"].reshape(7, 3, 4)
    for at in (slice(0, 2), slice(2, 6)):
        assert np.allclose(y[at].mean((0, 2)), 0.0, atol=1e-12)
        assert np.allclose(y[at].var((0, 2)), 1.0)
    assert np.isnan(y[6]).all()


@pytest.mark.parametrize("off", [None, [0, 2, 2, 5]])
@pytest.mark.parametrize("silu", [False, True])
def test_group_form_gradient_by_differences(off, silu):
    rng = np.random.default_rng(4)
    p = dict(x=rng.normal(size=(5, 6)), gate=rng.normal(size=(5, 6)), weight=rng.normal(size=6),
             bias=rng.normal(size=6))
    dy = rng.normal(size=(5, 6))
    more = dict(silu=silu, off=None if off is None else np.array(off), eps=1e-2)

    def loss():
        v, _ = attn_ref.group_norm(groups=2, **p, **more)
        return (v["y"] * dy).sum()

    val, _ = attn_ref.group_norm(groups=2, dy=dy, **p, **more)
    for key, name in dict(x="dx", gate="dgate", weight="dweight", bias="dbias").items():
        _differences(p[key], loss, val[name])


# ------------------------------------------------------------ refused calls

def _attn_in(lm, **kw):
    d = dict(type=lm.LOGMEL_F32, rows=10, heads=4, qk_heads=2, head_dk=8, head_dv=4, n_seq=2,
             d_seq_offsets=0x1000, max_frames=0, d_q=0x100000, q_stride=16, d_k=0x110000,
             k_stride=16, d_v=0x120000, v_stride=16, d_log_decay=0x130000, d_state=None,
             scale=1.0)
    d.update(kw)
    return lm.logmel_attention_input(**d)


def _attn(lm, inp, o=0x200000, os=16, so=None, ws=0x40000000, wsb=1 << 40):
    return lm._linear_attention(FAKE, inp, o, os, so, ws, wsb, None)


def _attn_back(lm, inp, ws=0x40000000, wsb=1 << 40, **kw):
    d = dict(d_do=0x300000, do_stride=16, d_dstate_out=None, d_dq=0x310000, dq_stride=16,
             d_dk=0x320000, dk_stride=16, d_dv=0x330000, dv_stride=16, d_dstate=None)
    d.update(kw)
    return lm._linear_attention_backward(FAKE, inp, lm.logmel_attention_grad(**d), ws, wsb, None)


_BAD = dict(
    rows=dict(rows=-1), heads=dict(heads=0), qk_heads=dict(qk_heads=0),
    shared=dict(heads=4, qk_heads=3), more_qk=dict(heads=2, qk_heads=4), dk=dict(head_dk=0),
    dv=dict(head_dv=-4), n_seq=dict(n_seq=-1), offsets_null=dict(d_seq_offsets=None),
    offsets_odd=dict(d_seq_offsets=0x1004), max_frames=dict(max_frames=-1), q_null=dict(d_q=None),
    q_odd=dict(d_q=0x100002), q_stride=dict(q_stride=15), k_null=dict(d_k=None),
    k_stride=dict(k_stride=0), v_null=dict(d_v=None), v_stride=dict(v_stride=15),
    decay_null=dict(d_log_decay=None), decay_odd=dict(d_log_decay=0x130001),
    state_odd=dict(d_state=0x140002), scale=dict(scale=float("nan")),
    scale_inf=dict(scale=float("inf")))


@pytest.mark.parametrize("name", sorted(_BAD))
def test_attention_refuses_bad_inputs(lm, name):
    inp = _attn_in(lm, **_BAD[name])
    assert _attn(lm, inp) == lm.LOGMEL_ERR_INVALID_ARGUMENT
    assert _attn_back(lm, inp) == lm.LOGMEL_ERR_INVALID_ARGUMENT
    if name != "state_odd":
        assert lm._linear_attention_workspace(FAKE, inp, 0) == -1


def test_attention_refuses_types_and_sizes(lm):
    assert _attn(lm, _attn_in(lm, type=lm.LOGMEL_I16)) == lm.LOGMEL_ERR_UNSUPPORTED
    most = lm.ATTENTION_MAX_HEAD_DIM
    for kw in (dict(head_dk=most + 1, q_stride=1 << 10, k_stride=1 << 10),
               dict(head_dv=most + 1, v_stride=1 << 10)):
        assert _attn(lm, _attn_in(lm, **kw)) == lm.LOGMEL_ERR_UNSUPPORTED
    long = lm.LOGMEL_ERR_INPUT_TOO_LONG
    assert _attn(lm, _attn_in(lm, rows=1 << 40, q_stride=1 << 61)) == long
    assert _attn(lm, _attn_in(lm, n_seq=1 << 60)) == long
    assert _attn(lm, _attn_in(lm, n_seq=1 << 58)) == long        # the states' count
    assert _attn(lm, _attn_in(lm, heads=1 << 30, qk_heads=1)) == long
    assert _attn(lm, _attn_in(lm, rows=1 << 54, q_stride=16, d_q=0x1 << 20)) == long


def test_attention_refuses_bad_outputs_and_overlap(lm):
    bad = lm.LOGMEL_ERR_INVALID_ARGUMENT
    assert _attn(lm, _attn_in(lm), o=None) == bad
    assert _attn(lm, _attn_in(lm), o=0x200002) == bad
    assert _attn(lm, _attn_in(lm), os=15) == bad
    assert lm._linear_attention(None, _attn_in(lm), 0x200000, 16, None, None, 0, None) == bad
    assert lm._linear_attention(FAKE, None, 0x200000, 16, None, None, 0, None) == bad
    for x in (0x100000, 0x110000, 0x120000, 0x130000, 0x1008):     # o is q, k, v, ...
        assert _attn(lm, _attn_in(lm), o=x) == bad
    assert _attn(lm, _attn_in(lm), so=0x200000 + 32) == bad         # state_out in o
    st = _attn_in(lm, d_state=0x600000)
    assert _attn(lm, st, so=0x600000 + 4) == bad                    # neither the state nor apart
    assert _attn(lm, _attn_in(lm), so=0x100000) == bad
    # slices of one product: v in columns 0..15, o would take 8..23 of 32
    assert _attn(lm, _attn_in(lm, v_stride=32), o=0x120000 + 32, os=32) == bad


def test_attention_backward_refuses(lm):
    bad = lm.LOGMEL_ERR_INVALID_ARGUMENT
    inp = _attn_in(lm)
    for name in ("d_do", "d_dq", "d_dk", "d_dv"):
        assert _attn_back(lm, inp, **{name: None}) == bad
    assert _attn_back(lm, inp, dq_stride=15) == bad
    assert _attn_back(lm, inp, d_dq=0x300000) == bad                # dq is do
    assert _attn_back(lm, inp, d_dk=0x310010) == bad                # dk in dq
    assert _attn_back(lm, inp, d_dstate=0x330000) == bad            # dstate in dv
    assert _attn_back(lm, inp, d_dstate_out=0x600000, d_dstate=0x600000) == bad
    need = lm._linear_attention_workspace(FAKE, inp, 1)             # q and k are shared
    assert need > 0
    assert _attn_back(lm, inp, ws=None) == bad
    assert _attn_back(lm, inp, wsb=need - 1) == bad
    assert _attn_back(lm, inp, ws=0x40000004) == bad
    assert _attn_back(lm, inp, ws=0x310000) == bad                  # workspace in dq


def _group_in(lm, **kw):
    d = dict(type=lm.LOGMEL_F32, rows=10, channels=8, groups=2, n_seq=2, d_seq_offsets=0x1000,
             max_frames=0, d_x=0x100000, x_stride=8, d_gate=None, gate_stride=0, d_weight=None,
             d_bias=None, activation=lm.LOGMEL_ACT_SILU, eps=1e-5)
    d.update(kw)
    return lm.logmel_group_norm_input(**d)


def _group(lm, inp, y=0x200000, ys=8, stats=None, ws=0x40000000, wsb=1 << 40):
    return lm._group_norm(FAKE, inp, y, ys, stats, ws, wsb, None)


def _group_back(lm, inp, stats=0x500000, ws=0x40000000, wsb=1 << 40, **kw):
    d = dict(d_dy=0x300000, dy_stride=8, d_dx=0x310000, dx_stride=8, d_dgate=None, dgate_stride=0,
             d_dweight=None, d_dbias=None)
    d.update(kw)
    return lm._group_norm_backward(FAKE, inp, stats, lm.logmel_group_norm_grad(**d), ws, wsb,
                                   None)


def test_group_norm_refuses(lm):
    bad = lm.LOGMEL_ERR_INVALID_ARGUMENT
    for kw in (dict(rows=-1), dict(channels=0), dict(groups=0), dict(groups=3), dict(groups=16),
               dict(n_seq=-1), dict(max_frames=-1), dict(d_seq_offsets=None),
               dict(d_seq_offsets=None, n_seq=0, max_frames=5), dict(d_seq_offsets=0x1004),
               dict(d_x=None), dict(d_x=0x100001), dict(x_stride=7),
               dict(d_gate=0x110000, gate_stride=7), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(d_weight=0x120001), dict(d_bias=0x120002)):
        assert _group(lm, _group_in(lm, **kw)) == bad, kw
        assert _group_back(lm, _group_in(lm, **kw)) == bad, kw
    wide = lm.NORM_MAX_CHANNELS + 2
    for kw in (dict(type=lm.LOGMEL_I16), dict(activation=2),
               dict(channels=wide, x_stride=wide)):
        assert _group(lm, _group_in(lm, **kw)) == lm.LOGMEL_ERR_UNSUPPORTED
    assert _group(lm, _group_in(lm, rows=1 << 40, x_stride=1 << 61)) == \
        lm.LOGMEL_ERR_INPUT_TOO_LONG
    assert _group(lm, _group_in(lm), y=None) == bad
    assert _group(lm, _group_in(lm), y=0x100000) == bad              # y is x
    assert _group(lm, _group_in(lm), stats=0x200010) == bad          # stats in y
    by_row = _group_in(lm, d_seq_offsets=None, n_seq=0)
    assert _group(lm, by_row, stats=0x500000) == bad                 # none by rows
    assert lm._group_norm(None, by_row, 0x200000, 8, None, None, 0, None) == bad


def test_group_norm_backward_refuses(lm):
    bad = lm.LOGMEL_ERR_INVALID_ARGUMENT
    inp = _group_in(lm)
    assert _group_back(lm, inp, stats=None) == bad
    assert _group_back(lm, inp, d_dy=None) == bad and _group_back(lm, inp, d_dx=None) == bad
    assert _group_back(lm, inp, d_dgate=0x320000, dgate_stride=8) == bad   # no gate
    assert _group_back(lm, _group_in(lm, d_gate=0x110000, gate_stride=8)) == bad
    assert _group_back(lm, inp, d_dweight=0x330000) == bad                 # no weight
    assert _group_back(lm, inp, d_dbias=0x330000) == bad
    assert _group_back(lm, inp, d_dx=0x300000) == bad
    by_row = _group_in(lm, d_seq_offsets=None, n_seq=0)
    assert _group_back(lm, by_row) == bad                                  # stats by rows
    assert _group_back(lm, inp, ws=None) == bad
    assert _group_back(lm, inp, ws=0x310000) == bad                        # workspace in dx


def test_group_norm_refuses_counts_that_overflow(lm):
    """Sequences whose statistics' count, and the workspace's, pass 64 bits."""
    inp = _group_in(lm, n_seq=1 << 58)
    assert _group(lm, inp) == lm.LOGMEL_ERR_INPUT_TOO_LONG
    assert _group_back(lm, inp) == lm.LOGMEL_ERR_INPUT_TOO_LONG
    assert lm._group_norm_workspace(FAKE, inp, 0) == -1


def test_attention_refuses_counts_that_overflow(lm):
    """A state whose size passes 64 bits is refused before it is multiplied out."""
    for kw in (dict(heads=1 << 40, head_dk=1 << 40), dict(head_dk=1 << 62, head_dv=1 << 62)):
        inp = _attn_in(lm, **kw)
        assert _attn(lm, inp) != lm.LOGMEL_OK
        assert lm._linear_attention_workspace(FAKE, inp, 1) == -1


def test_binding_refuses_host_tensors(lm):
    import torch

    class P:
        handle, device = None, 0

    x, g = torch.zeros(4, 8), torch.zeros(2)
    off = torch.tensor([0, 4])
    with pytest.raises(TypeError):
        lm.logmel_linear_attention(P(), x, x, x, g, off)
    with pytest.raises(TypeError):
        lm.logmel_linear_attention_backward(P(), x, x, x, x, g, off)
    with pytest.raises(TypeError):
        lm.logmel_group_norm(P(), x, 2)
    with pytest.raises(TypeError):
        lm.logmel_group_norm_backward(P(), x, x, 2)
