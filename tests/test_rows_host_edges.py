"""Calls of the row operators that are refused on the host, beside those of
test_rows_host.py."""

import pytest

from tests.test_rows_host import FAKE, _scan, _scan_in, lm   # noqa: F401


def test_scan_in_place_excuses_the_state_alone(lm):   # noqa: F811
    """state_out may be the state; another input at the same address is
    overwritten while it is read, and refused as if there were no state."""
    bad = lm.LOGMEL_ERR_INVALID_ARGUMENT
    at = 0x600000
    one = dict(n_seq=1, d_state=at)
    assert _scan(lm, _scan_in(lm, **one, d_bias=at), so=at) == bad
    assert _scan(lm, _scan_in(lm, **one, d_x=at), so=at) == bad
    assert _scan(lm, _scan_in(lm, **one, d_gate=at), so=at) == bad
    assert _scan(lm, _scan_in(lm, **one, d_seq_offsets=at), so=at) == bad
    # and where it only begins or ends in the state
    assert _scan(lm, _scan_in(lm, n_seq=2, d_state=at, d_bias=at + 32), so=at) == bad
    assert _scan(lm, _scan_in(lm, **one, d_x=at + 16), so=at) == bad
    # without a state nothing is excused
    assert _scan(lm, _scan_in(lm, n_seq=1, d_bias=at), so=at) == bad
    # the gradient writes its dstate apart from the state
    grad = lm.logmel_scan_grad(0x300000, 8, None, 0x310000, 8, 0x320000, 8, None, at)
    assert lm._gated_scan_backward(FAKE, _scan_in(lm, **one), 0x500000, grad, 0x400000, 1 << 30,
                                   None) == bad


def test_binding_refuses_a_graph_only_while_one_is_recorded(lm):   # noqa: F811
    import torch

    with pytest.raises(RuntimeError, match="x requires grad.*autograd"):
        lm._refuse_graph("x")
    with torch.no_grad():
        lm._refuse_graph("x")
    with torch.inference_mode():
        lm._refuse_graph("x")


def test_binding_refuses_a_stream_of_another_device(lm):   # noqa: F811
    """The kernels would run on that device, with the plan's memory."""
    import torch

    class P:
        handle, device = None, 0

    class Stream:
        cuda_stream, device = 0, torch.device("cuda", 1)

    x = torch.zeros(4, 8)
    off = torch.tensor([0, 4])
    for call in (lambda: lm.logmel_gated_scan(P(), x, x, off, stream=Stream()),
                 lambda: lm.logmel_gated_scan_backward(P(), x, x, x, off, x[:1], stream=Stream()),
                 lambda: lm.logmel_block_norm(P(), x, stream=Stream()),
                 lambda: lm.logmel_block_norm_backward(P(), x, dz=x, stream=Stream())):
        with pytest.raises(ValueError, match="stream must be on the plan's device 0"):
            call()
