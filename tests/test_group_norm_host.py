"""Group norm: host-side checks of the C ABI and of the binding (nothing is launched)."""

import ctypes

import pytest
import torch

import group_wise_dft_b200 as eq

L = eq.raw_lib()
P = ctypes.c_void_p(0x1000)      # aligned, never dereferenced: the calls fail before a launch
MIS = ctypes.c_void_p(0x1008)
BIG = 1 << 40
EPS = ctypes.c_float(1e-5)


def fwd(x=P, gamma=P, beta=P, y=P, mean=P, rstd=P, B=4, S=1000, F=16, N=8, G=4, eps=EPS, act=1, dtype=1, ws=P,
        bytes_=BIG):
    return L.eqlin_group_norm(x, gamma, beta, y, mean, rstd, B, S, F, N, G, eps, act, dtype, ws, bytes_, None)


def bwd(x=P, dy=P, mean=P, rstd=P, gamma=P, beta=P, dx=P, dg=P, db=P, B=4, S=1000, F=16, N=8, G=4, act=1, dtype=1,
        ws=P, bytes_=BIG):
    return L.eqlin_group_norm_backward(x, dy, mean, rstd, gamma, beta, dx, dg, db, B, S, F, N, G, act, dtype, ws,
                                       bytes_, None)


REFUSED = [
    (dict(N=0), eq.EQLIN_ERR_UNSUPPORTED),
    (dict(N=17), eq.EQLIN_ERR_UNSUPPORTED),
    (dict(dtype=3), eq.EQLIN_ERR_UNSUPPORTED),
    (dict(B=-1), eq.EQLIN_ERR_INVALID_ARG),
    (dict(S=-1), eq.EQLIN_ERR_INVALID_ARG),
    (dict(F=0), eq.EQLIN_ERR_INVALID_ARG),
    (dict(G=0), eq.EQLIN_ERR_INVALID_ARG),
    (dict(G=-4), eq.EQLIN_ERR_INVALID_ARG),
    (dict(G=5), eq.EQLIN_ERR_INVALID_ARG),                      # F % G != 0
    (dict(F=1 << 22, N=8, G=1), eq.EQLIN_ERR_UNSUPPORTED),      # F N > 2^24
    (dict(F=4096, G=4096), eq.EQLIN_ERR_UNSUPPORTED),           # too many groups
    (dict(B=1 << 62), eq.EQLIN_ERR_UNSUPPORTED),
    (dict(B=1 << 30, S=1 << 30), eq.EQLIN_ERR_UNSUPPORTED),
    (dict(act=3), eq.EQLIN_ERR_INVALID_ARG),
    (dict(act=-1), eq.EQLIN_ERR_INVALID_ARG),
    (dict(x=None), eq.EQLIN_ERR_INVALID_ARG),
    (dict(x=MIS), eq.EQLIN_ERR_ALIGN),
    (dict(gamma=MIS), eq.EQLIN_ERR_ALIGN),
    (dict(beta=MIS), eq.EQLIN_ERR_ALIGN),
    (dict(ws=None), eq.EQLIN_ERR_INVALID_ARG),
    (dict(ws=MIS), eq.EQLIN_ERR_ALIGN),
    (dict(bytes_=16), eq.EQLIN_ERR_SIZE),
]


@pytest.mark.parametrize("args,code", REFUSED)
def test_refusals(args, code):
    assert fwd(**args) == code and len(L.eqlin_last_error()) > 0
    assert bwd(**args) == code and len(L.eqlin_last_error()) > 0


@pytest.mark.parametrize("args,code", [
    (dict(y=None), eq.EQLIN_ERR_INVALID_ARG), (dict(y=MIS), eq.EQLIN_ERR_ALIGN),
    (dict(mean=MIS), eq.EQLIN_ERR_ALIGN), (dict(rstd=MIS), eq.EQLIN_ERR_ALIGN),
    (dict(eps=ctypes.c_float(-1.0)), eq.EQLIN_ERR_INVALID_ARG),
    (dict(eps=ctypes.c_float(float("nan"))), eq.EQLIN_ERR_INVALID_ARG),
])
def test_forward_refusals(args, code):
    assert fwd(**args) == code


@pytest.mark.parametrize("args,code", [
    (dict(dy=None), eq.EQLIN_ERR_INVALID_ARG), (dict(dx=None), eq.EQLIN_ERR_INVALID_ARG),
    (dict(mean=None), eq.EQLIN_ERR_INVALID_ARG), (dict(rstd=None), eq.EQLIN_ERR_INVALID_ARG),
    (dict(dy=MIS), eq.EQLIN_ERR_ALIGN), (dict(dx=MIS), eq.EQLIN_ERR_ALIGN), (dict(mean=MIS), eq.EQLIN_ERR_ALIGN),
    (dict(dg=MIS), eq.EQLIN_ERR_ALIGN), (dict(db=MIS), eq.EQLIN_ERR_ALIGN),
])
def test_backward_refusals(args, code):
    assert bwd(**args) == code


def test_empty_forward_is_a_no_op():
    assert fwd(x=None, y=None, ws=None, bytes_=0, B=0) == eq.EQLIN_OK
    assert fwd(x=None, y=None, ws=None, bytes_=0, S=0) == eq.EQLIN_OK
    assert bwd(x=None, dy=None, dx=None, dg=None, db=None, ws=None, bytes_=0, B=0) == eq.EQLIN_OK


def test_workspace_sizes():
    ws, wb = L.eqlin_group_norm_workspace_bytes, L.eqlin_group_norm_backward_workspace_bytes
    assert ws(131072, 1, 160, 8, 1, 1) == 0           # tokens: one pass
    assert ws(2, 4096, 160, 8, 32, 1) > 0
    assert wb(2, 4096, 160, 8, 32, 1) > 0 and wb(10, 1, 160, 8, 1, 1) > 0
    for f in (ws, wb):
        assert f(0, 10, 16, 8, 4, 1) == 0
        assert f(-1, 10, 16, 8, 4, 1) == 0 and f(2, 10, 16, 8, 3, 1) == 0 and f(2, 10, 16, 17, 4, 1) == 0


def test_binding_refuses_bad_tensors():
    x = torch.zeros(2, 16, 8)
    with pytest.raises(ValueError):
        eq.group_norm(x[0], 4)                               # not [B, .., F, N]
    with pytest.raises(ValueError):
        eq.group_norm(x, 4, gamma=torch.zeros(15))
    with pytest.raises(ValueError):
        eq.group_norm(x, 4, beta=torch.zeros(16, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        eq.group_norm(x, 4, y=torch.zeros(2, 16, 4))
    with pytest.raises(ValueError):
        eq.group_norm(x, 4, mean=torch.zeros(2, 3))
    with pytest.raises(ValueError):
        eq.group_norm(x, 4)                                  # not on a GPU
    with pytest.raises(TypeError):
        eq.group_norm(x.double(), 4)
    m = torch.zeros(2, 4)
    with pytest.raises(ValueError):
        eq.group_norm_backward(x, x[:1], m, m, 4)
    with pytest.raises(ValueError):
        eq.group_norm_backward(x, x, m[:, :2], m, 4)
    with pytest.raises(ValueError):
        eq.group_norm_backward(x, x, m.half(), m, 4)
