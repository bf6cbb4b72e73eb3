"""Gated cyclic feed-forward layer: host-side checks of the C ABI and of the binding (nothing is launched)."""

import ctypes

import pytest
import torch

import group_wise_dft_b200 as eq

L = eq.raw_lib()
P = ctypes.c_void_p(0x1000)      # aligned, never dereferenced: the calls fail before a launch
MIS = ctypes.c_void_p(0x1008)
BIG = 1 << 40


def spec(W=P, N=6, C=10, H=5, dtype=0, out=P, bytes_=BIG):
    return L.eqlin_cyclic_gated_weight_spectrum(W, N, C, H, dtype, out, bytes_, None)


def adj(W=P, N=6, C=10, H=5, dtype=0, out=P, bytes_=BIG):
    return L.eqlin_cyclic_gated_weight_spectrum_adjoint(W, N, C, H, dtype, out, bytes_, None)


def fwd(x=P, spec=P, h=P, T=9, N=6, C=10, H=5, act=1, dtype=0, path=0, ws=None, bytes_=0):
    return L.eqlin_cyclic_gated_forward(x, spec, h, T, N, C, H, act, dtype, path, ws, bytes_, None)


def bwd(x=P, dh=P, spec=P, adj=P, dx=P, dW=P, T=9, N=6, C=10, H=5, act=1, dtype=0, path=0, ws=P, bytes_=BIG):
    return L.eqlin_cyclic_gated_backward(x, dh, spec, adj, dx, dW, T, N, C, H, act, dtype, path, ws, bytes_, None)


SHAPES = [
    (dict(N=0), eq.EQLIN_ERR_UNSUPPORTED), (dict(N=17), eq.EQLIN_ERR_UNSUPPORTED),
    (dict(C=0), eq.EQLIN_ERR_INVALID_ARG), (dict(H=0), eq.EQLIN_ERR_INVALID_ARG),
    (dict(H=-3), eq.EQLIN_ERR_INVALID_ARG), (dict(H=1 << 30), eq.EQLIN_ERR_INVALID_ARG),
    (dict(C=1 << 23), eq.EQLIN_ERR_UNSUPPORTED), (dict(H=1 << 22), eq.EQLIN_ERR_UNSUPPORTED),
    (dict(dtype=5), eq.EQLIN_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("args,code", SHAPES)
def test_shapes(args, code):
    for call in (spec, adj, fwd, bwd):
        assert call(**args) == code and len(L.eqlin_last_error()) > 0
    a = dict(N=6, C=10, H=5, dtype=0)
    a.update(args)
    shape = (a["N"], a["C"], a["H"], a["dtype"])
    assert L.eqlin_cyclic_gated_spectrum_bytes(*shape) == 0
    assert L.eqlin_cyclic_gated_adjoint_bytes(*shape) == 0
    assert L.eqlin_cyclic_gated_auto_path(*shape) == -1
    assert L.eqlin_cyclic_gated_forward_workspace_bytes(9, *shape) == 0
    assert L.eqlin_cyclic_gated_backward_workspace_bytes(9, *shape) == 0


@pytest.mark.parametrize("args,code", [
    (dict(T=-1), eq.EQLIN_ERR_INVALID_ARG), (dict(T=1 << 62), eq.EQLIN_ERR_UNSUPPORTED),
    (dict(act=3), eq.EQLIN_ERR_INVALID_ARG), (dict(act=-1), eq.EQLIN_ERR_INVALID_ARG),
    (dict(path=3), eq.EQLIN_ERR_INVALID_ARG), (dict(path=eq.PATH_TC), eq.EQLIN_ERR_UNSUPPORTED),
    (dict(x=None), eq.EQLIN_ERR_INVALID_ARG), (dict(spec=None), eq.EQLIN_ERR_INVALID_ARG),
    (dict(x=MIS), eq.EQLIN_ERR_ALIGN), (dict(spec=MIS), eq.EQLIN_ERR_ALIGN),
])
def test_calls(args, code):
    for call in (fwd, bwd):
        assert call(**args) == code and len(L.eqlin_last_error()) > 0


def test_forward_output():
    assert fwd(h=None) == eq.EQLIN_ERR_INVALID_ARG
    assert fwd(h=MIS) == eq.EQLIN_ERR_ALIGN
    assert fwd(x=None, spec=None, h=None, T=0) == eq.EQLIN_OK


@pytest.mark.parametrize("args,code", [
    (dict(dx=None, dW=None), eq.EQLIN_ERR_INVALID_ARG), (dict(dh=None), eq.EQLIN_ERR_INVALID_ARG),
    (dict(adj=None), eq.EQLIN_ERR_INVALID_ARG), (dict(ws=None), eq.EQLIN_ERR_INVALID_ARG),
    (dict(dh=MIS), eq.EQLIN_ERR_ALIGN), (dict(dx=MIS), eq.EQLIN_ERR_ALIGN), (dict(dW=MIS), eq.EQLIN_ERR_ALIGN),
    (dict(adj=MIS), eq.EQLIN_ERR_ALIGN), (dict(ws=ctypes.c_void_p(0x1010)), eq.EQLIN_ERR_ALIGN),
    (dict(bytes_=64), eq.EQLIN_ERR_SIZE),
])
def test_backward_buffers(args, code):
    assert bwd(**args) == code


@pytest.mark.parametrize("call", [spec, adj])
def test_spectrum_buffers(call):
    assert call(W=None) == eq.EQLIN_ERR_INVALID_ARG
    assert call(out=None) == eq.EQLIN_ERR_INVALID_ARG
    assert call(W=MIS) == eq.EQLIN_ERR_ALIGN
    assert call(out=MIS) == eq.EQLIN_ERR_ALIGN
    assert call(bytes_=128) == eq.EQLIN_ERR_SIZE


def test_forward_workspace():
    """Some tensor-core shapes need one; they are refused without it when asked for."""
    need = L.eqlin_cyclic_gated_forward_workspace_bytes(100, 16, 96, 64, eq.EQLIN_BF16)
    assert need >= 100 * 96 * 16 * 2 and need % 256 == 0
    assert L.eqlin_cyclic_gated_forward_workspace_bytes(100000, 8, 96, 64, eq.EQLIN_BF16) == 0
    assert L.eqlin_cyclic_gated_forward_workspace_bytes(100, 16, 96, 64, eq.EQLIN_F32) == 0
    tc = dict(T=100, N=16, C=96, H=64, dtype=eq.EQLIN_BF16, path=eq.PATH_TC)
    assert fwd(**tc) == eq.EQLIN_ERR_SIZE
    assert fwd(**tc, ws=P, bytes_=need - 1) == eq.EQLIN_ERR_SIZE
    assert fwd(**tc, ws=ctypes.c_void_p(0x1010), bytes_=need) == eq.EQLIN_ERR_SIZE
    # T past what the kernels index: refused, not cut
    assert fwd(T=1 << 31, N=16, C=96, H=64, dtype=eq.EQLIN_BF16, path=eq.PATH_TC, ws=P, bytes_=BIG) == \
        eq.EQLIN_ERR_UNSUPPORTED


def test_binding_refuses_bad_tensors():
    with pytest.raises(ValueError):
        eq.cyclic_gated_weight_spectrum(torch.zeros(4, 3, 8))
    with pytest.raises(ValueError):
        eq.cyclic_gated_weight_spectrum(torch.zeros(4, 3, 5, 8))
    with pytest.raises(ValueError):
        eq.cyclic_gated_weight_spectrum(torch.zeros(4, 2, 5, 8))          # not on a GPU
    with pytest.raises(eq.EqlinError):
        eq.cyclic_gated_weight_spectrum(torch.zeros(4, 2, 5, 17))
    x = torch.zeros(3, 5, 8)
    small = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        eq.cyclic_gated_forward(x, small, 4)
    with pytest.raises(ValueError):
        eq.cyclic_gated_forward(x, torch.zeros(1 << 20), 4)               # not bytes
    with pytest.raises(ValueError):
        eq.cyclic_gated_forward(x, torch.zeros(1 << 20, dtype=torch.uint8), 4, h=torch.zeros(3, 5, 8))
    with pytest.raises(ValueError):
        eq.cyclic_gated_backward(x, torch.zeros(2, 4, 8), small, small)   # another T
    with pytest.raises(ValueError):
        eq.cyclic_gated_backward(x, torch.zeros(3, 4, 8).half(), small, small)
