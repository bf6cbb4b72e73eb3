"""The feed-forward block (token group norm, gated layer, contraction): refusals on the CPU, and on a B200 the
block against its definition in 64 bits and a training step's forward and backward of its parts.

Tolerance: every intermediate tensor and the result are rounded to the type (half a step each), and on tensor cores
the half spectra of x, of the hidden layer and of both weights (half a step each); with independent roundings of rms
half a step / sqrt 3 and the activation's factor of at most 1.6, as for the gated layer, the CUDA-core result is
within 2 half steps (Frobenius), the tensor cores' within 3.  fp32: 4e-6 more for its sums.
"""

import ctypes
import math

import pytest
import torch

import group_wise_dft_b200 as eq

L = eq.raw_lib()
P, MIS, BIG = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008), 1 << 40


def call(x=P, gamma=P, beta=P, w1=P, w2=P, y=P, T=9, N=6, C=12, H=5, G=3, eps=1e-5, act=1, dtype=0, path=0, ws=P,
         bytes_=BIG):
    return L.eqlin_cyclic_gated_mlp(x, gamma, beta, w1, w2, y, T, N, C, H, G, ctypes.c_float(eps), act, dtype, path, ws,
                                    bytes_, None)


@pytest.mark.parametrize("args,code", [
    (dict(N=17), eq.EQLIN_ERR_UNSUPPORTED), (dict(H=0), eq.EQLIN_ERR_INVALID_ARG), (dict(C=0), eq.EQLIN_ERR_INVALID_ARG),
    (dict(T=-1), eq.EQLIN_ERR_INVALID_ARG), (dict(G=5), eq.EQLIN_ERR_INVALID_ARG), (dict(G=-1), eq.EQLIN_ERR_INVALID_ARG),
    (dict(act=9), eq.EQLIN_ERR_INVALID_ARG), (dict(path=9), eq.EQLIN_ERR_INVALID_ARG), (dict(dtype=9), eq.EQLIN_ERR_UNSUPPORTED),
    (dict(path=eq.PATH_TC), eq.EQLIN_ERR_UNSUPPORTED),
    (dict(x=None), eq.EQLIN_ERR_INVALID_ARG), (dict(y=None), eq.EQLIN_ERR_INVALID_ARG), (dict(w2=None), eq.EQLIN_ERR_INVALID_ARG),
    (dict(x=MIS), eq.EQLIN_ERR_ALIGN), (dict(y=MIS), eq.EQLIN_ERR_ALIGN), (dict(w1=MIS), eq.EQLIN_ERR_ALIGN),
    (dict(gamma=MIS), eq.EQLIN_ERR_ALIGN), (dict(eps=-1.0), eq.EQLIN_ERR_INVALID_ARG),
    (dict(ws=None), eq.EQLIN_ERR_INVALID_ARG), (dict(ws=MIS), eq.EQLIN_ERR_ALIGN), (dict(bytes_=256), eq.EQLIN_ERR_SIZE),
])
def test_refusals(args, code):
    assert call(**args) == code and len(L.eqlin_last_error()) > 0


def test_no_tokens_and_sizes():
    assert call(x=None, y=None, w1=None, w2=None, ws=None, bytes_=0, T=0) == eq.EQLIN_OK
    need = L.eqlin_cyclic_gated_mlp_workspace_bytes
    assert need(9, 6, 12, 5, 3, 0) >= 9 * 6 * (12 + 5) * 4
    assert need(9, 6, 12, 5, 5, 0) == 0 and need(0, 6, 12, 5, 3, 0) == 0 and need(9, 17, 12, 5, 3, 0) == 0
    bad = L.eqlin_cyclic_gated_mlp_contract_spectrum
    assert bad(None, 6, 5, 12, 0, P, BIG, None) == eq.EQLIN_ERR_INVALID_ARG
    assert bad(P, 6, 5, 12, 0, P, 16, None) == eq.EQLIN_ERR_SIZE
    assert bad(MIS, 6, 5, 12, 0, P, BIG, None) == eq.EQLIN_ERR_ALIGN
    assert bad(P, 0, 5, 12, 0, P, BIG, None) == eq.EQLIN_ERR_UNSUPPORTED


def circulant(W):
    R, C, N = W.shape
    at = (torch.arange(N)[:, None] - torch.arange(N)[None, :]) % N
    return W[..., at.to(W.device)].permute(0, 2, 1, 3).reshape(R * N, C * N)


def reference(x, W1, W2, G, gamma, beta, act):
    T, C, N = x.shape
    H = W1.shape[0]
    x = x.double()
    if G:
        v = x.reshape(T, G, -1)
        d = v - v.mean(-1, keepdim=True)
        x = (d * ((d * d).mean(-1, keepdim=True) + 1e-5).rsqrt()).reshape(T, C, N)
        x = x * gamma.double()[:, None] + beta.double()[:, None]
    p = (x.reshape(T, -1) @ circulant(W1.double().reshape(2 * H, C, N)).t()).reshape(T, H, 2, N)
    g = p[:, :, 0]
    a = g * torch.sigmoid(g) if act == eq.ACT_SILU else 0.5 * g * (1 + torch.erf(g / math.sqrt(2)))
    return ((a * p[:, :, 1]).reshape(T, -1) @ circulant(W2.double()).t()).reshape(T, C, N)


def tensors(T, C, H, N, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    return ((r(T, C, N) * 2 + 0.5).to(dtype), (r(H, 2, C, N) / math.sqrt(C * N)).to(dtype),
            (r(C, H, N) / math.sqrt(H * N)).to(dtype), (1 + 0.2 * r(C)).to(dtype), (0.2 * r(C)).to(dtype))


CASES = [
    (1, 160, 432, 8, 1, torch.bfloat16, 3), (300, 160, 432, 8, 1, torch.bfloat16, 3), (2000, 48, 320, 8, 4, torch.bfloat16, 3),
    (77, 33, 50, 6, 3, torch.float32, 2), (129, 40, 96, 16, 0, torch.bfloat16, 3), (50, 24, 30, 4, 2, torch.float16, 2),
    (200, 64, 40, 12, 8, torch.float32, 2), (5, 700, 8, 8, 1, torch.float32, 2),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,C,H,N,G,dtype,halves", CASES)
def test_block(T, C, H, N, G, dtype, halves):
    x, W1, W2, gamma, beta = tensors(T, C, H, N, dtype)
    s1, s2 = eq.cyclic_gated_weight_spectrum(W1), eq.cyclic_gated_mlp_contract_spectrum(W2)
    for act in (eq.ACT_SILU, eq.ACT_GELU):
        y = torch.full_like(x, float("nan"))
        eq.cyclic_gated_mlp(x, s1, s2, H, groups=G, gamma=gamma, beta=beta, act=act, y=y)
        want = reference(x, W1, W2, G, gamma, beta, act)
        err = (y.double() - want).norm() / want.norm()
        assert err <= halves * torch.finfo(dtype).eps / 2 + 4e-6, float(err)
    assert eq.device_fault(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,C,H,N,G,dtype,halves", CASES[1:5])
def test_block_is_its_parts_and_replays(T, C, H, N, G, dtype, halves):
    """The block's kernels are the parts' own; a captured block replays on new inputs."""
    x, W1, W2, gamma, beta = tensors(T, C, H, N, dtype, 1)
    s1, s2 = eq.cyclic_gated_weight_spectrum(W1), eq.cyclic_gated_mlp_contract_spectrum(W2)
    y = eq.cyclic_gated_mlp(x, s1, s2, H, groups=G, gamma=gamma, beta=beta)
    n = eq.group_norm(x, G, gamma, beta)[0] if G else x
    h = eq.cyclic_gated_forward(n, s1, H)
    want = torch.einsum("tjh,cjgh->tcg", h.double(), circulant(W2.double()).reshape(C, N, H, N).permute(0, 2, 1, 3))
    err = (y.double() - want).norm() / want.norm()
    assert err <= 2 * torch.finfo(dtype).eps / 2 + 4e-6, float(err)
    xs = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = eq.cyclic_gated_mlp(xs, s1, s2, H, groups=G, gamma=gamma, beta=beta)
    xs.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y)


@pytest.mark.gpu
@pytest.mark.parametrize("T,C,H,N,dtype,tol", [(60, 24, 40, 6, torch.float32, 2e-5), (300, 32, 64, 8, torch.bfloat16, 2e-2)])
def test_a_training_step(T, C, H, N, dtype, tol):
    """Pre-norm and gated layer with their backward passes as one composite: gradients of sum(dh * gated(norm(x)))
    with respect to x, gamma, beta and W against autograd of the definition in 64 bits.  The chain carries the roundings
    of n, dp and dn beside its own parts': 5 half steps of bf16 at most."""
    x, W, _, gamma, beta = tensors(T, C, H, N, dtype, 2)
    dh = tensors(T, H, H, N, dtype, 3)[0]
    n, mean, rstd = eq.group_norm(x, 4, gamma, beta)
    spec, adj = eq.cyclic_gated_weight_spectrum(W), eq.cyclic_gated_weight_spectrum_adjoint(W)
    eq.cyclic_gated_forward(n, spec, H)
    dn, dW = eq.cyclic_gated_backward(n, dh, spec, adj)
    dx, dgamma, dbeta = eq.group_norm_backward(x, dn, mean, rstd, 4, gamma, beta)
    leaves = [t.double().requires_grad_() for t in (x, gamma, beta, W)]
    v = leaves[0].reshape(T, 4, -1)
    d = v - v.mean(-1, keepdim=True)
    nn = (d * ((d * d).mean(-1, keepdim=True) + 1e-5).rsqrt()).reshape(T, C, N)
    nn = nn * leaves[1][:, None] + leaves[2][:, None]
    p = (nn.reshape(T, -1) @ circulant(leaves[3].reshape(2 * H, C, N)).t()).reshape(T, H, 2, N)
    h = torch.nn.functional.silu(p[:, :, 0]) * p[:, :, 1]
    want = torch.autograd.grad(h, leaves, dh.double())
    for got, ref in zip((dx, dgamma, dbeta, dW), want):
        assert (got.double() - ref).norm() <= tol * ref.norm()
