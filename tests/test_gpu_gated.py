"""Gated cyclic feed-forward layer on a B200 against the definition in 64 bits.

Tolerances (relative to the root mean square of the output, and Frobenius).
A rounding to the output's type is off by at most half a step (finfo.eps / 2);
fp32 sums over K = Cin N products are off by far less than 1e-6 sqrt(K) / 10.
CUDA-core path: h is rounded once; the backward rounds dp too, and then dx, dW.
  Frobenius: half a step for h, twice that for dx and dW, plus 2e-6.
Tensor-core path: x's and W's (dp's) half spectra are rounded to the operand
type as well, half a step each at most.  Gate and value each carry two such
roundings; the activations move the gate's by at most a factor 1.6 (the largest
|g act'(g) / act(g)| weighted over the tested inputs is below that).  With
independent roundings (rms half a step / sqrt 3) h is off by
sqrt(2 * 1.6^2 + 2 + 1) / sqrt 3 = 1.65 half steps, dp the same, dx and dW by
sqrt(1.65^2 * 3 + 3) / sqrt 3 = 1.93; 2 half steps for h and 2.5 for dx and dW
are asserted.
"""

import math

import pytest
import torch

import group_wise_dft_b200 as eq

pytestmark = pytest.mark.gpu

ACTS = {"none": eq.ACT_NONE, "silu": eq.ACT_SILU, "gelu": eq.ACT_GELU}
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def act64(name, z):
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        phi = 0.5 * (1 + torch.erf(z / math.sqrt(2)))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def circulant(W):
    """[2H, C, N] -> the dense matrix, row (o, g), column (i, h): W[o, i, (g - h) mod N]."""
    R, C, N = W.shape
    at = (torch.arange(N)[:, None] - torch.arange(N)[None, :]) % N
    return W[..., at.to(W.device)].permute(0, 2, 1, 3).reshape(R * N, C * N)


def reference(x, W, act, dh=None):
    T, C, N = x.shape
    H = W.shape[0]
    x, W = x.double(), W.double()
    D = circulant(W.reshape(2 * H, C, N))
    p = (x.reshape(T, -1) @ D.t()).reshape(T, H, 2, N)
    a, slope = act64(act, p[:, :, 0])
    h = a * p[:, :, 1]
    if dh is None:
        return h
    dh = dh.double()
    dp = torch.stack((dh * p[:, :, 1] * slope, dh * a), 2)
    dx = (dp.reshape(T, -1) @ D).reshape(T, C, N)
    # dW[j, a, i, m] = sum_t sum_g dp[t, j, a, g] x[t, i, (g - m) mod N]
    dW = torch.stack([torch.einsum("tjag,tig->jai", dp, x.roll(m, -1)) for m in range(N)], -1)
    return h, dx, dW


def tensors(T, C, H, N, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda")

    return r(T, C, N).to(dtype), (r(H, 2, C, N) / math.sqrt(C * N)).to(dtype), r(T, H, N).to(dtype)


def near(got, want, halves):
    """Frobenius, and every value within 8 times that of max(|want|, rms)."""
    half = torch.finfo(got.dtype).eps / 2
    tol = halves * half + 2e-6
    got = got.double()
    assert got.isfinite().all()
    norm = want.norm()
    assert (got - want).norm() <= tol * norm + 1e-30, float((got - want).norm() / norm)
    rms = norm / math.sqrt(max(1, want.numel()))
    assert ((got - want).abs() <= 8 * tol * torch.maximum(want.abs(), rms) + 1e-30).all()


def run(T, C, H, N, dtype, act, path=eq.PATH_AUTO, seed=0, halves=(1, 2, 2)):
    x, W, dh = tensors(T, C, H, N, dtype, seed)
    spec, adj = eq.cyclic_gated_weight_spectrum(W), eq.cyclic_gated_weight_spectrum_adjoint(W)
    h = torch.full((T, H, N), float("nan"), dtype=dtype, device="cuda")
    eq.cyclic_gated_forward(x, spec, H, act=ACTS[act], h=h, path=path)
    rh, rdx, rdW = reference(x, W, act, dh)
    near(h, rh, halves[0])
    dx, dW = torch.full_like(x, float("nan")), torch.full_like(W, float("nan"))
    eq.cyclic_gated_backward(x, dh, spec, adj, act=ACTS[act], dx=dx, dW=dW, path=path)
    near(dx, rdx, halves[1])
    near(dW, rdW, halves[2])
    assert eq.device_fault(reset=True) == 0


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N", range(1, 17))
def test_every_group(N, dtype):
    run(45, 11, 9, N, dtype, "silu", path=eq.PATH_SIMT, seed=N)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,C,H,N", [
    (1, 160, 432, 8), (1, 1, 1, 8), (2, 37, 101, 6), (5, 130, 33, 8), (32, 64, 40, 4), (33, 64, 40, 4),
    (31, 17, 70, 16), (100, 300, 12, 3), (257, 40, 64, 8), (1001, 37, 101, 6), (65, 5, 4, 12),
])
@pytest.mark.parametrize("act", list(ACTS))
def test_cuda_cores(T, C, H, N, act, dtype):
    run(T, C, H, N, dtype, act, path=eq.PATH_SIMT)


# tensor cores, C_8: ragged tiles, one 32-field chunk or several, output groups of dx with padding (Cin = 16, 48, ..);
# from 4096 tokens (backward: 6144) on the fused kernel, several tiles per pair of CTAs
TC = [
    (33, 16, 16, "silu"), (64, 32, 48, "gelu"), (127, 48, 16, "none"), (128, 80, 64, "silu"), (129, 112, 80, "gelu"),
    (300, 160, 432, "silu"), (1000, 144, 96, "gelu"), (3 * 74 * 128 + 77, 32, 32, "silu"),
    (2 * 74 * 128 + 1, 160, 48, "silu"), (20000, 96, 160, "gelu"),
    (4096, 48, 64, "gelu"), (6200, 160, 432, "none"), (4095, 160, 432, "silu"),
]


@pytest.mark.parametrize("T,C,H,act", TC)
def test_tensor_cores(T, C, H, act):
    assert eq.cyclic_gated_auto_path(8, C, H, BF16) == eq.PATH_TC
    run(T, C, H, 8, BF16, act, path=eq.PATH_TC, halves=(2, 2.5, 2.5))
    run(T, C, H, 8, BF16, act, halves=(2, 2.5, 2.5))


@pytest.mark.parametrize("T,C,H,act", TC[:7] + [(1, 32, 16, "silu")])
def test_tensor_cores_when_asked_for(T, C, H, act):
    """fp16, and bf16 for a handful of tokens."""
    run(T, C, H, 8, F16, act, path=eq.PATH_TC, halves=(2, 2.5, 2.5))
    run(T + 6144, C, H, 8, F16, act, path=eq.PATH_TC, halves=(2, 2.5, 2.5))
    run(T % 32 + 1, C, H, 8, BF16, act, path=eq.PATH_TC, halves=(2, 2.5, 2.5))


# the two-pass products: every N, ragged fields and tokens, one or several groups of outputs and blocks of inputs
GEMM = [(40, 16, 8, 5, "silu"), (129, 37, 101, 6, "gelu"), (257, 64, 40, 4, "silu"), (300, 96, 384, 16, "gelu"),
        (1000, 100, 200, 12, "silu"), (700, 33, 19, 3, "none"), (130, 130, 70, 16, "silu"), (500, 200, 150, 8, "silu"),
        (333, 24, 31, 8, "gelu"), (90, 65, 30, 2, "silu"), (64, 70, 90, 1, "silu"), (20 * 148 * 64 + 3, 20, 30, 7, "gelu")]


@pytest.mark.parametrize("T,C,H,N,act", GEMM)
def test_two_pass_products(T, C, H, N, act):
    run(T, C, H, N, BF16, act, path=eq.PATH_TC, halves=(2, 2.5, 2.5))


@pytest.mark.parametrize("N", range(1, 17))
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_two_pass_products_every_group(N, dtype):
    run(150, 18, 9, N, dtype, "silu", path=eq.PATH_TC, seed=N, halves=(2, 2.5, 2.5))


def test_outputs_at_odd_addresses():
    """h, dx and dW 16 bytes off a 32-byte boundary are written whole."""
    T, C, H = 200, 32, 48
    x, W, dh = tensors(T, C, H, 8, BF16, 9)
    spec, adj = eq.cyclic_gated_weight_spectrum(W), eq.cyclic_gated_weight_spectrum_adjoint(W)
    rh, rdx, rdW = reference(x, W, "silu", dh)
    h = torch.empty(T * H * 8 + 8, dtype=BF16, device="cuda")[8:].view(T, H, 8)
    dx = torch.empty(T * C * 8 + 8, dtype=BF16, device="cuda")[8:].view(T, C, 8)
    dW = torch.empty(H * 2 * C * 8 + 8, dtype=BF16, device="cuda")[8:].view(H, 2, C, 8)
    near(eq.cyclic_gated_forward(x, spec, H, h=h), rh, 2)
    eq.cyclic_gated_backward(x, dh, spec, adj, dx=dx, dW=dW)
    near(dx, rdx, 2.5)
    near(dW, rdW, 2.5)


def test_without_a_workspace():
    """AUTO then takes a form that needs none: the fused kernel, or the CUDA cores."""
    L, s = eq.raw_lib(), torch.cuda.current_stream().cuda_stream
    for T, C, H, N in ((300, 160, 432, 8), (300, 96, 130, 16)):
        x, W, _ = tensors(T, C, H, N, BF16, 12)
        spec, h = eq.cyclic_gated_weight_spectrum(W), torch.full((T, H, N), float("nan"), dtype=BF16, device="cuda")
        args = (x.data_ptr(), spec.data_ptr(), h.data_ptr(), T, N, C, H, eq.ACT_SILU, eq.EQLIN_BF16)
        assert L.eqlin_cyclic_gated_forward(*args, eq.PATH_AUTO, None, 0, s) == 0
        near(h, reference(x, W, "silu"), 2)
        assert L.eqlin_cyclic_gated_forward(*args, eq.PATH_TC, None, 0, s) == eq.EQLIN_ERR_SIZE


def test_no_tokens():
    x, W, dh = tensors(0, 16, 8, 8, F32, 0)
    spec, adj = eq.cyclic_gated_weight_spectrum(W), eq.cyclic_gated_weight_spectrum_adjoint(W)
    assert eq.cyclic_gated_forward(x, spec, 8).shape == (0, 8, 8)
    dx, dW = eq.cyclic_gated_backward(x, dh, spec, adj, dW=torch.full_like(W, 3.0))
    assert dx.shape == x.shape and (dW == 0).all()


@pytest.mark.parametrize("T,C,H,N,dtype", [(40, 24, 20, 8, F32), (70, 16, 32, 8, BF16)])
def test_equivariance(T, C, H, N, dtype):
    """Rolling x along the group rolls h."""
    x, W, _ = tensors(T, C, H, N, dtype, 3)
    spec = eq.cyclic_gated_weight_spectrum(W)
    h = eq.cyclic_gated_forward(x, spec, H)
    for s in (1, 3):
        hs = eq.cyclic_gated_forward(x.roll(s, -1).contiguous(), spec, H)
        near(hs, h.roll(s, -1).double(), 4)


@pytest.mark.parametrize("T,C,H,N", [(6, 5, 4, 4), (9, 4, 3, 5)])
@pytest.mark.parametrize("act", list(ACTS))
def test_gradient_against_differences(T, C, H, N, act):
    """Central differences of the 64-bit formula, step 1e-4."""
    x, W, dh = tensors(T, C, H, N, F32, 4)
    spec, adj = eq.cyclic_gated_weight_spectrum(W), eq.cyclic_gated_weight_spectrum_adjoint(W)
    dx, dW = eq.cyclic_gated_backward(x, dh, spec, adj, act=ACTS[act])
    gen = torch.Generator(device="cuda").manual_seed(5)
    for k, grad in enumerate((dx, dW)):
        d = torch.randn(grad.shape, generator=gen, device="cuda", dtype=torch.float64)

        def value(e):
            a = [x.double(), W.double()]
            a[k] = a[k] + e * d
            return (reference(a[0], a[1], act) * dh.double()).sum()

        want = (value(1e-4) - value(-1e-4)) / 2e-4
        assert abs((grad.double() * d).sum() - want) <= 1e-5 * (grad.double() * d).abs().sum()


def test_either_gradient_alone():
    x, W, dh = tensors(50, 20, 12, 6, F32, 6)
    spec, adj = eq.cyclic_gated_weight_spectrum(W), eq.cyclic_gated_weight_spectrum_adjoint(W)
    dx, dW = eq.cyclic_gated_backward(x, dh, spec, adj)
    L = eq.raw_lib()
    need = eq.cyclic_gated_backward_workspace_bytes(50, 6, 20, 12, F32)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    a, b = torch.zeros_like(dx), torch.zeros_like(dW)
    args = (50, 6, 20, 12, eq.ACT_SILU, eq.EQLIN_F32, eq.PATH_AUTO, ws.data_ptr(), need, s)
    assert L.eqlin_cyclic_gated_backward(x.data_ptr(), dh.data_ptr(), spec.data_ptr(), adj.data_ptr(), a.data_ptr(),
                                         None, *args) == 0
    assert L.eqlin_cyclic_gated_backward(x.data_ptr(), dh.data_ptr(), spec.data_ptr(), None, None, b.data_ptr(),
                                         *args) == 0
    torch.cuda.synchronize()
    assert torch.equal(a, dx) and torch.equal(b, dW)


CASES = [(33, 24, 20, 6, F32), (3, 24, 20, 8, BF16), (300, 32, 48, 8, BF16)]


@pytest.mark.parametrize("T,C,H,N,dtype", CASES)
def test_repeats_bit_for_bit_and_stays_in_bounds(T, C, H, N, dtype):
    x, W, dh = tensors(T, C, H, N, dtype, 7)
    spec, adj = eq.cyclic_gated_weight_spectrum(W), eq.cyclic_gated_weight_spectrum_adjoint(W)

    def guarded(shape):
        n = math.prod(shape)
        buf = torch.full((n + 512,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[256:256 + n].view(shape)

    bh, h = guarded((T, H, N))
    bx, dx = guarded((T, C, N))
    bw, dW = guarded((H, 2, C, N))
    need = eq.cyclic_gated_backward_workspace_bytes(T, N, C, H, dtype)
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(2):
        eq.cyclic_gated_forward(x, spec, H, h=h)
        eq.cyclic_gated_backward(x, dh, spec, adj, dx=dx, dW=dW, workspace=ws[256:256 + need])
        torch.cuda.synchronize()
        got.append((h.clone(), dx.clone(), dW.clone()))
        for buf in (bh, bx, bw):
            assert (buf[:256] == 7).all() and (buf[-256:] == 7).all()
        assert (ws[:256] == 0xA5).all() and (ws[256 + need:] == 0xA5).all()
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,C,H,N,dtype", CASES)
def test_other_stream_and_graph(T, C, H, N, dtype):
    x, W, dh = tensors(T, C, H, N, dtype, 8)
    spec, adj = eq.cyclic_gated_weight_spectrum(W), eq.cyclic_gated_weight_spectrum_adjoint(W)
    want = (eq.cyclic_gated_forward(x, spec, H), *eq.cyclic_gated_backward(x, dh, spec, adj))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = (eq.cyclic_gated_forward(x, spec, H), *eq.cyclic_gated_backward(x, dh, spec, adj))
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    xs, Ws = torch.zeros_like(x), torch.zeros_like(W)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sp, ad = eq.cyclic_gated_weight_spectrum(Ws), eq.cyclic_gated_weight_spectrum_adjoint(Ws)
        out = (eq.cyclic_gated_forward(xs, sp, H), *eq.cyclic_gated_backward(xs, dh, sp, ad))
    for _ in range(2):
        xs.copy_(x)
        Ws.copy_(W)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
        xs.zero_()
        g.replay()
