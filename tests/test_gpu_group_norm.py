"""Group norm on a B200 against the definition in 64 bits, forward and backward.

Tolerances.  Inputs are rounded to their type first and both sides read the
same values.  An output is rounded once to its type: half a step, finfo.eps / 2
relative.  What comes before is fp32, each rounding half a step 2^-24:
  forward: (x - mean) rstd gamma + beta has 4 roundings of terms bounded by
  A = (|x| + |mean|) rstd |gamma| + |beta| + 1; mean and rstd carry the error
  of sums whose partials are joined over at most a few dozen steps each, and
  the activations' slopes are at most 1.13 with an own error below 4 steps of
  their value: 64 steps of A cover all of it.
  backward: dx is rstd times a sum of three terms bounded by
  D = max |dy gamma| 1.13 of the item (each mean is at most that) times (1 + |xhat|^2):
  again 64 steps of rstd D, where xhat itself is good to 4 steps of A.
  dgamma, dbeta: sums of n terms in fp32, partial sums of at most a few hundred
  terms in a row, then joined: their error is within 512 steps of sum |term| / sqrt(n)
  for terms of independent rounding errors; 64 steps of sum |term| are asserted,
  the worst case of the first joining.
"""

import math

import pytest
import torch

import group_wise_dft_b200 as eq

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24
ACTS = {"none": eq.ACT_NONE, "silu": eq.ACT_SILU, "gelu": eq.ACT_GELU}


def act64(name, z):
    if name == "silu":
        return z * torch.sigmoid(z), torch.sigmoid(z) * (1 + z * (1 - torch.sigmoid(z)))
    if name == "gelu":
        phi = 0.5 * (1 + torch.erf(z / math.sqrt(2)))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def reference(x, gamma, beta, G, eps, act):
    x = x.double()
    B, F, N = x.shape[0], x.shape[-2], x.shape[-1]
    v = x.reshape(B, -1, G, F // G * N)
    mean = v.mean(dim=(1, 3))
    rstd = ((v - mean[:, None, :, None]) ** 2).mean(dim=(1, 3)).add(eps).rsqrt()
    xh = ((v - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape)
    ga = gamma.double()[:, None] if gamma is not None else torch.ones(F, 1, dtype=torch.float64, device=x.device)
    be = beta.double()[:, None] if beta is not None else torch.zeros(F, 1, dtype=torch.float64, device=x.device)
    y, slope = act64(act, xh * ga + be)
    return y, mean, rstd, xh, ga, be, slope


def spread(stat, x, G):
    """[B, G] -> the shape of x."""
    B, F, N = x.shape[0], x.shape[-2], x.shape[-1]
    S = x.numel() // (B * F * N)
    return stat[:, None, :, None].expand(B, S, G, F // G * N).reshape(x.shape)


def check(x, G, gamma, beta, eps, act, dy=None):
    y, mean, rstd = eq.group_norm(x, G, gamma, beta, eps=eps, act=ACTS[act])
    ry, rmean, rrstd, xh, ga, be, slope = reference(x, gamma, beta, G, eps, act)
    half = torch.finfo(x.dtype).eps / 2
    xa = x.double().abs()
    top = xa.reshape(x.shape[0], -1, G, x.shape[-2] // G * x.shape[-1]).amax(dim=(1, 3))
    assert ((mean.double() - rmean).abs() <= 16 * STEP * (top + 1e-30)).all()
    # var + eps loses (mean error)^2 and 32 steps of itself
    assert ((rstd.double() / rrstd - 1).abs() <= 64 * STEP * (1 + (top * rrstd) ** 2 * STEP)).all()
    A = (xa + spread(rmean.abs(), x, G)) * spread(rrstd, x, G) * ga.abs() + be.abs() + 1
    err = (y.double() - ry).abs()
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0     # half a subnormal step
    assert (err <= half * ry.abs() + tiny + 64 * STEP * A).all(), (err - half * ry.abs() - 64 * STEP * A).max()
    if dy is None:
        return
    dx, dgamma, dbeta = eq.group_norm_backward(x, dy, mean, rstd, G, gamma, beta, act=ACTS[act])
    dz = dy.double() * slope
    n = xh.numel() // (x.shape[0] * G)

    def per_group(t):
        return spread(t.reshape(x.shape[0], -1, G, x.shape[-2] // G * x.shape[-1]).sum(dim=(1, 3)) / n, x, G)

    dn = dz * ga
    rdx = spread(rrstd, x, G) * (dn - per_group(dn) - xh * per_group(dn * xh))
    D = (1.13 * dy.double().abs() * ga.abs())
    D = spread(D.reshape(x.shape[0], -1, G, x.shape[-2] // G * x.shape[-1]).amax(dim=(1, 3)), x, G)
    bound = 64 * STEP * spread(rrstd, x, G) * D * (1 + xh ** 2) * (1 + A)
    err = (dx.double() - rdx).abs()
    assert (err <= half * rdx.abs() + tiny + bound).all(), (err - half * rdx.abs() - bound).max()
    over = tuple(d for d in range(x.dim()) if d != x.dim() - 2)
    for got, term in ((dgamma, dz * xh), (dbeta, dz)):
        want = term.sum(dim=over)
        bound = 64 * STEP * ((dy.double() * 1.13).abs() * (1 + xh.abs()) * A).sum(dim=over)
        assert ((got.double() - want).abs() <= half * want.abs() + tiny + bound).all()


def tensors(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    F = shape[-2]

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda")

    x = (r(*shape) * scale + shift).to(dtype)
    return x, (r(F) * 0.3 + 1).to(dtype), (r(F) * 0.3).to(dtype), r(*shape).to(dtype)


TYPES = [torch.float32, torch.bfloat16, torch.float16]


# tokens and tiny maps (one warp an item): every vector width, fields that share a vector, groups of every size
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,G", [
    ((1, 160, 8), 1), ((77, 160, 8), 1), ((5, 160, 8), 32), ((9, 160, 8), 5), ((33, 96, 6), 16), ((7, 64, 4), 8),
    ((130, 40, 12), 40), ((3, 37, 3), 37), ((6, 7, 5), 1), ((4, 3, 7), 3), ((5, 1, 16), 1), ((2, 1, 1), 1),
    ((2001, 8, 8), 2), ((11, 3, 3, 10, 8), 5), ((6, 2, 3, 9, 2), 3), ((5, 17, 16, 1), 4), ((3, 130, 13), 1),
])
def test_rows(shape, G, dtype):
    x, gamma, beta, dy = tensors(shape, dtype, 1)
    for act in ACTS:
        check(x, G, gamma, beta, 1e-5, act, dy)


# items of 2 to 16 warps (wide tokens, small maps): each count of warps at its ends, fields that share a vector, more
# items than run at once, and the first sizes past the widest
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,G", [
    ((7, 161, 8), 1), ((5, 320, 8), 32), ((3001, 321, 8), 1), ((4, 640, 8), 4), ((650, 641, 8), 1), ((3, 1280, 8), 5),
    ((2, 1281, 8), 1), ((301, 10, 160, 8), 8), ((2, 2560, 8), 2560 // 8), ((2, 2561, 8), 1), ((9, 3, 96, 12), 8),
    ((33, 4, 80, 6), 1), ((5, 7, 80, 6), 20), ((6, 2, 1000, 3), 1), ((5, 1, 1500, 4), 1), ((4, 768, 8), 768),
    ((3, 1900, 3), 1), ((3, 2000, 2), 500),
    ((3, 6000, 1), 1), ((3, 6008, 1), 1), ((5, 2000, 3), 1), ((3, 2008, 3), 1), ((2, 768, 8), 2), ((2, 1200, 16), 3),
])
def test_items_of_several_warps(shape, G, dtype):
    x, gamma, beta, dy = tensors(shape, dtype, 14)
    for act in ("none", "silu", "gelu"):
        check(x, G, gamma, beta, 1e-5, act, dy)


def test_items_of_several_warps_repeat_and_stay_in_bounds():
    for shape, G in [((2500, 400, 8), 1), ((1500, 400, 8), 16), ((400, 9, 100, 8), 4), ((40, 2500, 8), 1)]:
        x, gamma, beta, dy = tensors(shape, torch.bfloat16, 15)
        n = x.numel()
        guard = torch.full((n + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
        y = guard[256:256 + n].view(shape)
        first = [t.clone() for t in eq.group_norm(x, G, gamma, beta, y=y)]
        grads = [t.clone() for t in eq.group_norm_backward(x, dy, first[1], first[2], G, gamma, beta, dx=y)]
        for _ in range(3):
            for a, b in zip(eq.group_norm(x, G, gamma, beta, y=y), first):
                assert torch.equal(a, b)
            for a, b in zip(eq.group_norm_backward(x, dy, first[1], first[2], G, gamma, beta, dx=y), grads):
                assert torch.equal(a, b)
        assert (guard[:256] == 7).all() and (guard[256 + n:] == 7).all()


# maps in chunks: ragged positions, odd groups and slots, positions wider than a CTA, one position only
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,G", [
    ((3, 31, 33, 160, 8), 32), ((2, 1000, 160, 8), 1), ((2, 57, 55, 96, 6), 16), ((1, 99, 101, 64, 4), 8),
    ((5, 333, 15, 3), 5), ((2, 700, 7, 5), 7), ((4, 129, 13, 16), 13), ((1, 5000, 1, 1), 1), ((9, 1, 700, 8), 4),
    ((2, 3, 1200, 12), 3), ((1, 2, 5000, 3), 1), ((1, 2, 3000, 16), 500), ((260, 60, 24, 8), 3),
])
def test_maps(shape, G, dtype):
    x, gamma, beta, dy = tensors(shape, dtype, 2)
    for act in ("none", "silu", "gelu"):
        check(x, G, gamma, beta, 1e-5, act, dy)


@pytest.mark.parametrize("shape,G", [((64, 40, 8), 4), ((2, 900, 40, 8), 4)])
def test_level_far_from_zero(shape, G):
    """A mean 3000 times the spread: sums of squares would cancel, running deviations do not."""
    x, gamma, beta, dy = tensors(shape, torch.float32, 3, scale=1.0, shift=3000.0)
    check(x, G, gamma, beta, 1e-5, "silu", dy)


@pytest.mark.parametrize("shape,G", [((6, 40, 8), 4), ((2, 900, 40, 8), 4)])
def test_an_outlier_in_first_place(shape, G):
    x, gamma, beta, dy = tensors(shape, torch.float32, 4)
    x.view(x.shape[0], -1)[:, 0] = 1.0e4
    check(x, G, gamma, beta, 1e-5, "none", dy)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,G", [((6, 40, 8), 4), ((2, 900, 40, 8), 4)])
def test_constant_input(shape, G, dtype):
    """No variance: xhat is 0 and rstd 1 / sqrt(eps)."""
    x, gamma, beta, dy = tensors(shape, dtype, 5)
    x.fill_(2.5)
    y, mean, rstd = eq.group_norm(x, G, gamma, beta, eps=1e-4)
    assert (mean == 2.5).all()
    assert ((rstd - 100.0).abs() <= 100 * 8 * STEP).all()
    assert torch.equal(y, beta[:, None].expand_as(y).contiguous())


@pytest.mark.parametrize("shape,G", [((6, 40, 8), 4), ((3, 900, 40, 8), 4)])
def test_nan_and_infinity_stay_in_their_group(shape, G):
    x, gamma, beta, dy = tensors(shape, torch.bfloat16, 6)
    clean = eq.group_norm(x, G, gamma, beta, act=eq.ACT_SILU)[0]
    bad = x.clone()
    v = bad.view(x.shape[0], -1, 40, 8)
    v[0, 0, 3, 2] = float("nan")      # item 0, group 0
    v[1, -1, 39, 7] = float("inf")    # item 1, group 3
    y = eq.group_norm(bad, G, gamma, beta, act=eq.ACT_SILU)[0].view(x.shape[0], -1, G, 10 * 8)
    assert y[0, :, 0].isnan().all() and y[1, :, 3].isnan().all()
    ok = torch.ones(x.shape[0], G, dtype=torch.bool)
    ok[0, 0] = ok[1, 3] = False
    want = clean.view_as(y)
    for b in range(x.shape[0]):
        for g in range(G):
            if ok[b, g]:
                assert torch.equal(y[b, :, g], want[b, :, g])


@pytest.mark.parametrize("shape,G", [((50, 24, 8), 3), ((2, 700, 24, 8), 3)])
def test_without_gamma_and_beta(shape, G):
    x, gamma, beta, dy = tensors(shape, torch.float32, 7)
    one, zero = torch.ones_like(gamma), torch.zeros_like(beta)
    for a, b in ((None, None), (gamma, None), (None, beta)):
        y, mean, rstd = eq.group_norm(x, G, a, b, act=eq.ACT_GELU)
        aa, bb = one if a is None else a, zero if b is None else b
        assert torch.equal(y, eq.group_norm(x, G, aa, bb, act=eq.ACT_GELU)[0])
        dx, dg, db = eq.group_norm_backward(x, dy, mean, rstd, G, a, b, act=eq.ACT_GELU)
        ex, eg, eb = eq.group_norm_backward(x, dy, mean, rstd, G, aa, bb, act=eq.ACT_GELU)
        assert torch.equal(dx, ex)
        assert (dg is None) == (a is None) and (db is None) == (b is None)
        if a is not None:
            assert torch.equal(dg, eg)
        if b is not None:
            assert torch.equal(db, eb)


@pytest.mark.parametrize("shape", [(0, 16, 8), (3, 0, 16, 8)])
def test_no_values(shape):
    x = torch.empty(shape, device="cuda")
    ga = torch.ones(16, device="cuda")
    y, mean, rstd = eq.group_norm(x, 4, ga, ga)
    assert y.shape == x.shape
    m = torch.zeros(shape[0], 4, device="cuda")
    dx, dg, db = eq.group_norm_backward(x, x, m, m, 4, ga, ga)
    assert (dg == 0).all() and (db == 0).all()


@pytest.mark.parametrize("shape,G", [((40, 24, 8), 3), ((2, 300, 24, 8), 3)])
def test_equivariance(shape, G):
    """Permuting the slots (C_8 shifts among the permutations) permutes the outputs; fp32 rounding of the sums aside."""
    x, gamma, beta, _ = tensors(shape, torch.float32, 8)
    y = eq.group_norm(x, G, gamma, beta, act=eq.ACT_SILU)[0]
    for s in (1, 3):
        ys = eq.group_norm(x.roll(s, -1).contiguous(), G, gamma, beta, act=eq.ACT_SILU)[0]
        assert ((ys - y.roll(s, -1)).abs() <= 64 * STEP * (1 + y.roll(s, -1).abs())).all()


@pytest.mark.parametrize("shape,G", [((300, 40, 8), 4), ((3, 900, 40, 8), 4)])
def test_repeats_bit_for_bit_and_stays_in_bounds(shape, G):
    x, gamma, beta, dy = tensors(shape, torch.bfloat16, 9)
    n = x.numel()
    guard = torch.full((n + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = guard[256:256 + n].view(shape)
    _, mean, rstd = eq.group_norm(x, G, gamma, beta, y=y)
    assert (guard[:256] == 7).all() and (guard[256 + n:] == 7).all()
    first = eq.group_norm_backward(x, dy, mean, rstd, G, gamma, beta)
    guard.fill_(7.0)
    again = eq.group_norm_backward(x, dy, mean, rstd, G, gamma, beta, dx=y)
    assert (guard[:256] == 7).all() and (guard[256 + n:] == 7).all()
    for a, b in zip(first, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shape,G", [((64, 40, 8), 4), ((2, 900, 40, 8), 4)])
def test_other_stream_and_graph(shape, G):
    x, gamma, beta, dy = tensors(shape, torch.bfloat16, 10)
    want = eq.group_norm(x, G, gamma, beta, act=eq.ACT_SILU)
    grads = eq.group_norm_backward(x, dy, want[1], want[2], G, gamma, beta, act=eq.ACT_SILU)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = eq.group_norm(x, G, gamma, beta, act=eq.ACT_SILU)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    xs = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = eq.group_norm(xs, G, gamma, beta, act=eq.ACT_SILU)
        back = eq.group_norm_backward(xs, dy, out[1], out[2], G, gamma, beta, act=eq.ACT_SILU)
    for _ in range(2):
        xs.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out + back, want + grads):
            assert torch.equal(a, b)
        xs.zero_()
        g.replay()


@pytest.mark.parametrize("shape,G", [((6, 8, 6), 2), ((2, 150, 10, 6), 5)])
def test_gradient_against_differences(shape, G):
    """Central differences of the 64-bit formula, step 1e-4: their error is O(step^2)."""
    x, gamma, beta, dy = tensors(shape, torch.float32, 11)
    _, mean, rstd = eq.group_norm(x, G, gamma, beta, act=eq.ACT_GELU)
    dx, dg, db = eq.group_norm_backward(x, dy, mean, rstd, G, gamma, beta, act=eq.ACT_GELU)
    gen = torch.Generator(device="cuda").manual_seed(12)
    for k, grad in enumerate((dx, dg, db)):
        args = [x.double(), gamma.double(), beta.double()]
        d = torch.randn(args[k].shape, generator=gen, device="cuda", dtype=torch.float64)

        def value(e):
            a = list(args)
            a[k] = a[k] + e * d
            return (reference(a[0], a[1], a[2], G, 1e-5, "gelu")[0] * dy.double()).sum()

        want = (value(1e-4) - value(-1e-4)) / 2e-4
        scale = (grad.double() * d).abs().sum()
        assert abs((grad.double() * d).sum() - want) <= 1e-5 * scale


def test_offsets_past_32_bits():
    """More than 2^31 values: the last item is normalised as it is alone."""
    B, S, F, N = 3, 90000, 1000, 8          # 2.16e9 values, 4.3 GB in bf16
    x = torch.zeros(B, S, F, N, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(13)
    x[-1] = torch.randn(S, F, N, generator=gen, device="cuda", dtype=torch.bfloat16)
    y, mean, rstd = eq.group_norm(x, 10)
    ref = reference(x[-1:, -8:], None, None, 10, 1e-5, "none")     # shape only
    m = x[-1].view(S, 10, -1).double().mean(dim=(0, 2))
    assert ((mean[-1].double() - m).abs() <= 16 * STEP * 5).all()
    part = x[-1, -8:].view(8, 10, -1).double()
    want = (part - m[None, :, None]) * rstd[-1].double()[None, :, None]
    got = y[-1, -8:].view(8, 10, -1).double()
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 64 * STEP * 10).all()
    assert ref[0].shape == (1, 8, F, N)
    dx, _, _ = eq.group_norm_backward(x, x, mean, rstd, 10)
    assert (dx[0] == 0).all() and dx[-1].isfinite().all()
    del x, y, dx
    torch.cuda.empty_cache()
