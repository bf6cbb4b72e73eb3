"""The gated layer as programs call it on a B200: streams side by side, one captured graph beside another, tokens that
hold NaN or infinity, batches past 2^31 values, and a backward pass captured while an eager one's results live."""

import math

import pytest
import torch

import group_wise_dft_b200 as eq

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16

# T, C, H, N, dtype, path: the few-token and the tile kernel, the two-pass products, the fused C_8 kernel
FORMS = [
    (7, 24, 20, 6, F32, eq.PATH_AUTO), (150, 24, 20, 6, BF16, eq.PATH_SIMT), (700, 48, 40, 12, BF16, eq.PATH_TC),
    (900, 24, 40, 5, F16, eq.PATH_TC), (6500, 32, 48, 8, BF16, eq.PATH_TC),
]


def tensors(T, C, H, N, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda")

    return r(T, C, N).to(dtype), (r(H, 2, C, N) / math.sqrt(C * N)).to(dtype), r(T, H, N).to(dtype)


def both(x, W, dh, path):
    spec, adj = eq.cyclic_gated_weight_spectrum(W), eq.cyclic_gated_weight_spectrum_adjoint(W)
    h = eq.cyclic_gated_forward(x, spec, W.shape[0], path=path)
    return (h, *eq.cyclic_gated_backward(x, dh, spec, adj, path=path))


@pytest.mark.parametrize("T,C,H,N,dtype,path", FORMS)
def test_calls_on_two_streams_at_once(T, C, H, N, dtype, path):
    sets = [tensors(T, C, H, N, dtype, s) for s in (1, 2)]
    want = [both(*s, path) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(4):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(both(*sets[k], path))
    torch.cuda.synchronize()
    for k in range(2):
        for run in got[k]:
            for a, b in zip(run, want[k]):
                assert torch.equal(a, b)
    assert eq.device_fault(reset=True) == 0


@pytest.mark.parametrize("T,C,H,N,dtype,path", FORMS)
def test_two_graphs_replayed_side_by_side(T, C, H, N, dtype, path):
    """Each capture has its own workspaces; an eager call's results live on meanwhile."""
    sets = [tensors(T, C, H, N, dtype, s) for s in (3, 4)]
    want = [both(*s, path) for s in sets]
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both(*s, path))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, ref in zip(outs, want):
        for a, b in zip(out, ref):
            assert torch.equal(a, b)
    assert eq.device_fault(reset=True) == 0


@pytest.mark.parametrize("T,C,H,N,dtype,path", FORMS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_and_infinity_stay_in_their_token(T, C, H, N, dtype, path, bad):
    x, W, dh = tensors(T, C, H, N, dtype, 5)
    clean = both(x, W, dh, path)
    x[T // 2, C - 1, 0] = bad
    got = both(x, W, dh, path)
    others = torch.arange(T, device="cuda") != T // 2
    for k in (0, 1):
        assert torch.equal(got[k][others], clean[k][others])
        assert not got[k][T // 2].isfinite().any()
    assert eq.device_fault(reset=True) == 0


# more than 2^31 values of x; only the last tokens are not zero, so that their results, and the weight
# gradient, are those of a short call
@pytest.mark.parametrize("T,C,H,N,dtype,path", [
    ((1 << 23) + 77, 128, 16, 4, BF16, eq.PATH_TC), ((1 << 24) + 133, 16, 16, 8, BF16, eq.PATH_TC),
    ((1 << 23) + 77, 64, 8, 4, F32, eq.PATH_AUTO),
])
def test_offsets_past_32_bits(T, C, H, N, dtype, path):
    tail = 200
    x, W, dh = tensors(tail, C, H, N, dtype, 6)
    want = both(x, W, dh, path)
    X = torch.zeros(T, C, N, dtype=dtype, device="cuda")
    D = torch.zeros(T, H, N, dtype=dtype, device="cuda")
    X[-tail:] = x
    D[-tail:] = dh
    assert X.numel() > 1 << 31
    h, dx, dW = both(X, W, D, path)
    # another order of the fp32 sums, so a value may round to its neighbour: a step of the value, or
    # of fp32 where sums cancel
    step = torch.finfo(dtype).eps
    for got, ref in ((h[-tail:], want[0]), (dx[-tail:], want[1]), (dW, want[2])):
        top = ref.float().abs().max()
        # (the intermediate roundings of dp and of the spectra may differ by a step as well)
        assert ((got.float() - ref.float()).abs() <= 4 * step * ref.float().abs() + (4 * step + 1e-5) * top).all()
    assert not h[:-tail].any() and not dx[:-tail].any()
    assert eq.device_fault(reset=True) == 0
    del X, D, h, dx
    torch.cuda.empty_cache()
