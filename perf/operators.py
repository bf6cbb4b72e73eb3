"""The channels-last group norm and the gated cyclic feed-forward layer as workloads: inputs, a plain form in
elementary torch operations, the library's calls, and the definitions in 64 bits.

An activation is x[..., F, N]: F fields of N group slots, the slot fastest.

Group norm ("norm", "norm_grad"): x[B, S, F, N], G groups of F / G fields.  Mean and (biased) variance over each
(item, group), y = act(gamma[f] * (x - mean) * rstd + beta[f]).  The gradient takes the saved mean and rstd.

Gated layer ("gated", "gated_grad"): x[T, C, N], W[H, 2, C, N] (row (j, 0) the gate, (j, 1) the value),
    p[t, j, a, g] = sum_i sum_h W[j, a, i, (g - h) mod N] x[t, i, h],    h = act(p[:, :, 0]) * p[:, :, 1].
The gradient takes dh and gives dx and dW.
"""

import math

import torch

own = False

_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one decoded token's pre-norm: launch latency
        {"name": "norm_one_token", "op": "norm", "type": "bf16", "B": 1, "S": 1, "F": 160, "N": 8, "G": 1, "act": "none"},
        # the pre-norm of a large batch of ViT-H-wide tokens
        {"name": "norm_tokens", "op": "norm", "type": "bf16", "B": 131072, "S": 1, "F": 160, "N": 8, "G": 1, "act": "none"},
        # feature maps of 32 x 32 positions between two equivariant layers
        {"name": "norm_maps", "op": "norm", "type": "bf16", "B": 64, "S": 1024, "F": 160, "N": 8, "G": 32, "act": "silu"},
        # a few large p4 maps with a ragged number of positions, fp32
        {"name": "norm_large_p4_maps", "op": "norm", "type": "fp32", "B": 3, "S": 99 * 101, "F": 64, "N": 4, "G": 8, "act": "gelu"},
        # a training step's backward: tokens
        {"name": "norm_grad_tokens", "op": "norm_grad", "type": "bf16", "B": 65536, "S": 1, "F": 160, "N": 8, "G": 1, "act": "none"},
        # and maps, with an odd group and an odd number of positions
        {"name": "norm_grad_maps", "op": "norm_grad", "type": "fp16", "B": 24, "S": 57 * 55, "F": 96, "N": 6, "G": 16, "act": "silu"},
        # one decoded token through the gated layer of a ViT-H-wide block (weights packed once)
        {"name": "gated_one_token", "op": "gated", "type": "bf16", "T": 1, "C": 160, "H": 432, "N": 8, "act": "silu", "packed": True},
        # its training forward over a large batch: the weights are packed in every step
        {"name": "gated_tokens", "op": "gated", "type": "bf16", "T": 131072, "C": 160, "H": 432, "N": 8, "act": "silu", "packed": False},
        # a C_16 layer over one image batch, GELU gate
        {"name": "gated_c16", "op": "gated", "type": "bf16", "T": 8192, "C": 96, "H": 384, "N": 16, "act": "gelu", "packed": True},
        # a small C_6 layer in fp32, nothing a multiple of anything
        {"name": "gated_ragged", "op": "gated", "type": "fp32", "T": 1001, "C": 37, "H": 101, "N": 6, "act": "silu", "packed": False},
        # the training backward of the wide layer
        {"name": "gated_grad_tokens", "op": "gated_grad", "type": "bf16", "T": 65536, "C": 160, "H": 432, "N": 8, "act": "silu"},
        # and of a p4 layer in fp32
        {"name": "gated_grad_p4", "op": "gated_grad", "type": "fp32", "T": 2040, "C": 64, "H": 128, "N": 4, "act": "gelu"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "gated", "gated", "gated_grad"])
    kind = rng.choice(["bf16", "bf16", "fp32", "fp16"])
    if op.startswith("norm"):
        n = rng.choice([2, 3, 4, 6, 8, 8, 8, 12, 16])
        g = rng.choice([1, 1, 2, 8, 16, 32])
        s = 1 if rng.random() < 0.4 else _log(rng, 2, 10000)
        # at least a dozen values in a group: the gradient of a group of two is nothing but cancellation
        f = g * max(1, _log(rng, 8, 192) // g, -(-12 // (n * s)))
        room = (6 * 10**7) // (f * n * s)
        b = _log(rng, 1, max(1, min(room, 100000 if s == 1 else 256)))
        return {"op": op, "type": kind, "B": b, "S": s, "F": f, "N": n, "G": g, "act": rng.choice(["none", "silu", "gelu"])}
    if rng.random() < 0.5:  # the widths of the wide layers: multiples of 16
        n, kind, c, h = 8, "bf16", 16 * rng.randint(1, 10), 16 * rng.randint(1, 30)
        t = _log(rng, 1, 60000)
    else:
        n, c, h = rng.choice([3, 4, 4, 5, 6, 8, 12, 16]), rng.randint(5, 100), rng.randint(5, 200)
        t = _log(rng, 1, 6000)
    case = {"op": op, "type": kind, "T": t, "C": c, "H": h, "N": n, "act": rng.choice(["silu", "gelu"])}
    if op == "gated":
        case["packed"] = rng.random() < 0.5
    return case


def _inputs(case, seed):
    dev = torch.device("cuda")
    dt = _TYPES[case["type"]]
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=gen, device=dev, dtype=torch.float32) * scale + shift).to(dt)

    n = case["N"]
    if case["op"].startswith("norm"):
        b, s, f, g = case["B"], case["S"], case["F"], case["G"]
        # residual-stream values: another level and spread in every field
        level = torch.randn(f, 1, generator=gen, device=dev)
        spread = torch.rand(f, 1, generator=gen, device=dev) * 1.5 + 0.5
        x = (torch.randn((b, s, f, n), generator=gen, device=dev) * spread + level).to(dt)
        st = {"x": x, "gamma": normal(f, scale=0.3, shift=1.0), "beta": normal(f, scale=0.3), "G": g, "eps": 1e-5}
        if case["op"] == "norm_grad":
            # what the forward saved
            v = x.view(b, s, g, f // g * n)
            mean = torch.empty(b, g, dtype=torch.float32, device=dev)
            rstd = torch.empty_like(mean)
            step = max(1, (1 << 26) // (s * f * n))
            for i in range(0, b, step):
                var, mu = torch.var_mean(v[i:i + step].double(), dim=(1, 3), correction=0)
                mean[i:i + step] = mu
                rstd[i:i + step] = (var + 1e-5).rsqrt()
            st.update(mean=mean, rstd=rstd, dy=normal(b, s, f, n))
        return st
    t, c, h = case["T"], case["C"], case["H"]
    st = {"x": normal(t, c, n), "W": normal(h, 2, c, n, scale=1.0 / math.sqrt(c * n))}
    if case["op"] == "gated_grad":
        st["dh"] = normal(t, h, n)
    return st


def prepare(case, seed):
    state = dict(_inputs(case, seed), op=case["op"], act=case["act"])
    if own and case["op"].startswith("gated") and case.get("packed", True):
        import group_wise_dft_b200 as eq
        # the weights that a server packs once, or that the same training step's forward has packed
        state["Wspec"] = eq.cyclic_gated_weight_spectrum(state["W"])
    return state


# ---------------------------------------------------------------- plain forms


def _act(name, v):
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    return v


def _act_slope(name, v):
    if name == "silu":
        s = torch.sigmoid(v)
        return s * (1.0 + v * (1.0 - s))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    return torch.ones_like(v)


def _plain_norm(st):
    x = st["x"].float()
    b, s, f, n = x.shape
    v = x.view(b, s, st["G"], f // st["G"] * n)
    mean = v.mean(dim=(1, 3))
    d = v - mean[:, None, :, None]
    rstd = ((d * d).mean(dim=(1, 3)) + st["eps"]).rsqrt()
    xhat = (d * rstd[:, None, :, None]).view(b, s, f, n)
    z = xhat * st["gamma"].float()[:, None] + st["beta"].float()[:, None]
    return _act(st["act"], z).to(st["x"].dtype), mean, rstd


def _plain_norm_grad(st):
    x, dy = st["x"].float(), st["dy"].float()
    b, s, f, n = x.shape
    g = st["G"]
    gamma, beta = st["gamma"].float()[:, None], st["beta"].float()[:, None]

    def per_group(t):
        return t[:, None, :, None]

    xhat = ((x.view(b, s, g, -1) - per_group(st["mean"])) * per_group(st["rstd"])).view(b, s, f, n)
    dz = dy * _act_slope(st["act"], xhat * gamma + beta)
    # per item first, then over the items: sums over a few million values
    dgamma = (dz * xhat).sum(dim=(1, 3)).double().sum(0)
    dbeta = dz.sum(dim=(1, 3)).double().sum(0)
    dn = (dz * gamma).view(b, s, g, -1)
    xg = xhat.view(b, s, g, -1)
    dx = per_group(st["rstd"]) * (dn - per_group(dn.mean(dim=(1, 3))) - xg * per_group((dn * xg).mean(dim=(1, 3))))
    dt = st["x"].dtype
    return dx.view(b, s, f, n).to(dt), dgamma.to(dt), dbeta.to(dt)


def _dense(W):
    """The dense matrix of W[H, 2, C, N]: row (j, a, g), column (i, h), entry W[j, a, i, (g - h) mod N]."""
    h, two, c, n = W.shape
    k = torch.arange(n, device=W.device)
    at = (k[:, None] - k[None, :]) % n
    return W[..., at].permute(0, 1, 3, 2, 4).reshape(h * two * n, c * n)


def _plain_gated(st):
    x, W = st["x"].float(), st["W"].float()
    t, c, n = x.shape
    p = (x.view(t, c * n) @ _dense(W).t()).view(t, W.shape[0], 2, n)
    return _act(st["act"], p[:, :, 0]).mul(p[:, :, 1]).to(st["x"].dtype)


def _plain_gated_grad(st):
    x, W, dh = st["x"].float(), st["W"].float(), st["dh"].float()
    t, c, n = x.shape
    h = W.shape[0]
    D = _dense(W)
    p = (x.view(t, c * n) @ D.t()).view(t, h, 2, n)
    gate, value = p[:, :, 0], p[:, :, 1]
    dp = torch.stack((dh * value * _act_slope(st["act"], gate), dh * _act(st["act"], gate)), dim=2).view(t, 2 * h * n)
    dx = (dp @ D).view(t, c, n)
    dD = (dp.t() @ x.view(t, c * n)).view(h, 2, n, c, n)
    # dW[j, a, i, m] = sum over g of dD[(j, a, g), (i, (g - m) mod N)]
    k = torch.arange(n, device=W.device)
    at = (k[:, None] - k[None, :]) % n
    dW = dD.permute(0, 1, 3, 2, 4).gather(4, at.expand(h, 2, c, n, n)).sum(3)
    return dx.to(st["x"].dtype), dW.to(st["x"].dtype)


# ---------------------------------------------------------------- one pass


def _own(st):
    import group_wise_dft_b200 as eq
    act = {"none": eq.ACT_NONE, "silu": eq.ACT_SILU, "gelu": eq.ACT_GELU}[st["act"]]
    if st["op"] == "norm":
        return eq.group_norm(st["x"], st["G"], st["gamma"], st["beta"], eps=st["eps"], act=act)
    if st["op"] == "norm_grad":
        return eq.group_norm_backward(st["x"], st["dy"], st["mean"], st["rstd"], st["G"], st["gamma"], st["beta"],
                                      act=act)
    W = st["W"]
    spec = st["Wspec"] if "Wspec" in st else eq.cyclic_gated_weight_spectrum(W)
    if st["op"] == "gated":
        return eq.cyclic_gated_forward(st["x"], spec, W.shape[0], act=act)
    return eq.cyclic_gated_backward(st["x"], st["dh"], spec, eq.cyclic_gated_weight_spectrum_adjoint(W), act=act)


def run(state):
    if own:
        return _own(state)
    if state["op"] == "norm":
        return _plain_norm(state)
    if state["op"] == "norm_grad":
        return _plain_norm_grad(state)
    if state["op"] == "gated":
        return _plain_gated(state)
    return _plain_gated_grad(state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    size = 4 if case["type"] == "fp32" else 2
    n = case["N"]
    if case["op"].startswith("norm"):
        values = case["B"] * case["S"] * case["F"] * n
        small = 2 * case["F"] * size + 2 * case["B"] * case["G"] * 4
        if case["op"] == "norm":
            return {"bytes": 2 * values * size + small, "flops": 8 * values}
        return {"bytes": 3 * values * size + small + 2 * case["F"] * size, "flops": 16 * values}
    t, c, h = case["T"], case["C"], case["H"]
    weights = 2 * h * c * n * size
    # per token and channel pair, the half spectrum's real products: one per real bin, four per complex bin
    products = (2 if n % 2 == 0 else 1) + 4 * ((n - 1) // 2)
    flops = 2 * t * c * 2 * h * products
    if case["op"] == "gated":
        return {"bytes": t * (c + h) * n * size + weights, "flops": flops}
    # the gate and value again, dx and dW
    return {"bytes": t * (2 * c + h) * n * size + 2 * weights, "flops": 3 * flops}


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_norm(st, act):
    x = st["x"].double()
    b, s, f, n = x.shape
    y = torch.empty_like(x)
    means, rstds = [], []
    for group in x.split(f // st["G"], dim=2):
        means.append(group.mean(dim=(1, 2, 3)))
        rstds.append(1.0 / torch.sqrt(group.var(dim=(1, 2, 3), unbiased=False) + st["eps"]))
    mean, rstd = torch.stack(means, 1), torch.stack(rstds, 1)
    fields = f // st["G"]
    for k in range(f):
        z = (x[:, :, k] - mean[:, k // fields, None, None]) * rstd[:, k // fields, None, None]
        y[:, :, k] = act(z * st["gamma"][k].double() + st["beta"][k].double())
    return y, mean, rstd


def _exact_norm_grad(st, act):
    x, dy = st["x"].double(), st["dy"].double()
    b, s, f, n = x.shape
    fields = f // st["G"]
    dx = torch.empty_like(x)
    dgamma, dbeta = [], []
    for k in range(st["G"]):
        at = slice(k * fields, (k + 1) * fields)
        mean, rstd = st["mean"][:, k].double(), st["rstd"][:, k].double()
        xh = (x[:, :, at] - mean[:, None, None, None]) * rstd[:, None, None, None]
        gamma = st["gamma"][at].double()[None, None, :, None]
        z = (xh * gamma + st["beta"][at].double()[None, None, :, None]).requires_grad_()
        with torch.enable_grad():
            (dz,) = torch.autograd.grad(act(z), z, dy[:, :, at])
        dgamma.append(torch.einsum("bsfn,bsfn->f", dz, xh))
        dbeta.append(dz.sum(dim=(0, 1, 3)))
        v = dz * gamma
        count = s * fields * n
        a = v.sum(dim=(1, 2, 3), keepdim=True) / count
        c = (v * xh).sum(dim=(1, 2, 3), keepdim=True) / count
        dx[:, :, at] = (v - a - xh * c) * rstd[:, None, None, None]
    return dx, torch.cat(dgamma), torch.cat(dbeta)


def _exact_products(x, W):
    """p[t, j, a, g], slot by slot: W[j, a, i, m] meets x[t, i, (g - m) mod N]."""
    t, c, n = x.shape
    rows = W.reshape(-1, c, n)
    p = torch.zeros(t, rows.shape[0], n, dtype=torch.float64, device=x.device)
    for g in range(n):
        turned = torch.stack([x[:, :, (g - m) % n] for m in range(n)], dim=2)
        p[:, :, g] = turned.reshape(t, c * n) @ rows.reshape(-1, c * n).t()
    return p.reshape(t, W.shape[0], 2, n)


def _exact_gated(st, act):
    p = _exact_products(st["x"].double(), st["W"].double())
    return act(p[:, :, 0]) * p[:, :, 1]


def _exact_gated_grad(st, act):
    x, W, dh = st["x"].double(), st["W"].double(), st["dh"].double()
    t, c, n = x.shape
    dx = torch.zeros_like(x)
    dW = torch.zeros_like(W)
    rows = W.reshape(-1, c, n)
    for lo in range(0, t, 16384):
        xs = x[lo:lo + 16384]
        p = _exact_products(xs, W).requires_grad_()
        with torch.enable_grad():
            (dp,) = torch.autograd.grad(act(p[:, :, 0]) * p[:, :, 1], p, dh[lo:lo + 16384])
        dp = dp.reshape(xs.shape[0], -1, n)
        for g in range(n):
            # slot g of the output meets input slot (g - m) mod N through W[..., m]
            back = (dp[:, :, g] @ rows.reshape(rows.shape[0], c * n)).reshape(-1, c, n)
            turned = torch.stack([xs[:, :, (g - m) % n] for m in range(n)], dim=2)
            dW += (dp[:, :, g].t() @ turned.reshape(-1, c * n)).reshape(W.shape)
            for m in range(n):
                dx[lo:lo + 16384, :, (g - m) % n] += back[:, :, m]
    return dx, dW


def exact(case, seed):
    act = {"none": lambda v: v, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[case["act"]]
    st = _inputs(case, seed)
    with torch.no_grad():
        if case["op"] == "norm":
            return _exact_norm(st, act)
        if case["op"] == "norm_grad":
            return _exact_norm_grad(st, act)
        if case["op"] == "gated":
            return _exact_gated(st, act)
        return _exact_gated_grad(st, act)
