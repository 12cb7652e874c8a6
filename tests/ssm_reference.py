"""The selective state space scan from its definition, a token at a time in
float64 (torch on the CPU), and its gradients by differentiating that; inputs
for the tests; and the bound that results are held to.

Bound per element: half a step of the result's type, eps/2 |r| (bf16 only, the
one rounding there is), plus float32 arithmetic.  Of the latter each token adds
at most about 2^-21 of its term (the exponential 2^-22, its argument's and the
products' roundings 2^-24 each); the terms have random signs, so T of them and
the sums over N states (or C channels) leave at most four times sqrt(T + N + C)
2^-21 of the tensor's largest value; a gradient passes through two such chains
and a product of both: four times that."""
import math

import torch

SHARED = ("A", "dt_bias", "feedthrough", "conv_weight", "conv_bias")


def inputs(B, H, T, D, N, G=1, W=4, dtype=torch.float32, seed=0, z=True, bias=True, feed=True, carried=True,
           gates="preact"):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    i = dict(x=normal(B, H, T, D).to(dtype), dt=(0.5 * normal(B, H, T, D)), Bm=normal(B, G, T, N).to(dtype),
             Cm=(normal(B, G, T, N) / math.sqrt(N)).to(dtype), A=-torch.arange(1, N + 1) * torch.exp(0.1 * normal(H, D, N)))
    step = 10 ** (-3 + 2 * torch.rand(H, D, generator=g))
    i["dt_bias"] = step + torch.log(-torch.expm1(-step)) if bias and gates == "preact" else None
    i["dt"] = i["dt"].to(dtype) if gates == "preact" else (0.1 * torch.sigmoid(i["dt"])).to(dtype)
    i["z"] = normal(B, H, T, D).to(dtype) if z else None
    i["feedthrough"] = 1 + 0.1 * normal(H, D) if feed else None
    i["conv_weight"] = normal(H, D, W) / math.sqrt(W) if W else None
    i["conv_bias"] = 0.1 * normal(H, D) if W and bias else None
    i["conv_state_in"] = normal(B, H, W - 1, D).to(dtype) if W > 1 and carried else None
    i["S0"] = 0.3 * normal(B, H, D, N) if carried else None
    return i


def scan(i, lengths=None, silu=True, gates="preact"):
    """(y with zeros behind the ends, ST, conv_state_out) in float64."""
    B, H, T, D = i["x"].shape
    G, N = i["Bm"].shape[1], i["A"].shape[-1]
    f64 = {n: (t.double() if t is not None else None) for n, t in i.items()}
    W = i["conv_weight"].shape[-1] if i["conv_weight"] is not None else 0
    lengths = [T] * B if lengths is None else [int(n) for n in lengths]
    ys, sts, css = [], [], []
    for b in range(B):
        s = f64["S0"][b] if f64["S0"] is not None else torch.zeros(H, D, N, dtype=torch.float64)
        past = list(f64["conv_state_in"][b].unbind(1)) if f64["conv_state_in"] is not None else \
            [torch.zeros(H, D, dtype=torch.float64)] * max(0, W - 1)
        rows = []
        for t in range(T):
            if t >= lengths[b]:
                rows.append(torch.zeros(H, D, dtype=torch.float64))
                continue
            u = f64["x"][b, :, t]
            if W:
                past = past + [u]
                u = sum(f64["conv_weight"][..., k] * past[-1 - k] for k in range(W))
                if f64["conv_bias"] is not None:
                    u = u + f64["conv_bias"]
                u = u * torch.sigmoid(u) if silu else u
                past = past[1:] if W > 1 else []
            d = f64["dt"][b, :, t]
            if f64["dt_bias"] is not None:
                d = d + f64["dt_bias"]
            if gates == "preact":
                d = torch.nn.functional.softplus(d, threshold=1000)
            bb, cc = (f64[m][b, :, t].repeat_interleave(H // G, 0)[:, None] for m in ("Bm", "Cm"))
            s = torch.exp(d[..., None] * f64["A"]) * s + (d * u)[..., None] * bb
            y = (s * cc).sum(-1)
            if f64["feedthrough"] is not None:
                y = y + f64["feedthrough"] * u
            if f64["z"] is not None:
                y = y * f64["z"][b, :, t] * torch.sigmoid(f64["z"][b, :, t])
            rows.append(y)
        ys.append(torch.stack(rows, 1) if rows else torch.zeros(H, 0, D, dtype=torch.float64))
        sts.append(s)
        css.append(torch.stack(past, 1) if W > 1 else None)
    return torch.stack(ys), torch.stack(sts), torch.stack(css) if W > 1 else None


NAMES = {"x": "dx", "dt": "ddt", "z": "dz", "Bm": "dB", "Cm": "dC", "A": "dA", "dt_bias": "ddt_bias", "feedthrough": "dfeed",
         "conv_weight": "dconv_weight", "conv_bias": "dconv_bias", "conv_state_in": "dconv_state_in", "S0": "dS0"}


def gradients(i, gy, gST=None, gcs=None, lengths=None, silu=True, gates="preact"):
    leaves = {n: (t.double().requires_grad_(True) if t is not None else None) for n, t in i.items()}
    y, ST, cs = scan(leaves, lengths, silu, gates)
    loss = (y * gy.double()).sum()
    if gST is not None:
        loss = loss + (ST * gST.double()).sum()
    if gcs is not None:
        loss = loss + (cs * gcs.double()).sum()
    loss.backward()
    return {NAMES[n]: (t.grad if t.grad is not None else torch.zeros_like(t)) for n, t in leaves.items() if t is not None}


def assert_near(got, want, terms, what, grad=False):
    got = got.detach().cpu()
    half = torch.finfo(got.dtype).eps / 2 if got.dtype == torch.bfloat16 else 0.0
    got, want = got.double(), want.detach().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if not want.numel():
        return
    bound = half * want.abs() + (4 if grad else 1) * 4 * math.sqrt(terms) * 2.0 ** -21 * want.abs().max()
    off = (got - want).abs()
    worst = (off / bound.clamp(min=1e-30)).max().item() if torch.isfinite(got).all() else math.inf
    assert worst <= 1, f"{what}: {worst:.2f} of the bound (largest value {want.abs().max():.3g}, largest error {off.max():.3g})"
