"""Cases, plain forms and 64-bit forms of the operators of hybrid layers:

  scan   selective state space scan over prompts, with its short causal convolution
  train  the same, forward and backward (a training step's share)
  step   one token of the scan, the state and the convolution's inputs updated in place
  fill   a prompt's keys and values into an 8-bit ring cache with a scale for each block and head
  decode one token of sliding-window shared-key attention over that cache

The scan, per channel (h, c), state n and token t (g is the head's group):

  u = silu(bias + sum_i w_i x_{t-i})            delta = softplus(dt + dt_bias)
  s_t = exp(delta A) s_{t-1} + delta u B_t      y = (sum_n C_t s_t + d u) silu(z)
"""
import math

import torch

own = False

NAMES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def listed():
    return [
        # the tail of a chunked prompt: a short odd piece carried on from a state, float32
        scan("scan_piece", "f32", B=2, H=6, G=1, T=37, D=32, N=16, ragged=False, carried=True),
        # prompts of unlike lengths in one padded batch through a 130M-scale layer (twice the 768 channels)
        scan("scan_layer_ragged", "bf16", B=8, H=24, G=1, T=2048, D=64, N=16, ragged=True, carried=False),
        # one long odd-sized context: few channels for the card, so the tokens have to be split
        scan("scan_long_context", "bf16", B=1, H=24, G=1, T=16387, D=64, N=16, ragged=False, carried=True),
        # a training step of a small model in float32, odd length, two groups
        train("train_small", "f32", B=2, H=4, G=2, T=509, D=32, N=16, ragged=False, carried=True),
        # a training step's share of the 130M-scale layer
        train("train_layer", "bf16", B=4, H=24, G=1, T=2048, D=64, N=16, ragged=False, carried=False),
        # one user's next token
        dict(name="step_one", op="step", dtype="bf16", B=1, H=24, G=1, D=64, N=16, W=4),
        # a serving batch with a larger state
        dict(name="step_batch", op="step", dtype="bf16", B=256, H=16, G=1, D=128, N=64, W=4),
        # prompts shorter and longer than the window into the cache of a 130M-scale layer
        dict(name="fill_layer", op="fill", cache="e4m3", B=8, H=12, T=2048, dk=64, dv=64, window=512, block=64, ragged=True),
        # long prompts into large rings whose last block is short
        dict(name="fill_long", op="fill", cache="int8", B=4, H=16, T=16384, dk=128, dv=128, window=8200, block=16, ragged=False),
        # few sequences, short rings not yet full: the least a decode step can cost
        dict(name="decode_small", op="decode", cache="int8", B=2, H=12, dk=64, dv=64, window=300, block=32, start=40, stride=17),
        # one user deep in a long window
        dict(name="decode_long_window", op="decode", cache="e4m3", B=1, H=16, dk=128, dv=128, window=32768, block=64, start=40001, stride=0),
        # batched decode at the 1.6B scale, sequences at different places of wrapped rings
        dict(name="decode_batch", op="decode", cache="e4m3", B=256, H=16, dk=128, dv=128, window=512, block=64, start=600, stride=37),
    ]


def scan(name, dtype, **sizes):
    return dict(name=name, op="scan", dtype=dtype, W=4, **sizes)


def train(name, dtype, **sizes):
    return dict(name=name, op="train", dtype=dtype, W=4, **sizes)


def draw(rng):
    op = rng.choice(["scan", "train", "step", "fill", "decode"])

    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    if op in ("scan", "train"):
        D, N, H = rng.choice([16, 32, 64, 128]), rng.choice([16, 16, 32, 64, 128]), log(1, 24)
        G = rng.choice([g for g in (1, 2, 3, 4, 6, 8) if H % g == 0])
        B = log(1, 8)
        # no more state updates than the largest listed case of the operator has
        most = (4 if op == "train" else 8) * 2048 * 24 * 64 * 16 // 2
        T = min(log(1, 8192 if op == "scan" else 2048), max(1, most // (B * H * D * N)))
        return dict(op=op, dtype=rng.choice(["f32", "bf16"]), B=B, H=H, G=G, T=T, D=D, N=N, W=rng.choice([0, 2, 3, 4, 4]),
                    ragged=rng.random() < 0.4, carried=rng.random() < 0.5)
    if op == "step":
        D, N, H = rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128]), log(1, 32)
        G = rng.choice([g for g in (1, 2, 4) if H % g == 0])
        B = min(log(1, 256), max(1, 256 * 16 * 128 * 64 // (H * D * N)))
        return dict(op=op, dtype=rng.choice(["f32", "bf16"]), B=B, H=H, G=G, D=D, N=N, W=rng.choice([0, 2, 3, 4, 4]))
    dk, dv, H, block = rng.choice([64, 128]), rng.choice([64, 128]), log(1, 24), rng.choice([16, 32, 64])
    window = log(1, 32768 if op == "decode" else 8192)
    B = min(log(1, 256 if op == "decode" else 8), max(1, 120_000_000 // (window * (dk + H * dv))))
    sizes = dict(op=op, cache=rng.choice(["e4m3", "int8"]), B=B, H=H, dk=dk, dv=dv, window=window, block=block)
    if op == "fill":
        T = min(log(1, 12000), max(1, 100_000_000 // (B * H * dv)))
        return dict(sizes, T=T, ragged=rng.random() < 0.5)
    return dict(sizes, start=rng.randrange(0, 3 * window), stride=rng.choice([0, 1, 7, 37]))


# ------------------------------------------------------------------ inputs


def lengths_of(c):
    """Tokens of each sequence: all T, or from T down to about a third of it."""
    if not c["ragged"]:
        return [c["T"]] * c["B"]
    return [c["T"] - (2 * b * c["T"]) // (3 * c["B"]) for b in range(c["B"])]


def positions_of(c):
    return [c["start"] + b * c["stride"] for b in range(c["B"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return (prepare_scan if case["op"] in ("scan", "train", "step") else prepare_cache)(dict(case), g)


def prepare_scan(c, g):
    B, H, G, D, N, W, dtype = c["B"], c["H"], c["G"], c["D"], c["N"], c["W"], NAMES[c["dtype"]]
    tokens = (c["T"],) if c["op"] != "step" else ()

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    s = {"case": c}
    s["x"] = normal(B, H, *tokens, D).to(dtype)
    s["dt"] = (0.5 * normal(B, H, *tokens, D)).to(dtype)
    s["Bm"] = normal(B, G, *tokens, N).to(dtype)
    s["Cm"] = (normal(B, G, *tokens, N) / math.sqrt(N)).to(dtype)
    s["z"] = normal(B, H, *tokens, D).to(dtype)
    # decay rates near 1..N and steps between 1e-3 and 1e-1, as such layers are initialised
    s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.1 * normal(H, D, N))
    step = torch.exp(torch.rand(H, D, device="cuda", generator=g) * math.log(100.0)) * 1e-3
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["feedthrough"] = 1 + 0.1 * normal(H, D)
    s["conv_weight"] = normal(H, D, W) / math.sqrt(W) if W else None
    s["conv_bias"] = 0.1 * normal(H, D) if W else None
    if c["op"] == "step":
        s["S"] = 0.1 * normal(B, H, D, N)
        s["conv_state"] = normal(B, H, W - 1, D).to(dtype) if W else None
        return s
    s["S0"] = 0.1 * normal(B, H, D, N) if c["carried"] else None
    s["conv_state_in"] = normal(B, H, W - 1, D).to(dtype) if W and c["carried"] else None
    s["lengths"] = torch.tensor(lengths_of(c), dtype=torch.int32, device="cuda") if c["ragged"] else None
    s["y"] = torch.zeros_like(s["x"])
    if c["op"] == "train":
        s["grad_y"] = normal(B, H, *tokens, D).to(dtype)
        s["grad_ST"] = normal(B, H, D, N) if c["carried"] else None
    return s


def prepare_cache(c, g):
    B, H, dk, dv, w, R = c["B"], c["H"], c["dk"], c["dv"], c["window"], c["block"]
    nb = -(-w // R)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g).to(torch.bfloat16)

    s = {"case": c}
    if c["op"] == "fill":
        s["k"], s["v"] = normal(B, c["T"], dk), normal(B, H, c["T"], dv)
        s["lengths"] = torch.tensor(lengths_of(c), dtype=torch.int32, device="cuda") if c["ragged"] else None
        kind = NAMES[c["cache"]]
        s["k_cache"] = torch.zeros(B, w, dk, device="cuda").to(kind)
        s["v_cache"] = torch.zeros(B * H, w, dv, dtype=torch.bfloat16, device="cuda").to(kind).view(B, H, w, dv)
        s["k_scale"], s["v_scale"] = torch.ones(B, nb, device="cuda"), torch.ones(B, H, nb, device="cuda")
        s["k_tail"] = torch.zeros(B, R, dk, dtype=torch.bfloat16, device="cuda")
        s["v_tail"] = torch.zeros(B, H, R, dv, dtype=torch.bfloat16, device="cuda")
        s["pos"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return s
    s["q"], s["k"], s["v"] = normal(B, H, dk), normal(B, dk), normal(B, H, dv)
    s["k_cache"], s["k_scale"] = quantise(padded(normal(B, w, dk), nb * R), R, c["cache"])
    parts = [quantise(padded(normal(H, w, dv), nb * R), R, c["cache"]) for _ in range(B)]
    s["k_cache"] = s["k_cache"][:, :w].contiguous()
    s["v_cache"] = torch.stack([p[0][:, :w] for p in parts])
    s["v_scale"] = torch.stack([p[1] for p in parts])
    s["k_tail"], s["v_tail"] = normal(B, R, dk), normal(B, H, R, dv)
    s["pos"] = torch.tensor(positions_of(c), dtype=torch.int32, device="cuda")
    return s


def padded(x, rows):
    return torch.cat([x, x.new_zeros(*x.shape[:-2], rows - x.shape[-2], x.shape[-1])], -2)


# ------------------------------------------------------------------ one pass


def run(s):
    op = s["case"]["op"]
    if own:
        import gated_linear_attention_ddts_b200 as rdm
        return globals()["own_" + op](rdm, s)
    return globals()["plain_" + op](s)


def own_scan(rdm, s):
    y, ST, conv = rdm.rdm_ssm_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], S0=s["S0"], z=s["z"], dt_bias=s["dt_bias"], feedthrough=s["feedthrough"],
                                  conv_weight=s["conv_weight"], conv_bias=s["conv_bias"], conv_state_in=s["conv_state_in"], lengths=s["lengths"],
                                  y=s["y"], return_state=True)
    return {"y": y, "ST": ST, "conv_state": conv} if s["case"]["W"] else {"y": y, "ST": ST}


def own_train(rdm, s):
    given = dict(S0=s["S0"], z=s["z"], dt_bias=s["dt_bias"], feedthrough=s["feedthrough"], conv_weight=s["conv_weight"], conv_bias=s["conv_bias"],
                 conv_state_in=s["conv_state_in"], lengths=s["lengths"])
    x, dt, A, Bm, Cm = s["x"], s["dt"], s["A"], s["Bm"], s["Cm"]
    saved = rdm.rdm_ssm_saved_states(x, A)
    y, _, _ = rdm.rdm_ssm_fwd(x, dt, A, Bm, Cm, y=s["y"], saved_states=saved, **given)
    grads = rdm.rdm_ssm_bwd(x, dt, A, Bm, Cm, s["grad_y"], s["grad_ST"], saved_states=saved, **given)
    return {"y": y, **{n: v for n, v in grads.items() if v is not None}}


def own_step(rdm, s):
    y = rdm.rdm_ssm_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["S"], z=s["z"], dt_bias=s["dt_bias"], feedthrough=s["feedthrough"],
                         conv_weight=s["conv_weight"], conv_bias=s["conv_bias"], conv_state=s["conv_state"])
    return {"y": y, "S": s["S"], "conv_state": s["conv_state"]} if s["case"]["W"] else {"y": y, "S": s["S"]}


CACHE = ("k_cache", "v_cache", "k_scale", "v_scale", "k_tail", "v_tail", "pos")


def own_fill(rdm, s):
    rdm.rdm_ska_q8_fill(s["k"], s["v"], *(s[n] for n in CACHE), lengths=s["lengths"])
    return {n: s[n] for n in CACHE}


def own_decode(rdm, s):
    o = rdm.rdm_ska_q8_decode(s["q"], s["k"], s["v"], *(s[n] for n in CACHE))
    return {"o": o, **{n: s[n] for n in CACHE}}


# ------------------------------------------------------------------ plain forms: the scan


def silu(x):
    return x / (1 + torch.exp(-x))


def softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def convolve(x, s, state):
    """The convolution's sum before its activation, and x with the W-1 inputs before it (x in float32, time the third axis)."""
    w = s["conv_weight"]
    W, T = w.shape[-1], x.shape[2]
    before = state.to(x.dtype) if state is not None else x.new_zeros(x.shape[0], x.shape[1], W - 1, x.shape[3])
    xs = torch.cat([before, x], 2)
    zc = s["conv_bias"].to(x.dtype)[:, None] + sum(w[:, None, :, i].to(x.dtype) * xs[:, :, W - 1 - i:W - 1 - i + T] for i in range(W))
    return zc, xs


def spread(m, H):
    """[B,G,T,N] of the groups as [T,B,H,1,N] of the heads, float32."""
    return m.float().repeat_interleave(H // m.shape[1], 1).permute(2, 0, 1, 3)[:, :, :, None]


def valid(s):
    """[B,T] truth values of the tokens that count, None for all."""
    if s["lengths"] is None:
        return None
    return torch.arange(s["x"].shape[2], device="cuda") < s["lengths"][:, None]


def plain_inputs(s):
    """u and delta as [T,B,H,D] float32 (delta 0 behind a sequence's end: the state stays), and the convolution's sum and inputs."""
    x = s["x"].float()
    zc, xs = convolve(x, s, s["conv_state_in"]) if s["case"]["W"] else (x, x)
    u = silu(zc) if s["case"]["W"] else x
    delta = softplus(s["dt"].float() + s["dt_bias"][:, None])
    if s["lengths"] is not None:
        delta = delta * valid(s)[:, None, :, None]
    return u.permute(2, 0, 1, 3), delta.permute(2, 0, 1, 3), zc, xs


def plain_states(s, u, delta, keep):
    """The recurrence a token at a time, 128 tokens' factors at once: sum_n C s as [T,B,H,D], the last state, and every state if `keep`."""
    c = s["case"]
    B, H, T, D, N = c["B"], c["H"], c["T"], c["D"], c["N"]
    Bm, Cm = spread(s["Bm"], H), spread(s["Cm"], H)
    state = s["S0"].clone() if s["S0"] is not None else u.new_zeros(B, H, D, N)
    y, kept = torch.empty_like(u), torch.empty(T if keep else 0, B, H, D, N, device="cuda")
    for t0 in range(0, T, 128):
        t1 = min(t0 + 128, T)
        a = torch.exp(delta[t0:t1, ..., None] * s["A"])
        b = torch.mul((delta[t0:t1] * u[t0:t1])[..., None], Bm[t0:t1], out=kept[t0:t1] if keep else None)
        for t in range(t1 - t0):
            state = torch.addcmul(b[t], a[t], state, out=b[t])
        y[t0:t1] = (b * Cm[t0:t1]).sum(-1)
    return y, state.clone(), kept


def last_inputs(s, xs):
    """The W-1 inputs before each sequence's end: the convolution's state behind it."""
    c = s["case"]
    end = s["lengths"].long() if s["lengths"] is not None else torch.full((c["B"],), c["T"], device="cuda")
    at = end[:, None] + torch.arange(c["W"] - 1, device="cuda")
    return torch.gather(xs, 2, at[:, None, :, None].expand(-1, c["H"], -1, c["D"]))


def plain_scan(s):
    u, delta, _, xs = plain_inputs(s)
    y, ST, _ = plain_states(s, u, delta, False)
    write_y(s, y, u)
    return {"y": s["y"], "ST": ST, "conv_state": last_inputs(s, xs).to(s["x"].dtype)} if s["case"]["W"] else {"y": s["y"], "ST": ST}


def write_y(s, y, u):
    y = (y + s["feedthrough"] * u).permute(1, 2, 0, 3) * silu(s["z"].float())
    keep = valid(s)
    s["y"].copy_(y if keep is None else torch.where(keep[:, None, :, None], y, s["y"].float()))


def plain_train(s):
    c = s["case"]
    B, H, G, T, D, N, W = c["B"], c["H"], c["G"], c["T"], c["D"], c["N"], c["W"]
    u, delta, zc, xs = plain_inputs(s)
    y, _, states = plain_states(s, u, delta, True)
    write_y(s, y, u)
    y = y + s["feedthrough"] * u
    z, gy = s["z"].float().permute(2, 0, 1, 3), s["grad_y"].float().permute(2, 0, 1, 3)
    if s["lengths"] is not None:
        gy = gy * valid(s).t()[:, :, None, None]
    sg = 1 / (1 + torch.exp(-z))
    p = gy * z * sg
    dz = gy * y * sg * (1 + z * (1 - sg))
    Bm, Cm = spread(s["Bm"], H), spread(s["Cm"], H)
    grad = s["grad_ST"].clone() if s["grad_ST"] is not None else u.new_zeros(B, H, D, N)
    du, ddelta = torch.empty_like(u), torch.empty_like(u)
    dB, dC = u.new_empty(T, B, G, N), u.new_empty(T, B, G, N)
    dA = u.new_zeros(H, D, N)
    for t1 in range(T, 0, -128):
        t0 = max(0, t1 - 128)
        st, d, x = states[t0:t1], delta[t0:t1, ..., None], u[t0:t1]
        a = torch.exp(d * s["A"])
        b = p[t0:t1, ..., None] * Cm[t0:t1]
        for t in range(t1 - t0 - 1, -1, -1):  # grad: dL/ds_t with all that follows; then through the decay into token t-1
            grad = b[t].add_(grad)
            grad = a[t] * grad
        w = b * (st - d * x[..., None] * Bm[t0:t1])
        q = (b * Bm[t0:t1]).sum(-1)
        ddelta[t0:t1] = x * q + (w * s["A"]).sum(-1)
        dA += (w * d).sum((0, 1))
        du[t0:t1] = delta[t0:t1] * q + s["feedthrough"] * p[t0:t1]
        dB[t0:t1] = (b * (d * x[..., None])).unflatten(2, (G, H // G)).sum((3, 4))
        dC[t0:t1] = (st * p[t0:t1, ..., None]).unflatten(2, (G, H // G)).sum((3, 4))
    dtype = s["x"].dtype
    ddt = ddelta * torch.sigmoid(s["dt"].float() + s["dt_bias"][:, None]).permute(2, 0, 1, 3)
    if s["lengths"] is not None:
        ddt = ddt * valid(s).t()[:, :, None, None]
    out = {"y": s["y"], "ddt": seq(ddt, dtype), "dz": seq(dz, dtype), "dB": seq(dB, dtype), "dC": seq(dC, dtype), "dA": dA,
           "ddt_bias": ddt.sum((0, 1)), "dfeed": (p * u).sum((0, 1))}
    if c["carried"]:
        out["dS0"] = grad
    du = du.permute(1, 2, 0, 3)
    if s["lengths"] is not None:
        du = du * valid(s)[:, None, :, None]
    if not W:
        return {**out, "dx": du.to(dtype)}
    sg = 1 / (1 + torch.exp(-zc))
    dzc = du * sg * (1 + zc * (1 - sg))
    dxs = torch.zeros_like(xs)
    dw = torch.empty_like(s["conv_weight"])
    for i in range(W):
        dxs[:, :, W - 1 - i:W - 1 - i + T] += s["conv_weight"][:, None, :, i] * dzc
        dw[..., i] = (dzc * xs[:, :, W - 1 - i:W - 1 - i + T]).sum((0, 2))
    out.update(dx=dxs[:, :, W - 1:].to(dtype), dconv_weight=dw, dconv_bias=dzc.sum((0, 2)))
    if c["carried"]:
        out["dconv_state_in"] = dxs[:, :, :W - 1].to(dtype)
    return out


def seq(m, dtype):
    """[T,B,H,D] as [B,H,T,D] in the inputs' type."""
    return m.permute(1, 2, 0, 3).to(dtype).contiguous()


def plain_step(s):
    c = s["case"]
    x = s["x"].float()
    if c["W"]:
        zc, xs = convolve(x[:, :, None], s, s["conv_state"])
        u = silu(zc[:, :, 0])
        s["conv_state"].copy_(xs[:, :, 1:])
    else:
        u = x
    delta = softplus(s["dt"].float() + s["dt_bias"])
    Bm, Cm = (s[n].float().repeat_interleave(c["H"] // c["G"], 1)[:, :, None] for n in ("Bm", "Cm"))
    s["S"].copy_(torch.exp(delta[..., None] * s["A"]) * s["S"] + (delta * u)[..., None] * Bm)
    y = ((s["S"] * Cm).sum(-1) + s["feedthrough"] * u) * silu(s["z"].float())
    out = {"y": y.to(s["x"].dtype), "S": s["S"]}
    return {**out, "conv_state": s["conv_state"]} if c["W"] else out


# ------------------------------------------------------------------ plain forms: the 8-bit cache


def quantise(x, R, cache):
    """Rows [.., n R, d] in blocks of R: the codes (float8 or int8 values) and the scales [.., n].

    e4m3: the least power of two that keeps the block's largest magnitude within 448, so that scaling is exact.
    int8: the largest magnitude over 127. A block of zeros has the scale 1."""
    b = x.float().unflatten(-2, (-1, R))
    most = b.abs().amax((-2, -1))
    if cache == "e4m3":
        m, e = torch.frexp(most)
        e = torch.clamp(e - torch.where(m > 0.875, 8, 9), min=-126)
        scale = torch.ldexp(torch.ones_like(most), torch.where(most > 0, e, torch.zeros_like(e)))
        codes = (b / scale[..., None, None]).to(torch.float8_e4m3fn)
    else:
        scale = torch.where(most > 0, most / torch.full_like(most, 127.0), torch.ones_like(most))
        codes = torch.clamp(torch.round(b / scale[..., None, None]), -127, 127).to(torch.int8)
    return codes.flatten(-3, -2), scale


def plain_fill(s):
    c = s["case"]
    w, R, T = c["window"], c["block"], c["T"]
    end = s["lengths"].long() if s["lengths"] is not None else torch.full((c["B"],), T, device="cuda")
    fill_rows(s["k"][:, None], s["k_cache"][:, None], s["k_scale"][:, None], s["k_tail"][:, None], end, w, R, c["cache"])
    fill_rows(s["v"], s["v_cache"], s["v_scale"], s["v_tail"], end, w, R, c["cache"])
    s["pos"].copy_(end)
    return {n: s[n] for n in CACHE}


def fill_rows(x, cache, scale, tail, end, w, R, kind):
    """Each slot's last token, if it has one, block by block; the unfinished block's tokens go to the tail and its slots keep the round before."""
    B, H, T, d = x.shape
    nb = scale.shape[-1]
    slot = torch.arange(nb * R, device="cuda")
    inside = slot < w
    last = end[:, None] - 1
    cur = last % w
    begun = (cur // R * R <= slot) & (slot <= cur) & ~((cur % R == R - 1) | (cur == w - 1))  # in the unfinished block, written this round
    rounds = torch.where(slot <= cur, last // w, last // w - 1) - begun.long()
    # a block is held whole: what the unfinished block's slots hold is the round before it
    token = rounds * w + slot
    has = inside & (rounds >= 0) & (end[:, None] > 0)
    rows = torch.gather(x, 2, token.clamp(0, T - 1)[:, None, :, None].expand(-1, H, -1, d))
    codes, scales = quantise(torch.where(has[:, None, :, None], rows, torch.zeros_like(rows)), R, kind)
    blocks = has.unflatten(1, (nb, R)).any(2)
    scale.copy_(torch.where(blocks[:, None], scales, scale))
    view = codes[:, :, :w].view(torch.uint8)
    cache.view(torch.uint8).copy_(torch.where(has[:, None, :w, None], view, cache.view(torch.uint8)))
    at = cur // R * R + torch.arange(R, device="cuda")
    mine = (torch.arange(R, device="cuda") <= cur % R) & ~((cur % R == R - 1) | (cur == w - 1)) & (end[:, None] > 0)
    rows = torch.gather(x, 2, ((last // w) * w + at).clamp(0, T - 1)[:, None, :, None].expand(-1, H, -1, d))
    tail.copy_(torch.where(mine[:, None, :, None], rows, tail))


def held(cache, scale, tail, pos, w, R):
    """The rows [B,H,w,d] that the cache stands for, float32: the current block's tokens up to `pos` from the tail."""
    B, H, _, d = cache.shape
    x = cache.float() * scale.repeat_interleave(R, -1)[..., :w, None]
    slot = torch.arange(w, device="cuda")
    cur = (pos.long() % w)[:, None]
    mine = (slot >= cur // R * R) & (slot <= cur)
    rows = torch.gather(tail.float(), 2, (slot % R)[None, None, :, None].expand(B, H, -1, d))
    return torch.where(mine[:, None, :, None], rows, x)


def plain_decode(s):
    c = s["case"]
    w, R, B, pos = c["window"], c["block"], c["B"], s["pos"]
    rows = torch.arange(B, device="cuda")
    cur = pos.long() % w
    s["k_tail"][rows, cur % R] = s["k"]
    s["v_tail"][rows, :, cur % R] = s["v"]
    n = torch.clamp(pos + 1, max=w)[:, None, None]
    keys = held(s["k_cache"][:, None], s["k_scale"][:, None], s["k_tail"][:, None], pos, w, R)[:, 0]
    scores = torch.matmul(s["q"].float(), keys.transpose(1, 2)) / math.sqrt(c["dk"])
    scores = torch.where(torch.arange(w, device="cuda") < n, scores, torch.full_like(scores, -math.inf))
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    values = held(s["v_cache"], s["v_scale"], s["v_tail"], pos, w, R)
    o = torch.matmul(p[:, :, None], values)[:, :, 0] / p.sum(-1, keepdim=True)
    close_blocks(s["k_cache"][:, None], s["k_scale"][:, None], s["k_tail"][:, None], cur, w, R, c["cache"])
    close_blocks(s["v_cache"], s["v_scale"], s["v_tail"], cur, w, R, c["cache"])
    pos.add_(1)
    return {"o": o.to(torch.bfloat16), **{n: s[n] for n in CACHE}}


def close_blocks(cache, scale, tail, cur, w, R, kind):
    """Sequences whose block is full with this token: its rows go from the tail into the cache."""
    B, H, _, d = cache.shape
    rows = torch.arange(B, device="cuda")
    full = (cur % R == R - 1) | (cur == w - 1)
    at = torch.clamp((cur // R * R)[:, None] + torch.arange(R, device="cuda"), max=w - 1)  # a short last block repeats its last row
    codes, scales = quantise(torch.gather(tail, 2, (at % R)[:, None, :, None].expand(-1, H, -1, d)), R, kind)
    raw = cache.view(torch.uint8)
    old = raw[rows[:, None], :, at].permute(0, 2, 1, 3)
    new = torch.where(full[:, None, None, None], codes.view(torch.uint8), old)
    raw[rows[:, None], :, at] = new.permute(0, 2, 1, 3)
    scale[rows, :, cur // R] = torch.where(full[:, None], scales[..., 0], scale[rows, :, cur // R])


# ------------------------------------------------------------------ work


def work(case):
    c = case
    if c["op"] in ("scan", "train"):
        tokens, e = sum(lengths_of(c)), 2 if c["dtype"] == "bf16" else 4
        channels = c["H"] * c["D"]
        state = c["B"] * channels * c["N"] * 4
        weights = channels * 4 * (c["N"] + 2 + (c["W"] + 1 if c["W"] else 0))
        fwd = tokens * e * (4 * channels + 2 * c["G"] * c["N"]) + state * (2 if c["carried"] else 1) + weights
        steps = tokens * channels * c["N"]
        if c["op"] == "scan":
            return {"bytes": fwd, "flops": 6 * steps}
        # the step reads x, dt, z, B, C and the gradient of y once and writes y and every gradient
        both = tokens * e * (8 * channels + 4 * c["G"] * c["N"]) + state * (3 if c["carried"] else 0) + 2 * weights
        return {"bytes": both, "flops": 20 * steps}
    if c["op"] == "step":
        e = 2 if c["dtype"] == "bf16" else 4
        channels = c["B"] * c["H"] * c["D"]
        rows = 4 + (2 * (c["W"] - 1) if c["W"] else 0)
        shared = c["H"] * c["D"] * 4 * (c["N"] + 2 + (c["W"] + 1 if c["W"] else 0))
        return {"bytes": channels * (8 * c["N"] + rows * e) + c["B"] * c["G"] * 2 * c["N"] * e + shared, "flops": channels * 6 * c["N"]}
    row = c["dk"] + c["H"] * c["dv"]
    if c["op"] == "fill":
        rows = sum(min(n, c["window"]) for n in lengths_of(c))
        return {"bytes": rows * row * 3, "flops": rows * row * 2}
    at = positions_of(c)
    rows = sum(min(p + 1, c["window"]) for p in at)
    tail = sum(p % c["window"] % c["block"] + 1 for p in at)
    io = c["B"] * 2 * (c["H"] * (c["dk"] + c["dv"]) + 2 * row)
    return {"bytes": rows * row + tail * row + io, "flops": rows * 2 * c["H"] * (c["dk"] + c["dv"])}


# ------------------------------------------------------------------ from the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return globals()["exact_" + case["op"]](s)


def exact_scan_of(s, x, dt, A, Bm, Cm, z, bias, feed, cw, cb, S0, before, T, lengths):
    """y [B,H,T,D] with zeros behind the ends, the last states and the last inputs: a token at a time, from the definition."""
    c = s["case"]
    W, per = c["W"], c["H"] // c["G"]
    window = list(before.unbind(2)) if W else []
    state, ys, inputs = S0, [], list(window)
    for t in range(T):
        xt = x[:, :, t]
        if W:
            window = window + [xt]
            inputs.append(xt)
            zc = cb + sum(cw[..., i] * window[-1 - i] for i in range(W))
            u = zc * torch.sigmoid(zc)
            window = window[1:]
        else:
            u = xt
        delta = torch.nn.functional.softplus(dt[:, :, t] + bias, threshold=1000)
        b, cc = (m[:, :, t].repeat_interleave(per, 1)[:, :, None] for m in (Bm, Cm))
        new = torch.exp(delta[..., None] * A) * state + (delta * u)[..., None] * b
        zt = z[:, :, t]
        y = ((new * cc).sum(-1) + feed * u) * zt * torch.sigmoid(zt)
        if lengths is not None:
            live = (t < lengths)[:, None, None]
            new, y = torch.where(live[..., None], new, state), torch.where(live, y, torch.zeros_like(y))
        state = new
        ys.append(y)
    return torch.stack(ys, 2), state, inputs


def exact_args(s):
    c = s["case"]
    d = {n: s[n].double() if s.get(n) is not None else None for n in ("x", "dt", "A", "Bm", "Cm", "z", "dt_bias", "feedthrough", "conv_weight", "conv_bias", "S0", "conv_state_in")}
    if d["S0"] is None:
        d["S0"] = torch.zeros(c["B"], c["H"], c["D"], c["N"], dtype=torch.float64, device="cuda")
    if d["conv_state_in"] is None and c["W"]:
        d["conv_state_in"] = torch.zeros(c["B"], c["H"], c["W"] - 1, c["D"], dtype=torch.float64, device="cuda")
    return d


def exact_scan(s):
    c = s["case"]
    d = exact_args(s)
    y, ST, inputs = exact_scan_of(s, *d.values(), c["T"], s["lengths"])
    if not c["W"]:
        return {"y": y, "ST": ST}
    ends = lengths_of(c)
    state = torch.stack([torch.stack([inputs[ends[b] + i][b] for i in range(c["W"] - 1)], 1) for b in range(c["B"])])
    return {"y": y, "ST": ST, "conv_state": state}


def exact_train(s):
    """The gradients by differentiating the definition, a token at a time, in 64 bits."""
    c = s["case"]
    if c["B"] * c["H"] * c["D"] * c["N"] * c["T"] > 300_000_000:
        return None
    d = exact_args(s)
    for v in d.values():
        if v is not None:
            v.requires_grad_(True)
    y, ST, _ = exact_scan_of(s, *d.values(), c["T"], s["lengths"])
    loss = (y * s["grad_y"].double()).sum()
    if s["grad_ST"] is not None:
        loss = loss + (ST * s["grad_ST"].double()).sum()
    loss.backward()
    out = {"y": y.detach(), "dx": d["x"].grad, "ddt": d["dt"].grad, "dz": d["z"].grad, "dB": d["Bm"].grad, "dC": d["Cm"].grad, "dA": d["A"].grad,
           "ddt_bias": d["dt_bias"].grad, "dfeed": d["feedthrough"].grad}
    if c["carried"]:
        out["dS0"] = d["S0"].grad
    if c["W"]:
        out.update(dconv_weight=d["conv_weight"].grad, dconv_bias=d["conv_bias"].grad)
        if c["carried"]:
            out["dconv_state_in"] = d["conv_state_in"].grad
    return out


def exact_step(s):
    c = s["case"]
    d = exact_args({**s, "S0": s["S"], "conv_state_in": s["conv_state"]})
    for n in ("x", "dt", "Bm", "Cm", "z"):
        d[n] = d[n][:, :, None]
    y, S, inputs = exact_scan_of(s, *d.values(), 1, None)
    return {"y": y[:, :, 0], "S": S, "conv_state": torch.stack(inputs[1:], 2)} if c["W"] else {"y": y[:, :, 0], "S": S}


def exact_codes(rows, cache):
    """(codes or None, scale) of one block's rows [H,n,d]: int8 codes have values next to a border that the scale's rounding decides."""
    most = rows.abs().amax((1, 2))
    if cache == "int8":
        return None, torch.where(most > 0, most / 127, torch.ones_like(most))
    scale = torch.where(most > 0, torch.exp2(torch.ceil(torch.log2(most / 448))), torch.ones_like(most))
    v = rows / scale[:, None, None]
    grid = torch.exp2(torch.clamp(torch.floor(torch.log2(v.abs().clamp(min=1e-30))), min=-6) - 3)
    return torch.round(v / grid) * grid, scale


def exact_rows(out, name, b, at, rows, blk, cache):
    """Puts one finished block of one sequence into the caches in `out`."""
    codes, scale = exact_codes(rows, cache)
    if codes is not None:
        out[name + "_cache"][b, :, at:at + rows.shape[1]] = codes
    out[name + "_scale"][b, :, blk] = scale


def exact_state(s):
    """The cache of the state in 64 bits, the keys with a head axis of 1."""
    out = {n: s[n].double() for n in CACHE if n != "pos"}
    for n in ("k_cache", "k_scale", "k_tail"):
        out[n] = out[n][:, None]
    return out


def exact_out(s, out):
    for n in ("k_cache", "k_scale", "k_tail"):
        out[n] = out[n][:, 0]
    if s["case"]["cache"] == "int8":
        out["k_cache"] = out["v_cache"] = None
    return out


def exact_fill(s):
    """The state that decoding the prompt a token at a time leaves: each block as it was when it was last full."""
    c = s["case"]
    w, R = c["window"], c["block"]
    if c["B"] * -(-w // R) > 20000:
        return None
    out = exact_state(s)
    x = {"k": s["k"][:, None].double(), "v": s["v"].double()}
    for b, end in enumerate(lengths_of(c)):
        for blk in range(-(-w // R)):
            at, stop = blk * R, min(blk * R + R, w)
            if end < stop:
                continue
            first = (end - stop) // w * w + at  # the last round in which the block became full
            for n in ("k", "v"):
                exact_rows(out, n, b, at, x[n][b, :, first:first + stop - at], blk, c["cache"])
        slot = (end - 1) % w
        if end and (slot + 1) % R and slot + 1 < w:
            count = slot % R + 1
            for n in ("k", "v"):
                out[n + "_tail"][b, :, :count] = x[n][b, :, end - count:end]
    return exact_out(s, out)


def exact_decode(s):
    """A sequence at a time."""
    c = s["case"]
    w, R = c["window"], c["block"]
    out = exact_state(s)
    o = torch.empty(c["B"], c["H"], c["dv"], dtype=torch.float64, device="cuda")
    for b, pos in enumerate(positions_of(c)):
        slot, n = pos % w, min(pos + 1, w)
        at, i = slot // R * R, slot % R
        out["k_tail"][b, 0, i], out["v_tail"][b, :, i] = s["k"][b].double(), s["v"][b].double()
        rows = {}
        for m in ("k", "v"):
            r = out[m + "_cache"][b, :, :n] * out[m + "_scale"][b].repeat_interleave(R, -1)[:, :n, None]
            r[:, at:slot + 1] = out[m + "_tail"][b, :, :i + 1]
            rows[m] = r
        p = torch.softmax(s["q"][b].double() @ rows["k"][0].t() / math.sqrt(c["dk"]), -1)
        o[b] = (p[:, None] @ rows["v"])[:, 0]
        if i == R - 1 or slot == w - 1:
            for m in ("k", "v"):
                exact_rows(out, m, b, at, out[m + "_tail"][b, :, :i + 1], at // R, c["cache"])
    return {"o": o, **exact_out(s, out)}
