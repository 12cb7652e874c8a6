"""GPU test of the scan's gradients where decays are strong: each element of dA and
of ddt against its formula in float64, within a bound relative to the magnitudes of
that element's own terms.

  dA = sum_t delta G_t a_t s_{t-1}     ddt_t = u sum_n G_t B_t + sum_n G_t a_t s_{t-1} A
  a_t = exp(delta A)   G_t = C_t p_t + a_{t+1} G_{t+1}

Nearly all of s_t is delta u B_t there, so a form of a_t s_{t-1} as a difference from
s_t has no digits left.  Bound: with |x| <= 25 the exponent (in powers of two), two
roundings of 2^-24 |x| leave 35 2^-24 of a decay (its argument, ln 2), the decay of the
term and those of the chains as much each, exponentials 4 2^-24: 128 2^-24; a token
rounds each of the two chains and the sums over tokens and states by 2^-24 a few times:
8 T 2^-24."""
import pytest
import torch

import gated_linear_attention_ddts_b200 as rdm
from tests import ssm_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [16, 64, 128])
@pytest.mark.parametrize("T", [1, 5, 12, 100])
def test_gradients_of_strong_decays(cuda_ok, dtype, N, T):
    B, H, D = 2, 2, 16
    i = ref.inputs(B, H, T, D, N, W=0, dtype=dtype, seed=N + T, z=False, feed=False, gates="activated")
    g = torch.Generator().manual_seed(7)
    i["A"] = -torch.linspace(1.0, 128.0, N).expand(H, D, N).contiguous() * torch.exp(0.1 * torch.randn(H, D, N, generator=g).clamp(-2, 2))
    i["dt"] = (0.05 + 0.05 * torch.rand(B, H, T, D, generator=g)).to(dtype)
    gy = torch.randn(B, H, T, D, generator=g).to(dtype)
    gST = torch.randn(B, H, D, N, generator=g)
    d = {n: (t.cuda() if t is not None else None) for n, t in i.items()}
    got = rdm.rdm_ssm_bwd(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], gy.cuda(), gST.cuda(), S0=d["S0"], gates="activated")
    x, dt, A, S0, p = (t.double() for t in (i["x"], i["dt"], i["A"], i["S0"], gy))
    Bm, Cm = i["Bm"].double()[:, :, :, None], i["Cm"].double()[:, :, :, None]

    def sums(mag):  # the formula's values, or those of its terms' magnitudes
        f = torch.abs if mag else (lambda t: t)
        s, states, a = f(S0), [], [torch.exp(dt[:, :, t, :, None] * A) for t in range(T)]
        for t in range(T):
            states.append(s)
            s = a[t] * s + f((dt * x)[:, :, t, :, None] * Bm[:, :, t])
        G, dA, ddt = f(gST.double()), torch.zeros_like(A), torch.zeros_like(dt)
        for t in reversed(range(T)):
            G = f(Cm[:, :, t] * p[:, :, t, :, None]) + G
            w = G * a[t] * states[t]
            dA += (dt[:, :, t, :, None] * w).sum(0)
            ddt[:, :, t] = f(x[:, :, t]) * (G * f(Bm[:, :, t])).sum(-1) + (w * f(A)).sum(-1)
            G = a[t] * G
        return dA, ddt

    (dA, ddt), (mA, mt) = sums(False), sums(True)
    for name, want, terms, half in (("dA", dA, mA, 0.0), ("ddt", ddt, mt, torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else 0.0)):
        off = (got[name].cpu().double() - want).abs()
        worst = (off / (half * want.abs() + (128 + 8 * T) * 2.0 ** -24 * terms)).max().item()
        assert worst <= 1, f"{name}: {worst:.3g} of the bound"
