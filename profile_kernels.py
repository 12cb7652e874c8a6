#!/usr/bin/env python
"""Small launches of each kernel, the command that profiler captures wrap.

    python profile_kernels.py fwd1|fwd1pre|fwd1feed|fwd1lr|fwd2|fwdbwd3|bwdwide3|decode4|conv1|ska1|ska4|
                              ssm1|ssmbwd1|ssmstep|q8fill|q8dec

One workload per call: the mode draws its inputs on the device, runs the
kernel(s) three times and synchronises.  fwd1 is the 130M-scale layer forward
(B8 H6 T2048 d_k64 d_v128), fwd1pre the same with the gates passed before
their activations, fwd2 the long-context forward (B1 H16 T32768 d_k=d_v=128),
fwdbwd3 the training forward (saving chunk states) and backward (B4 H16 T4096
d_k64 d_v128), bwdwide3 the same with one chunk of every 16th head too wide for
one decay reference (g scaled by 40 there; the exact backward recomputes those
heads), decode4 four steps of the batched decode (B256 H16 d_k64 d_v128;
only 4 steps of inputs are drawn instead of 1024, the kernel is the same),
fwd1feed the 130M-scale layer forward with the feedthrough, fwd1lr the same
layer with the gates passed before their activations and a rank-16 beta_hat, conv1 the
ShortConv forward and backward (width 4, SiLU) on a q-shaped tensor of that
layer (B8 H6 T2048 D64), ska1 the sliding-window shared-key attention forward
(B8 H12 T2048 d_k=d_v=64, window 512) and ska4 its batched decode step against
full ring caches (B256 H16 d_k=d_v=128, window 512); ssm1 the selective scan
forward (B8 H24 T512 D64 N16, width-4 convolution, gate), ssmbwd1 its forward with
saved states and backward (B4), ssmstep one token of it (B256 H16 D128 N64), q8fill
four prompts into 8-bit rings (H16 T16384 d128, 8200 slots in blocks of 16, int8) and
q8dec the decode step of ska4 over 8-bit rings (e4m3, blocks of 64).
Exit status 0 only when the library's device status word is clear."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import gated_linear_attention_ddts_b200 as rdm  # noqa: E402
from gated_linear_attention_ddts_b200.workloads import (SKA_DEC, SKA_FWD, WORKLOADS,  # noqa: E402
                                                        draw_decode, draw_lowrank, draw_workload)

SEQ = ("q", "k", "v", "g", "tau", "beta")


def main(mode: str) -> int:
    if mode in ("fwd1", "fwd1pre", "fwd1feed", "fwd2", "fwd1lr"):
        w = WORKLOADS[2 if mode == "fwd2" else 1]
        pre = mode in ("fwd1pre", "fwd1lr")
        x = draw_workload(w, device="cuda", preact=pre)
        d = torch.randn(w.H, w.dv, device="cuda") if mode == "fwd1feed" else None
        lr = draw_lowrank(w.B, w.H, w.T, w.dv, 16, seed=w.seed + 40, device="cuda") \
            if mode == "fwd1lr" else None
        for _ in range(3):
            rdm.rdm_ddts_fwd(*(x[n] for n in SEQ[:5]), None if lr else x["beta"], x["S0"],
                             return_state=w.return_state, gates="preact" if pre else "activated",
                             feedthrough=d, beta_lowrank=lr)
    elif mode == "conv1":
        w = WORKLOADS[1]
        x = torch.randn(w.B, w.H, w.T, w.dk, device="cuda").to(torch.bfloat16)
        wt = torch.randn(w.H, w.dk, 4, device="cuda") / 4
        b = torch.randn(w.H, w.dk, device="cuda") * 0.1
        gy = torch.randn_like(x)
        for _ in range(3):
            rdm.rdm_shortconv_fwd(x, wt, b, None, silu=True)
            rdm.rdm_shortconv_bwd(x, wt, b, None, gy, None, silu=True)
    elif mode in ("ska1", "ska4"):
        gen = torch.Generator(device="cuda").manual_seed(5)
        if mode == "ska1":
            B, H, T, d, win = SKA_FWD
            q = torch.randn(B, H, T, d, device="cuda", generator=gen).to(torch.bfloat16)
            k = torch.randn(B, T, d, device="cuda", generator=gen).to(torch.bfloat16)
            v = torch.randn(B, H, T, d, device="cuda", generator=gen).to(torch.bfloat16)
            for _ in range(3):
                rdm.rdm_ska_fwd(q, k, v, win)
        else:
            B, H, d, win, _ = SKA_DEC
            kc = torch.randn(B, win, d, device="cuda", generator=gen).to(torch.bfloat16)
            vc = torch.randn(B, H, win, d, device="cuda", generator=gen).to(torch.bfloat16)
            q = torch.randn(B, H, d, device="cuda", generator=gen).to(torch.bfloat16)
            k = torch.randn(B, d, device="cuda", generator=gen).to(torch.bfloat16)
            v = torch.randn(B, H, d, device="cuda", generator=gen).to(torch.bfloat16)
            pos = torch.full((B,), 1000, dtype=torch.int32, device="cuda")
            for _ in range(3):
                rdm.rdm_ska_decode(q, k, v, kc, vc, pos)
    elif mode in ("ssm1", "ssmbwd1", "ssmstep"):
        step = mode == "ssmstep"
        B, H, T, D, N = {"ssm1": (8, 24, (512,), 64, 16), "ssmbwd1": (4, 24, (512,), 64, 16),
                         "ssmstep": (256, 16, (), 128, 64)}[mode]
        bf = dict(device="cuda", dtype=torch.bfloat16)
        x, dt, z = torch.randn(B, H, *T, D, **bf), torch.randn(B, H, *T, D, **bf), torch.randn(B, H, *T, D, **bf)
        Bm, Cm = torch.randn(B, 1, *T, N, **bf), torch.randn(B, 1, *T, N, **bf)
        A = -torch.arange(1.0, N + 1, device="cuda").expand(H, D, N).contiguous()
        given = dict(z=z, dt_bias=torch.full((H, D), -4.0, device="cuda"), feedthrough=torch.ones(H, D, device="cuda"),
                     conv_weight=torch.randn(H, D, 4, device="cuda") / 2, conv_bias=torch.zeros(H, D, device="cuda"))
        if step:
            S, cs = torch.zeros(B, H, D, N, device="cuda"), torch.zeros(B, H, 3, D, **bf)
        saved = rdm.rdm_ssm_saved_states(x, A) if mode == "ssmbwd1" else None
        for _ in range(3):
            if step:
                rdm.rdm_ssm_step(x, dt, A, Bm, Cm, S, conv_state=cs, **given)
                continue
            y, _, _ = rdm.rdm_ssm_fwd(x, dt, A, Bm, Cm, saved_states=saved, **given)
            if saved is not None:
                rdm.rdm_ssm_bwd(x, dt, A, Bm, Cm, y, saved_states=saved, **given)
    elif mode in ("q8fill", "q8dec"):
        bf = dict(device="cuda", dtype=torch.bfloat16)
        if mode == "q8fill":
            cache = rdm.rdm_ska_q8_cache(4, 16, 128, 128, 8200, block=16, dtype=torch.int8)
            k, v = torch.randn(4, 16384, 128, **bf), torch.randn(4, 16, 16384, 128, **bf)
            for _ in range(3):
                rdm.rdm_ska_q8_fill(k, v, *cache)
        else:
            B, H, d, win, _ = SKA_DEC
            cache = rdm.rdm_ska_q8_cache(B, H, d, d, win)
            rdm.rdm_ska_q8_fill(torch.randn(B, win, d, **bf), torch.randn(B, H, win, d, **bf), *cache)
            q, k, v = torch.randn(B, H, d, **bf), torch.randn(B, d, **bf), torch.randn(B, H, d, **bf)
            cache[6].copy_(1000 + 37 * torch.arange(B, device="cuda"))
            for _ in range(3):
                rdm.rdm_ska_q8_decode(q, k, v, *cache)
    elif mode in ("fwdbwd3", "bwdwide3"):
        w = WORKLOADS[3]
        x = draw_workload(w, device="cuda")
        if mode == "bwdwide3":
            gw = x["g"].float()
            gw[:, ::16, 64 * 20:64 * 21] *= 40.0
            x["g"] = gw.clamp(min=0.05).to(torch.bfloat16)
        saved = torch.empty(rdm.rdm_ddts_saved_states_size(w.B, w.H, w.T, w.dk, w.dv, 64) // 4,
                            device="cuda")
        for _ in range(3):
            rdm.rdm_ddts_fwd(*(x[n] for n in SEQ), x["S0"], saved_states=saved)
            rdm.rdm_ddts_bwd(*(x[n] for n in SEQ), x["S0"], x["dO"], None, saved)
    elif mode == "decode4":
        w = WORKLOADS[4]
        xd = draw_decode(w.B, w.H, w.dk, w.dv, 4, device="cuda")
        S = torch.zeros(w.B, w.H, w.dk, w.dv, device="cuda")
        for s in range(4):
            rdm.rdm_ddts_decode_step(*(xd[n][s] for n in SEQ), S)
    else:
        raise SystemExit(f"unknown mode {mode}")
    torch.cuda.synchronize()
    st = rdm.rdm_ddts_sync_status()
    print(mode, "status", st)
    return 0 if st == 0 else 1


if __name__ == "__main__":
    sys.exit(main(sys.argv[1]))
