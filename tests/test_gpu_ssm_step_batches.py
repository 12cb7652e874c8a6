"""GPU tests of rdm_ssm_step for batches so large that a block takes eight sequences:
groups of eight that are not full, blocks that span heads or are not full of channels,
every state size, against the float64 reference over two tokens."""
import pytest
import torch

import gated_linear_attention_ddts_b200 as rdm
from tests import ssm_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,D,H,G,B,W", [
    (16, 16, 5, 5, 453, 4), (16, 64, 14, 2, 67, 1), (16, 16, 3, 1, 891, 0), (16, 128, 32, 4, 17, 4),
    (32, 16, 7, 7, 229, 0), (32, 128, 8, 2, 29, 3),
    (64, 16, 9, 3, 101, 2), (64, 32, 6, 1, 77, 4), (64, 128, 16, 16, 8, 4),
    (128, 16, 5, 5, 93, 4), (128, 128, 32, 1, 2, 4), (128, 128, 7, 7, 9, 1), (128, 64, 13, 13, 13, 0)])
def test_eight_sequences_a_block(cuda_ok, dtype, N, D, H, G, B, W):
    blocks = -(-H * D // (1024 // N)) * B
    assert blocks > 6 * torch.cuda.get_device_properties(0).multi_processor_count
    z, gates = B % 3 != 0, "activated" if W == 3 else "preact"
    i = ref.inputs(B, H, 2, D, N, G=G, W=W, dtype=dtype, seed=N + B, z=z, feed=B % 2 == 1, gates=gates)
    yr, Sr, csr = ref.scan(i, gates=gates)
    d = {n: (t.cuda() if t is not None else None) for n, t in i.items()}
    # updated in place, with rows of another sequence behind the last that stay
    S = torch.full((B + 9, H, D, N), 7.0, device="cuda")
    S[:B] = d["S0"]
    cs = torch.full((B + 9, H, W - 1, D), 7.0, device="cuda", dtype=dtype) if W > 1 else None
    if W > 1:
        cs[:B] = d["conv_state_in"]
    for t in range(2):
        y = torch.full((B + 9, H, D), 7.0, device="cuda", dtype=dtype)
        row = {n: d[n][:, :, t].contiguous() if d[n] is not None else None for n in ("x", "dt", "Bm", "Cm", "z")}
        rdm.rdm_ssm_step(row["x"], row["dt"], d["A"], row["Bm"], row["Cm"], S[:B], z=row["z"], dt_bias=d["dt_bias"],
                         feedthrough=d["feedthrough"], conv_weight=d["conv_weight"], conv_bias=d["conv_bias"],
                         conv_state=cs[:B] if W > 1 else None, gates=gates, y=y[:B])
        ref.assert_near(y[:B], yr[:, :, t], 2 + N, f"token {t}")
        assert (y[B:] == 7).all()
    ref.assert_near(S[:B], Sr, 2 + N, "state")
    assert (S[B:] == 7).all()
    if W > 1:
        assert torch.equal(cs[:B].cpu().double(), csr) and (cs[B:] == 7).all()
