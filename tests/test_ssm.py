"""Selective scan without a GPU: the float64 reference against a worked example
and against differences, and the refusals of the C ABI and of the binding."""
import ctypes
import math

import pytest
import torch

import gated_linear_attention_ddts_b200 as rdm
from gated_linear_attention_ddts_b200 import _binding
from tests import ssm_reference as ref

FAKE = 1 << 20  # aligned placeholder; every call below is refused before it is used


@pytest.fixture(scope="module")
def lib():
    from gated_linear_attention_ddts_b200 import build
    build.build()
    return _binding.load()


def test_reference_worked_example():
    """One channel, two equal states, two tokens, by hand."""
    one = torch.ones(1, 1, 2, 1)
    i = dict(x=torch.tensor([1.0, 2.0]).view(1, 1, 2, 1), dt=0.5 * one, Bm=torch.ones(1, 1, 2, 2), Cm=torch.ones(1, 1, 2, 2),
             A=-torch.ones(1, 1, 2), dt_bias=None, z=None, feedthrough=torch.tensor([[3.0]]),
             conv_weight=torch.tensor([[[1.0, 10.0]]]), conv_bias=None, conv_state_in=torch.full((1, 1, 1, 1), 0.5), S0=None)
    y, ST, cs = ref.scan(i, silu=False, gates="activated")
    u1, u2 = 1 + 5.0, 2 + 10.0
    s1 = 0.5 * u1
    s2 = math.exp(-0.5) * s1 + 0.5 * u2
    assert torch.allclose(y.flatten(), torch.tensor([2 * s1 + 3 * u1, 2 * s2 + 3 * u2], dtype=torch.float64))
    assert torch.allclose(ST.flatten(), torch.tensor([s2, s2], dtype=torch.float64))
    assert cs.item() == 2.0


def test_reference_gradients_match_differences():
    i = ref.inputs(2, 2, 7, 3, 4, G=1, W=3, seed=5)
    i = {n: t.double() for n, t in i.items()}
    g = torch.Generator().manual_seed(6)
    w = [torch.randn(2, 2, 7, 3, generator=g).double(), torch.randn(2, 2, 3, 4, generator=g).double(),
         torch.randn(2, 2, 2, 3, generator=g).double()]
    lengths = [7, 4]

    def loss(j):
        return sum((a * b).sum() for a, b in zip(ref.scan(j, lengths), w)).item()

    grads = ref.gradients(i, *w, lengths=lengths)
    for n, t in i.items():
        v = torch.randn(t.shape, generator=g).double()
        h = 1e-5
        diff = (loss({**i, n: t + h * v}) - loss({**i, n: t - h * v})) / (2 * h)
        assert diff == pytest.approx((grads[ref.NAMES[n]] * v).sum().item(), rel=1e-6, abs=1e-7), n


def fwd_args(**kw):
    base = dict(B=2, H=4, G=2, T=8, D=64, N=16, W=0, dtype=1, gate_inputs=1, conv_silu=1, x=FAKE, dt=FAKE, Bm=FAKE, Cm=FAKE,
                A=FAKE, y=FAKE)
    return _binding.SsmArgs(**{**base, **kw})


BAD = [(dict(B=0), 1), (dict(H=0), 1), (dict(G=0), 1), (dict(G=3), 1), (dict(T=-1), 1), (dict(D=48), 2), (dict(N=8), 2), (dict(N=256), 2),
       (dict(W=5, conv_weight=FAKE), 2), (dict(W=-1), 1), (dict(W=2), 1), (dict(conv_weight=FAKE), 1), (dict(dtype=2), 1),
       (dict(gate_inputs=2), 1), (dict(x=None), 1), (dict(A=None), 1), (dict(Cm=None), 1), (dict(x=FAKE + 8), 1), (dict(A=FAKE + 4), 1),
       (dict(lengths=FAKE + 2), 1), (dict(S0=FAKE + 8), 1), (dict(conv_bias=FAKE), 1), (dict(conv_state_in=FAKE), 1),
       (dict(dt_bias=FAKE, gate_inputs=0), 1), (dict(T=(1 << 30) + 1), 1), (dict(workspace=FAKE + 8), 1)]


@pytest.mark.parametrize("kw,status", BAD + [(dict(y=None), 1), (dict(y=FAKE + 2), 1), (dict(ST=FAKE + 8), 1), (dict(conv_state_out=FAKE), 1)])
def test_fwd_refusals(lib, kw, status):
    assert lib.rdm_ssm_fwd(ctypes.byref(fwd_args(**kw)), None) == status


@pytest.mark.parametrize("kw,status", BAD)
def test_bwd_refusals(lib, kw, status):
    a = _binding.SsmBwdArgs(fwd_args(**kw), grad_y=FAKE, grad_x=FAKE, grad_dt=FAKE, grad_B=FAKE, grad_C=FAKE, grad_A=FAKE)
    assert lib.rdm_ssm_bwd(ctypes.byref(a), None) == status
    assert lib.rdm_ssm_bwd_workspace_size(ctypes.byref(a)) == ctypes.c_size_t(-1).value


@pytest.mark.parametrize("kw,f,status", [
    (dict(grad_y=None), {}, 1), (dict(grad_x=None), {}, 1), (dict(grad_A=None), {}, 1), (dict(grad_dt=FAKE + 8), {}, 1),
    (dict(), dict(z=FAKE), 1), (dict(grad_dt_bias=FAKE), dict(gate_inputs=0), 1), (dict(grad_feedthrough=FAKE), {}, 1),
    (dict(grad_conv_weight=FAKE), {}, 1), (dict(grad_conv_state_out=FAKE), {}, 1), (dict(grad_S0=FAKE + 4), {}, 1),
    (dict(), {}, 5), (dict(), dict(workspace=FAKE, workspace_bytes=16), 5)])
def test_bwd_gradient_refusals(lib, kw, f, status):
    base = dict(grad_y=FAKE, grad_x=FAKE, grad_dt=FAKE, grad_B=FAKE, grad_C=FAKE, grad_A=FAKE)
    a = _binding.SsmBwdArgs(fwd_args(**f), **{**base, **kw})
    assert lib.rdm_ssm_bwd(ctypes.byref(a), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(G=3), 1), (dict(D=48), 2), (dict(N=8), 2), (dict(W=5, conv_weight=FAKE, conv_state=FAKE), 2), (dict(S=None), 1),
    (dict(S=FAKE + 8), 1), (dict(W=2, conv_weight=FAKE), 1), (dict(conv_state=FAKE), 1), (dict(W=1, conv_weight=FAKE, conv_state=FAKE), 1),
    (dict(dt_bias=FAKE, gate_inputs=0), 1), (dict(y=None), 1), (dict(dtype=3), 1)])
def test_step_refusals(lib, kw, status):
    base = dict(B=2, H=4, G=2, D=64, N=16, W=0, dtype=1, gate_inputs=1, conv_silu=1, x=FAKE, dt=FAKE, Bm=FAKE, Cm=FAKE, A=FAKE, S=FAKE, y=FAKE)
    assert lib.rdm_ssm_step(ctypes.byref(_binding.SsmStepArgs(**{**base, **kw})), None) == status


@pytest.mark.parametrize("kw", [
    dict(S0=FAKE + 64, ST=FAKE + 64), dict(y=FAKE), dict(z=FAKE + 64, y=FAKE + 64), dict(x=FAKE + 64, y=FAKE + 64),
    dict(W=2, conv_weight=FAKE, conv_state_in=FAKE + 64, conv_state_out=FAKE + 64)])
def test_fwd_refuses_outputs_in_place(lib, kw):
    """Segments read the carried state while the last one writes the new one."""
    assert lib.rdm_ssm_fwd(ctypes.byref(fwd_args(**{"y": FAKE + 128, **kw})), None) == 1


@pytest.mark.parametrize("kw", [
    dict(grad_ST=FAKE, grad_S0=FAKE), dict(grad_conv_state_in=FAKE, grad_conv_state_out=FAKE)])
def test_bwd_refuses_outputs_in_place(lib, kw):
    base = dict(grad_y=FAKE, grad_x=FAKE, grad_dt=FAKE, grad_B=FAKE, grad_C=FAKE, grad_A=FAKE)
    a = _binding.SsmBwdArgs(fwd_args(W=2, conv_weight=FAKE), **{**base, **kw})
    assert lib.rdm_ssm_bwd(ctypes.byref(a), None) == 1


def test_refuses_more_channels_than_an_index_holds(lib):
    a = fwd_args(B=1, H=1 << 25, G=1, T=1, y=FAKE + 128)
    assert lib.rdm_ssm_fwd(ctypes.byref(a), None) == 1
    s = _binding.SsmStepArgs(B=1, H=1 << 25, G=1, D=64, N=16, W=0, dtype=1, gate_inputs=1, conv_silu=1, x=FAKE, dt=FAKE,
                             Bm=FAKE, Cm=FAKE, A=FAKE, S=FAKE, y=FAKE)
    assert lib.rdm_ssm_step(ctypes.byref(s), None) == 1


def test_sizes(lib):
    assert rdm.rdm_ssm_saved_states_size(2, 3, 33, 64, 16) == 2 * 3 * 3 * 64 * 16 * 4
    assert rdm.rdm_ssm_saved_states_size(2, 3, 33, 64, 17) == 0


def test_binding_refuses_cpu_tensors(lib):
    i = ref.inputs(1, 1, 4, 16, 16, W=0, carried=False)
    with pytest.raises(ValueError):
        rdm.rdm_ssm_fwd(i["x"], i["dt"], i["A"], i["Bm"], i["Cm"])
    with pytest.raises(ValueError):
        rdm.rdm_ssm_step(i["x"][:, :, 0], i["dt"][:, :, 0], i["A"], i["Bm"][:, :, 0], i["Cm"][:, :, 0], torch.zeros(1, 1, 16, 16))
