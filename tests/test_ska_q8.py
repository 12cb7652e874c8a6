"""8-bit ring cache without a GPU: the reference's rounding, and the refusals of
the C ABI and of the binding."""
import ctypes

import pytest
import torch

import gated_linear_attention_ddts_b200 as rdm
from gated_linear_attention_ddts_b200 import _binding
from tests import ska_q8_reference as ref

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from gated_linear_attention_ddts_b200 import build
    build.build()
    return _binding.load()


def test_reference_rounds_to_the_e4m3_values():
    x = torch.randn(64, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16) * 3
    q, s = ref.round_block(x, torch.float8_e4m3fn)
    assert 224 < (x.abs().max().item() / s) <= 448
    assert torch.equal(q, (x.float() / s).to(torch.float8_e4m3fn).double())


@pytest.mark.parametrize("most,scale", [(448.0, 1.0), (450.0, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (1.7578125, 2.0 ** -7)])
def test_reference_e4m3_scales(most, scale):
    assert ref.round_block(torch.tensor([[most, -0.5 * most]]).to(torch.bfloat16), torch.float8_e4m3fn)[1] == scale


def test_reference_int8_by_hand():
    q, s = ref.round_block(torch.tensor([[127.0, -63.5, 0.5, 1.5]]).to(torch.bfloat16), torch.int8)
    assert s == 1.0 and q.tolist() == [[127, -64, 0, 2]]
    assert ref.round_block(torch.zeros(2, 4, dtype=torch.bfloat16), torch.int8)[1] == 1.0


def cache(**kw):
    base = dict(B=2, H=4, dk=64, dv=128, window=100, block=16, type=0, k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, k_tail=FAKE,
                v_tail=FAKE, pos=FAKE)
    return _binding.SkaQ8Cache(**{**base, **kw})


BAD = [(dict(B=0), 1), (dict(H=0), 1), (dict(window=0), 1), (dict(window=32769), 2), (dict(block=0), 2), (dict(block=48), 2),
       (dict(block=128), 2), (dict(dk=32), 2), (dict(dv=256), 2), (dict(type=2), 1), (dict(k=None), 1), (dict(v_scale=None), 1),
       (dict(k_tail=FAKE + 8), 1), (dict(pos=FAKE + 2), 1), (dict(v=FAKE + 4), 1)]


@pytest.mark.parametrize("kw,status", BAD)
def test_cache_refusals(lib, kw, status):
    f = _binding.SkaQ8FillArgs(cache(**kw), 8, 1, FAKE, FAKE, None)
    assert lib.rdm_ska_q8_fill(ctypes.byref(f), None) == status
    d = _binding.SkaQ8DecodeArgs(cache(**kw), 0.0, 1, FAKE, FAKE, FAKE, FAKE, 1, None, 0)
    assert lib.rdm_ska_q8_decode(ctypes.byref(d), None) == status
    assert lib.rdm_ska_q8_decode_workspace_size(ctypes.byref(d)) == ctypes.c_size_t(-1).value


@pytest.mark.parametrize("T,dtype,k,lengths,status", [
    (-1, 1, FAKE, None, 1), (8, 0, FAKE, None, 2), (8, 7, FAKE, None, 1), (8, 1, None, None, 1), (8, 1, FAKE + 8, None, 1),
    (8, 1, FAKE, FAKE + 2, 1), ((1 << 30) + 1, 1, FAKE, None, 1)])
def test_fill_refusals(lib, T, dtype, k, lengths, status):
    a = _binding.SkaQ8FillArgs(cache(), T, dtype, k, FAKE, lengths)
    assert lib.rdm_ska_q8_fill(ctypes.byref(a), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(scale=-1.0), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(dtype=0), 2), (dict(dtype=5), 1),
    (dict(q=None), 1), (dict(o=None), 1), (dict(k=FAKE + 2), 1), (dict(workspace=FAKE + 8), 1)])
def test_decode_refusals(lib, kw, status):
    base = dict(cache=cache(), scale=0.0, dtype=1, q=FAKE, k=FAKE, v=FAKE, o=FAKE)
    assert lib.rdm_ska_q8_decode(ctypes.byref(_binding.SkaQ8DecodeArgs(**{**base, **kw})), None) == status


def test_binding_refuses(lib):
    c = rdm.rdm_ska_q8_cache(1, 2, 64, 64, 40, block=16, device="cpu")
    assert [tuple(t.shape) for t in c] == [(1, 40, 64), (1, 2, 40, 64), (1, 3), (1, 2, 3), (1, 16, 64), (1, 2, 16, 64), (1,)]
    with pytest.raises(ValueError):  # not on a GPU
        rdm.rdm_ska_q8_decode(torch.zeros(1, 2, 64), torch.zeros(1, 64), torch.zeros(1, 2, 64), *c)
    with pytest.raises(TypeError):
        rdm.rdm_ska_q8_cache(1, 2, 64, 64, 40, dtype=torch.uint8, device="cpu")
