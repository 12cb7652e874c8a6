"""GPU tests of the scan's backward at state sizes and head dimensions whose blocks
run one, two or four an SM, so that sequences are cut differently: forward and every
gradient against the float64 reference."""
import pytest
import torch

from tests import ssm_reference as ref
from tests.test_gpu_ssm import check_all

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,D,N,T,lengths", [
    (1, 2, 16, 16, 700, None), (2, 3, 16, 16, 333, [333, 97]), (1, 1, 32, 32, 400, None), (2, 1, 16, 128, 300, [300, 33]),
    (1, 2, 128, 128, 150, None), (1, 1, 64, 64, 260, None), (1, 14, 64, 128, 130, None)])
@pytest.mark.parametrize("saved", [False, True])
def test_cuts(cuda_ok, B, H, D, N, T, lengths, saved):
    check_all(ref.inputs(B, H, T, D, N, dtype=torch.bfloat16 if N == 16 else torch.float32, seed=T), lengths=lengths, saved=saved)
