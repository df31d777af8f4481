"""GPU test that the interference probe's GEMMs compute the products they are
named for, from what their calls hold."""
import inspect

import pytest
import torch

from shard_placement_amd import probe
from tests import linear_ref as ref
from tests.test_linear_gpu import within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(96, 64, 40), (200, 136, 333), (512, 256, 256)])
@pytest.mark.parametrize("gemm", probe.GEMMS)
def test_probe_gemm_results(gemm, M, N, K):
    """M x N sums of K terms: those of the call's operands, in bf16."""
    call, _ = probe._gemm(gemm, M, N, K, torch.device("cuda:0"))
    held = inspect.getclosurevars(call).nonlocals
    got = call()
    if gemm == "matmul":
        a, b = held["a"].double(), held["b"].double()
    elif gemm == "forward":
        a, b = held["x"].double(), held["layer"].weight.double().T.contiguous()
    else:
        x8 = held["x8"]
        a = held["dy"].double().T.contiguous()
        b = ref.unpack_ref(x8.data.view(torch.uint8), x8.scales.view(torch.uint8), N)
        got = held["layer"].weight_grad
    assert a.shape == (M, K) and b.shape == (K, N) and got.shape == (M, N)
    want, e = a @ b, (K + 8) * ref.F32 * (a.abs() @ b.abs())
    within(got, want, e + ref.BF16 * (want.abs() + e), gemm)
