"""GPU test of the interference probe with each of its GEMMs."""
import pytest
import torch

from shard_placement_amd import configs, harness, probe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gemm", probe.GEMMS)
def test_probe_runs_each_gemm(gemm):
    w = configs.get(1)
    st = harness.setup(w, device="cuda:0", with_ag=False)
    r = probe.run([("default launches", st.plan, 0, 0)], harness.rs_bytes(w), iters=4, M=512, N=256,
                  K=256, gemm=gemm)
    assert r["t_gemm_alone_ms"] > 0 and len(r["modes"]) == 1
    assert {"matmul": "torch.matmul", "forward": "forward of 512 tokens",
            "weight-grad": "gradient of a [512,256] weight"}[gemm] in r["gemm"]


@pytest.mark.parametrize("gemm", probe.GEMMS)
def test_probe_gemms_are_the_product(gemm):
    """Each call computes M x N sums of K terms on the current stream."""
    call, _ = probe._gemm(gemm, 96, 64, 40, torch.device("cuda:0"))
    got = call()
    if gemm == "weight-grad":
        assert got is None
    else:
        assert got.shape == (96, 64)
    with pytest.raises(ValueError, match="gemm must be one of"):
        probe._gemm("none", 1, 1, 1, "cuda")
