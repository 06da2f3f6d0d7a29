"""What gemm_device_status says after several operators' calls."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [100, 1500])
def test_a_wait_given_up_is_reported_also_after_an_index_out_of_range(rows):
    # (an index out of range leaves every result as documented, a wait given up leaves none)
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    X = torch.ones(rows, 256, dtype=torch.bfloat16, device="cuda")
    W = torch.ones(520, 256, dtype=torch.bfloat16, device="cuda")
    down = torch.ones(4, 16, 256, dtype=torch.bfloat16, device="cuda")
    up = torch.ones(4, 520, 16, dtype=torch.bfloat16, device="cuda")
    Y = torch.empty(rows, 520, dtype=torch.bfloat16, device="cuda")
    good = torch.zeros(rows, dtype=torch.int32, device="cuda")
    bad = good.clone()
    bad[7] = 4
    with Gemm() as g:
        g.run_adapters(X, W, Y, down, up, good)
        assert g.device_status() == (0, 0)
        g.set_wait_limit(50_000_000)
        g.run_adapters(X, W, Y, down, up, bad)
        torch.cuda.synchronize()
        g.set_test_stall(True)
        g.run_adapters(X, W, Y, down, up, good)
        code, word = g.device_status()
        assert code == 5 and word >> 24 == 1, (code, hex(word))
        g.set_test_stall(False)
        g.set_wait_limit(2_000_000_000)
        g.run_adapters(X, W, Y, down, up, bad)
        assert g.device_status()[0] == 6
        g.run_adapters(X, W, Y, down, up, good)
        assert g.device_status() == (0, 0)
        assert (Y == 256 + 16 * 256).all()
