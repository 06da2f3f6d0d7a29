"""The projections of a decoding step run together, as the one-shape driver offers them."""
import json

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 9, 600])
def test_serve_step(capsys, rows):
    from dense_gemm_blackwell_02_gb300 import run
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    assert run.main(["--serve", str(rows), "--vocab", "1500", "--adapters", "5", "--rank", "8",
                     "--reps", "2"]) == 0
    line = json.loads(capsys.readouterr().out.strip().splitlines()[-1])
    assert line["status"] == 0 and line["finite"]
    assert all(0 <= t < 1500 for t in line["tokens"]) and len(line["tokens"]) == min(rows, 8)
