"""The values of a decoding step (run.serve_step): its operators queued one behind the other,
several steps of it, against the formulas applied to what each stage alone gives."""
import numpy as np
import pytest
import torch

from tests import parity
from tests.test_gpu_logits import _check as check_logits
from tests.test_gpu_rotary import _check as check_rotary
from tests.test_gpu_rotary import _expect as expect_rotary

pytestmark = pytest.mark.gpu

BF16, F32 = 1, 2


def _numpy(t):
    return t.double().cpu().numpy()


def _near(got, want, magnitude, K, code):
    """A product of length K in binary32 (parity.tau_of over the terms' root of squares), and a
    rounding."""
    got, want = _numpy(got), _numpy(want)
    bound = parity.ulp_of(want, code) / 2 + parity.tau_of(_numpy(magnitude), K)
    bad = np.argwhere(~(np.abs(got - want) <= bound * (1 + 1e-9)))
    assert bad.size == 0, f"{len(bad)} off, first {bad[0]}: {got[tuple(bad[0])]} for {want[tuple(bad[0])]}"


# 600 rows of 5 adapters: adapters in the product's tiles; the others: the kernels for few rows
@pytest.mark.parametrize("rows,vocab", [(1, 1500), (9, 1500), (64, 33001), (600, 1500)])
def test_every_stage_of_a_step_gives_its_formulas_values(rows, vocab):
    from dense_gemm_blackwell_02_gb300 import run
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    s = run.serve_state(rows, vocab, 5, 8, torch.device("cuda", 0), gen)
    with Gemm() as g:
        s["qkv"].fill_(float("nan"))
        s["logits"].fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(4):                       # nothing waits in between
            tokens = run.serve_step(g, s)
        torch.cuda.synchronize()
        assert g.device_status() == (0, 0)
        # each stage on its own
        alone = torch.empty_like(s["qkv"])
        g.run_adapters(s["x"], s["w_qkv"], alone, s["down"], s["up"], s["ids"])
        torch.cuda.synchronize()
        head = torch.empty_like(s["logits"])
        g.run(s["hidden"], s["w_out"], head)
        torch.cuda.synchronize()
        assert g.device_status() == (0, 0)

    X, W = s["x"].double(), s["w_qkv"].double()
    want, squares = X @ W.T, (X ** 2) @ (W ** 2).T
    extra = torch.zeros_like(want)
    for a in range(5):
        r = s["ids"] == a
        u = X[r] @ s["down"][a].double().T
        want[r] += u @ s["up"][a].double().T
        # u's own error (a product of length K) through |Up|, and 2^-16 of its terms
        e = torch.from_numpy(parity.tau_of(_numpy(((X[r] ** 2) @ (s["down"][a].double() ** 2).T).sqrt()),
                                           run.HIDDEN)).cuda() + 2.0 ** -16 * u.abs()
        extra[r] = e @ s["up"][a].double().abs().T
    got, exact = _numpy(alone), _numpy(want)
    bound = parity.ulp_of(exact, BF16) / 2 + parity.tau_of(_numpy(squares.sqrt()), run.HIDDEN) + _numpy(extra)
    assert (np.abs(got - exact) <= bound * (1 + 1e-9)).all()

    heads = run.HEADS_Q + run.HEADS_KV
    turned = heads * run.HEAD_DIM
    assert torch.equal(s["qkv"][:, turned:], alone[:, turned:])
    y, mag = expect_rotary(alone[:, :turned].cpu().unflatten(1, (heads, run.HEAD_DIM)), s["cos"].cpu(),
                           s["sin"].cpu(), s["positions"].cpu(), s["axes"], False, False)
    check_rotary(s["qkv"][:, :turned].unflatten(1, (heads, run.HEAD_DIM)), y, mag, "bf16")

    H, O = s["hidden"].double(), s["w_out"].double()
    _near(head, H @ O.T, ((H ** 2) @ (O ** 2).T).sqrt(), run.HIDDEN, F32)
    t = {k: v.cpu() for k, v in s["adjust"].items()}
    check_logits(s["logits"], dict(t, logits=head.cpu()), F32)
    best = s["logits"].max(dim=1).values
    assert torch.equal(s["logits"].gather(1, tokens[:, None])[:, 0], best)
