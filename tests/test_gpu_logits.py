"""Adjusted logits (gemm_adjust_logits) against the definition in 64 bits.

Tolerance.  In binary32 the repetition penalty rounds once, the frequency and presence
penalties twice and the biases once per entry; each is within 2^-24 of the magnitudes added
so far: m = |z| max(rep, 1 / rep) + freq c + pres + sum |w|.  So ulp / 2 + 8 * 2^-24 * m,
with at most four biases for one token here.  Untouched values convert exactly (same type) or
round once; -infinity and NaN are compared as such.
"""
import math

import numpy as np
import pytest
import torch

from tests import parity

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"f16": 0, "bf16": 1, "f32": 2}


@pytest.fixture(scope="module")
def g():
    from dense_gemm_blackwell_02_gb300.binding import Gemm
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    h = Gemm()
    yield h
    h.close()


def _inputs(B, V, H, nb, masks, dt, seed):
    gen = torch.Generator().manual_seed(seed)

    def ints(lo, hi, shape):
        return torch.randint(lo, hi, shape, generator=gen)
    t = {"logits": (torch.randn(B, V, generator=gen) * 4).to(DT[dt])}
    if H:
        lens = ints(0, H + 1, (B,))
        lens[-1] = H
        if B > 2:
            lens[1] = 0
        tok = (torch.rand(int(lens.sum()), generator=gen) ** 3 * V).int().clamp(max=V - 1)
        tok[::17] = -1                                # padding
        if len(tok) > 5:
            tok[5] = V
        t.update(tokens=tok, token_start=torch.cat([torch.zeros(1), lens.cumsum(0)]).long(),
                 prompt_len=(lens * torch.rand(B, generator=gen)).int(),
                 repetition=0.7 + torch.rand(B, generator=gen),
                 frequency=torch.rand(B, generator=gen) - 0.3,
                 presence=torch.rand(B, generator=gen) - 0.3)
    if nb:
        rows = []
        for _ in range(B):
            n = int(ints(0, nb + 1, (1,)))
            own = ints(0, V, (n,))
            own[n // 2:n // 2 + 2] = own[n // 2:n // 2 + 1]   # one token twice
            rows.append(torch.sort(own).values)
        lens = torch.tensor([len(r) for r in rows])
        t.update(bias_tokens=torch.cat(rows).int(),
                 bias_values=torch.randn(int(lens.sum()), generator=gen) * 5,
                 bias_start=torch.cat([torch.zeros(1), lens.cumsum(0)]).long())
    if masks:
        words = (V + 31) // 32 + 1                    # a row of masks may be longer
        m = ints(-2 ** 31, 2 ** 31, (masks, words)).int()
        m[-1] = 0                                     # nothing may follow
        t.update(mask=m, mask_row=ints(-1, masks, (B,)).int())
    return t


def _expect(t):
    z = t["logits"].double().numpy().copy()
    B, V = z.shape
    m = np.abs(z)
    for i in range(B):
        if "tokens" in t:
            s0, s1 = t["token_start"][i:i + 2].tolist()
            h = t["tokens"][s0:s1].numpy()
            pl = int(t["prompt_len"][i]) if "prompt_len" in t else 0
            seen = np.unique(h[(h >= 0) & (h < V)])
            rep = float(t["repetition"][i]) if "repetition" in t else 1.0
            z[i, seen] = np.where(z[i, seen] > 0, z[i, seen] / rep, z[i, seen] * rep)
            m[i, seen] *= max(rep, 1 / rep)
            said = h[pl:]
            v, c = np.unique(said[(said >= 0) & (said < V)], return_counts=True)
            f = float(t["frequency"][i]) if "frequency" in t else 0.0
            q = float(t["presence"][i]) if "presence" in t else 0.0
            z[i, v] -= f * c + q
            m[i, v] += abs(f) * c + abs(q)
        if "bias_tokens" in t:
            s0, s1 = t["bias_start"][i:i + 2].tolist()
            v = t["bias_tokens"][s0:s1].numpy()
            w = t["bias_values"][s0:s1].double().numpy()
            np.add.at(z[i], v, w)
            np.add.at(m[i], v, np.abs(w))
        if "mask" in t:
            r = int(t["mask_row"][i]) if "mask_row" in t else i
            if 0 <= r < len(t["mask"]):
                bits = np.unpackbits(t["mask"][r].numpy().view(np.uint8), bitorder="little")[:V]
                z[i, bits == 0] = -math.inf
    return z, m


def _check(out, t, code):
    z, m = _expect(t)
    got = out.double().cpu().numpy()
    same = (got == z) | (np.isnan(got) & np.isnan(z))
    with np.errstate(invalid="ignore"):
        finite = np.isfinite(z)
        zf = np.where(finite, z, 0.0)
        bound = parity.ulp_of(zf, code) / 2 + 8 * 2.0 ** -24 * np.where(finite, m, 0.0)
        ok = same | (finite & (np.abs(got - zf) <= bound * (1 + 1e-9)))
    bad = np.argwhere(~ok)
    assert bad.size == 0, f"{len(bad)} off, first {bad[0]}: {got[tuple(bad[0])]} for {z[tuple(bad[0])]}"


def _run(g, t, out_dt, logits=None, out=None):
    d = {k: v.cuda() for k, v in t.items()}
    x = d.pop("logits") if logits is None else logits
    d.pop("logits", None)
    if out is None:
        out = torch.full(x.shape, 77.0, dtype=out_dt, device="cuda")
    g.adjust_logits(x, out, **d)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("din,dout", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16"),
                                      ("bf16", "bf16"), ("f32", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("B,V,H,nb,masks", [
    (1, 1, 3, 1, 1),
    (1, 131, 40, 5, 2),
    (3, 32, 10, 3, 3),
    (5, 1000, 500, 20, 2),
    (2, 50257, 3000, 300, 2),
    (17, 4099, 100, 0, 0),
    (4, 8191, 0, 10, 0),
    (4, 8193, 0, 0, 3),
    (3, 33000, 0, 0, 0),
    (400, 515, 60, 4, 7),
    (1, 140001, 6000, 50, 1),
])
def test_logits_against_the_definition(g, din, dout, B, V, H, nb, masks):
    t = _inputs(B, V, H, nb, masks, din, seed=B + V)
    _check(_run(g, t, DT[dout]), t, CODE[dout])
    assert g.device_status()[0] == 0


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V,stride,offset", [(1000, 1008, 0), (1001, 1003, 0), (4097, 4100, 3),
                                             (33000, 33001, 5), (999, 1024, 8)])
def test_rows_of_any_stride_and_alignment_and_in_place(g, dt, V, stride, offset):
    B = 6
    t = _inputs(B, V, 200, 8, 3, dt, seed=V)
    wide = torch.full((B, stride + offset), 5.0, dtype=DT[dt], device="cuda")
    x = wide[:, offset:offset + V]
    x.copy_(t["logits"])
    out_wide = torch.full((B, V + 7), 9.0, dtype=DT[dt], device="cuda")
    out = out_wide[:, 2:2 + V]
    _run(g, t, None, logits=x, out=out)
    _check(out, t, CODE[dt])
    assert torch.equal(x.cpu(), t["logits"])
    assert (out_wide[:, :2] == 9).all() and (out_wide[:, 2 + V:] == 9).all()
    _run(g, t, None, logits=x, out=x)
    assert torch.equal(x, out)
    assert (wide[:, :offset] == 5).all() and (wide[:, offset + V:] == 5).all()


def test_parts_left_out(g):
    t = _inputs(5, 2000, 300, 6, 5, "f32", seed=2)
    for drop in (["prompt_len"], ["repetition"], ["frequency"], ["presence"],
                 ["mask_row"], ["repetition", "frequency", "presence", "prompt_len"]):
        u = {k: v for k, v in t.items() if k not in drop}
        _check(_run(g, u, torch.float32), u, 2)


def test_infinities_nan_and_extremes(g):
    t = _inputs(4, 3000, 400, 0, 2, "f32", seed=6)
    x = t["logits"]
    x[0, ::7] = float("nan")
    x[1, ::5] = float("-inf")
    x[2, ::3] = float("inf")
    x[3, ::2] = torch.finfo(torch.float32).min
    t["mask_row"] = torch.tensor([0, -1, 1, 0], dtype=torch.int32)   # mask 1 bans everything
    t["repetition"] = torch.ones(4)
    out = _run(g, t, torch.float32)
    _check(out, t, 2)
    assert (out[2] == -math.inf).all()


def test_one_token_repeated_throughout_a_long_history(g):
    B, V, H = 2, 700, 200000
    t = {"logits": torch.randn(B, V), "tokens": torch.full((B * H,), 699, dtype=torch.int32),
         "token_start": torch.tensor([0, H, 2 * H]), "prompt_len": torch.tensor([0, H], dtype=torch.int32),
         "repetition": torch.tensor([1.5, 1.5]), "frequency": torch.tensor([0.25, 0.25]),
         "presence": torch.tensor([1.0, 1.0])}
    out = _run(g, t, torch.float32)
    _check(out, t, 2)
    assert out[0, 699] < -49000 and out[1, 699] > -10


def test_mask_row_out_of_range_is_reported_and_not_followed(g):
    t = _inputs(5, 900, 0, 0, 3, "f32", seed=1)
    t["mask_row"] = torch.tensor([0, 3, 2 ** 31 - 1, -2 ** 31, 1], dtype=torch.int32)
    out = _run(g, t, torch.float32)
    code, word = g.device_status()
    assert code == 6 and word >> 24 == 2 and (word >> 16) & 0xFF == 3
    _check(out, t, 2)


def test_same_result_every_time(g):
    t = _inputs(64, 20000, 2000, 30, 4, "bf16", seed=3)
    first = _run(g, t, torch.float32)
    for _ in range(3):
        assert torch.equal(first, _run(g, t, torch.float32))


def test_empty_calls_and_refusals(g):
    from dense_gemm_blackwell_02_gb300.binding import GemmError, GemmLogits, lib
    import ctypes
    x = torch.zeros(3, 100, device="cuda")
    out = torch.empty_like(x)
    g.adjust_logits(x[:0], out[:0])
    g.adjust_logits(x[:, :0], out[:, :0])
    g.adjust_logits(x, out)
    assert torch.equal(x, out)
    i32 = dict(dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="token_start"):
        g.adjust_logits(x, out, tokens=torch.zeros(4, **i32), token_start=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(GemmError, match="INVALID_ARG"):
        g.adjust_logits(x, out, tokens=torch.zeros(4, **i32))
    with pytest.raises(ValueError, match="tokens"):
        g.adjust_logits(x, out, tokens=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(GemmError, match="INVALID_ARG"):
        g.adjust_logits(x, out, bias_tokens=torch.zeros(4, **i32))
    with pytest.raises(ValueError, match="bias_values"):
        g.adjust_logits(x, out, bias_tokens=torch.zeros(4, **i32), bias_values=torch.zeros(3, device="cuda"),
                        bias_start=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(GemmError, match="INVALID_ARG"):
        g.adjust_logits(x, out, mask=torch.zeros(3, 3, **i32))       # 100 tokens need 4 words
    with pytest.raises(GemmError, match="INVALID_ARG"):
        g.adjust_logits(x, out, mask=torch.zeros(2, 4, **i32))       # a mask for every row
    with pytest.raises(ValueError, match="repetition"):
        g.adjust_logits(x, out, repetition=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        g.adjust_logits(x[:, ::2], out[:, :50])
    with pytest.raises(ValueError, match="overlap"):
        g.adjust_logits(x[:1].expand(3, 100), out)
    # in place with another type: through the C call (torch has no such tensors)
    a = GemmLogits()
    assert lib().gemm_adjust_logits(g.handle, x.data_ptr(), x.data_ptr(), 3, 100, 100, 100, 2, 1,
                                    ctypes.byref(a), None) == 1
    assert lib().gemm_adjust_logits(g.handle, x.data_ptr(), out.data_ptr(), 3, 100, 99, 100, 2, 2,
                                    ctypes.byref(a), None) == 1
    assert lib().gemm_adjust_logits(g.handle, x.data_ptr(), out.data_ptr(), 3, 100, 100, 100, 3, 2,
                                    ctypes.byref(a), None) == 2
    assert g.device_status()[0] == 0


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("B,V,H,nb", [(4, 1000, 0, 50), (3, 30000, 64, 700), (5, 5000, 40000, 9)])
def test_biases_in_any_order(g, dt, B, V, H, nb):
    # rows in the order of their tokens beside rows in none, padding at the end of one, a fall
    # at the last entry alone
    t = _inputs(B, V, H, nb, 0, dt, seed=V + nb)
    gen = torch.Generator().manual_seed(nb)
    for i in range(B):
        s0, s1 = t["bias_start"][i:i + 2].tolist()
        if i % 3 == 0:
            p = torch.randperm(s1 - s0, generator=gen)
            t["bias_tokens"][s0:s1] = t["bias_tokens"][s0:s1][p]
            t["bias_values"][s0:s1] = t["bias_values"][s0:s1][p]
        elif i % 3 == 1 and s1 - s0 > 4:
            t["bias_tokens"][s1 - 2:s1] = -1
        elif s1 - s0 > 4:
            t["bias_tokens"][s1 - 1] = t["bias_tokens"][s0]
    out = torch.full(t["logits"].shape, 7.0, dtype=DT[dt], device="cuda")
    d = {k: v.cuda() for k, v in t.items()}
    g.adjust_logits(d.pop("logits"), out, **d)
    # (the formula's index of the padding would be the last token's: a bias of 0 for the first)
    padding = t["bias_tokens"] < 0
    t["bias_values"][padding], t["bias_tokens"][padding] = 0.0, 0
    _check(out, t, CODE[dt])
    assert g.device_status()[0] == 0


def test_an_empty_mask_is_refused_where_a_row_could_ask_for_it(g):
    x = torch.zeros(2, 70, device="cuda")
    rows = torch.zeros(2, dtype=torch.int32, device="cuda")
    for shape in ((0, 3), (2, 0)):
        mask = torch.zeros(shape, dtype=torch.int32, device="cuda")
        with pytest.raises(ValueError, match="mask"):
            g.adjust_logits(x, torch.empty_like(x), mask=mask, mask_row=rows)
        with pytest.raises(ValueError, match="mask"):
            g.adjust_logits(x, torch.empty_like(x), mask=mask)
    none = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    g.adjust_logits(x[:0], torch.empty_like(x[:0]), mask=none, mask_row=rows[:0])
