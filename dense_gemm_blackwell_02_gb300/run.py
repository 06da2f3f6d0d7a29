"""Run one GEMM shape, one grouped MoE workload or the projections of a decoding step on
the GPU through the C ABI: a driver for profilers and sweeps.

    python -m dense_gemm_blackwell_02_gb300.run M N K [--in f16|bf16|e4m3|e5m2]
                                                [--out f16|bf16|f32] [--reps R]
                                                [--config JSON] [--blockwise BM]
    python -m dense_gemm_blackwell_02_gb300.run --moe NAME [--experts E] [--reps R]
    python -m dense_gemm_blackwell_02_gb300.run --serve B [--vocab V] [--adapters L] [--rank R]
                                                [--reps R]

Operands are drawn on the device (uniform [-1, 1], fixed seed), then `gemm_run` (or,
with --moe, `gemm_run_grouped` over the workload's experts, the first E of them with
--experts; with --blockwise BM and FP8 inputs, `gemm_run_blockwise` with scales in
[2^-3, 2^3] per BM rows of A and 128 of K, and per 128 x 128 of B) is called R times on
one stream.  Prints the kernel configuration the
library chose and the device status word; exits non-zero if a launch or the status
reports an error.

--serve B is what a decoding step of B requests asks of the library, attention left out: the
fused QKV projection with each request's low-rank adapter (`gemm_run_adapters`), rotary
positions with three axes on the query and key heads in place (`gemm_rotary`), the output
head's product (`gemm_run`), and penalties, biases and grammar masks on its logits, in place
(`gemm_adjust_logits`), of which the largest are the next tokens.
"""
from __future__ import annotations

import argparse
import json
import sys

import torch

from .binding import Gemm

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _moe_problems(name: str, experts: int, dev, gen):
    import seeded_inputs as si
    wl = si.MOE_WORKLOADS[name]
    counts = si.moe_counts(wl.experts, wl.rows, wl.seed)
    if experts:
        counts = counts[:experts]
    tin, tout = si.TORCH_DTYPE[wl.dtype_in], si.TORCH_DTYPE[wl.dtype_out]
    return [((torch.rand(m, wl.K, generator=gen, device=dev) * 2 - 1).to(tin),
             (torch.rand(wl.N, wl.K, generator=gen, device=dev) * 2 - 1).to(tin),
             torch.empty(m, wl.N, dtype=tout, device=dev)) for m in counts]


# The projections of serve(): hidden size, query, key and value heads of 128 (10240 columns).
HIDDEN, HEADS_Q, HEADS_KV, HEAD_DIM = 8192, 64, 8, 128


def serve_state(rows: int, vocab: int, adapters: int, rank: int, dev, gen) -> dict:
    """The model and the requests of serve()."""
    from .binding import pair_axes

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * std).bfloat16()

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device=dev, dtype=torch.int32)
    heads, half = HEADS_Q + HEADS_KV, HEAD_DIM // 2
    cols = (heads + HEADS_KV) * HEAD_DIM
    # the model: projections, a pool of adapters, the rotary tables
    s = {"w_qkv": normal(cols, HIDDEN, std=HIDDEN ** -0.5),
         "w_out": normal(vocab, HIDDEN, std=HIDDEN ** -0.5),
         "down": normal(adapters, rank, HIDDEN, std=HIDDEN ** -0.5),
         "up": normal(adapters, cols, rank, std=0.02)}
    angle = (torch.arange(4096, device=dev, dtype=torch.float64)[:, None]
             * 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half))
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    s["axes"] = pair_axes([half - 2 * (3 * half // 8), 3 * half // 8, 3 * half // 8])
    # the requests: their adapters (one in nine without), positions, histories, grammars
    s["ids"], s["positions"] = ints(-1, adapters, rows), ints(0, 4096, 3, rows)
    length = ints(1, 1025, rows).long()
    start = torch.cat([length.new_zeros(1), length.cumsum(0)])
    tokens = ints(0, vocab, int(start[-1]))
    ones = torch.ones(rows, device=dev)
    mask = ints(-2 ** 31, 2 ** 31 - 1, 2, (vocab + 31) // 32)
    mask_row = ints(-1, 2, rows)
    s["adjust"] = dict(tokens=tokens, token_start=start, prompt_len=(length // 2).int(),
                       repetition=1.1 * ones, frequency=0.1 * ones, presence=0.1 * ones, mask=mask,
                       mask_row=mask_row)
    s["x"], s["hidden"] = normal(rows, HIDDEN), normal(rows, HIDDEN)
    s["qkv"] = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
    s["logits"] = torch.empty(rows, vocab, device=dev)
    return s


def serve_step(g: Gemm, s: dict):
    """One decoding step: fills s["qkv"] and s["logits"], returns the tokens."""
    g.run_adapters(s["x"], s["w_qkv"], s["qkv"], s["down"], s["up"], s["ids"])
    heads = HEADS_Q + HEADS_KV
    qk = s["qkv"][:, :heads * HEAD_DIM].unflatten(1, (heads, HEAD_DIM))
    g.rotary(qk, qk, s["cos"], s["sin"], s["positions"], pair_axis=s["axes"])
    # (attention over qkv and the layers after it would give `hidden`)
    g.run(s["hidden"], s["w_out"], s["logits"])
    g.adjust_logits(s["logits"], s["logits"], **s["adjust"])
    return s["logits"].argmax(dim=1)


def serve(g: Gemm, rows: int, vocab: int, adapters: int, rank: int, reps: int, dev, gen) -> dict:
    """`reps` decoding steps of `rows` requests; returns the last step's tokens."""
    s = serve_state(rows, vocab, adapters, rank, dev, gen)
    for _ in range(reps):
        chosen = serve_step(g, s)
    return {"serve": rows, "vocab": vocab, "adapters": adapters, "rank": rank,
            "finite": bool(torch.isfinite(s["qkv"]).all()), "tokens": chosen[:8].tolist()}


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("M", type=int, nargs="?")
    ap.add_argument("N", type=int, nargs="?")
    ap.add_argument("K", type=int, nargs="?")
    ap.add_argument("--in", dest="din", default="f16", choices=["f16", "bf16", "e4m3", "e5m2"])
    ap.add_argument("--out", dest="dout", default="f16", choices=["f16", "bf16", "f32"])
    ap.add_argument("--reps", type=int, default=5)
    ap.add_argument("--config", default=None, help="JSON gemm_config_t fields")
    ap.add_argument("--moe", default=None, help="a grouped MoE workload of seeded_inputs")
    ap.add_argument("--experts", type=int, default=0, help="with --moe: only the first E experts")
    ap.add_argument("--blockwise", type=int, default=0,
                    help="FP8 inputs: block scales, one per BM rows of A and 128 of K")
    ap.add_argument("--serve", type=int, default=0, metavar="B",
                    help="the projections of a decoding step of B requests")
    ap.add_argument("--vocab", type=int, default=128256, help="with --serve")
    ap.add_argument("--adapters", type=int, default=64, help="with --serve: adapters in the pool")
    ap.add_argument("--rank", type=int, default=16, help="with --serve: the adapters' rank")
    a = ap.parse_args(argv)
    if a.moe is None and not a.serve and None in (a.M, a.N, a.K):
        ap.error("M N K are required without --moe or --serve")
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev)
    gen.manual_seed(0)
    with Gemm() as g:
        if a.config:
            g.set_config(**json.loads(a.config))
        if a.serve:
            shape = serve(g, a.serve, a.vocab, a.adapters, a.rank, a.reps, dev, gen)
        elif a.moe:
            probs = _moe_problems(a.moe, a.experts, dev, gen)
            for _ in range(a.reps):
                g.run_grouped(probs)
            shape = {"moe": a.moe, "experts": len(probs), "rows": sum(p[0].shape[0] for p in probs)}
        else:
            A = (torch.rand(a.M, a.K, generator=gen, device=dev) * 2 - 1).to(DTYPES[a.din])
            B = (torch.rand(a.N, a.K, generator=gen, device=dev) * 2 - 1).to(DTYPES[a.din])
            C = torch.empty(a.M, a.N, dtype=DTYPES[a.dout], device=dev)
            if a.blockwise:
                nkb = -(-a.K // 128)
                sfa = torch.exp2(torch.rand(nkb, -(-a.M // a.blockwise), generator=gen, device=dev) * 6 - 3)
                sfb = torch.exp2(torch.rand(nkb, -(-a.N // 128), generator=gen, device=dev) * 6 - 3)
            for _ in range(a.reps):
                if a.blockwise:
                    g.run_blockwise(A, B, C, sfa, sfb, a.blockwise)
                else:
                    g.run(A, B, C)
            shape = {"M": a.M, "N": a.N, "K": a.K, "in": a.din, "out": a.dout,
                     "blockwise": a.blockwise}
        torch.cuda.synchronize()
        code, word = g.device_status()
        print(json.dumps({**shape, "kernel": g.last_config(), "status": code, "status_word": word}))
    return 1 if code else 0


if __name__ == "__main__":
    sys.exit(main())
