"""Workloads of the serving operators around the projections: per-request low-rank
adapters beside a shared projection, rotary positions with several axes, and the
adjustment of logits (penalties for repeated tokens, biases, grammar masks).

``listed()`` names the fixed cases, ``draw(rng)`` gives further ones of the same ranges,
``prepare`` makes a case's inputs on the GPU, and ``run`` computes one pass: with ``own``
false in elementary torch operations in 32 bits, with ``own`` true through this package's
entry points.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"f16": 2, "bf16": 2, "f32": 4}

# The largest products, rotations and logits among the listed cases: what draw() stays within.
MAX_MACS = 8192 * 10240 * 8192
MAX_ROTARY_BYTES = 8192 * 72 * 128 * 2
MAX_LOGITS = 256 * 128256


def listed():
    return [
        # one request generates one token with its adapter: the smallest adapted projection
        {"name": "adapters_token", "op": "adapters", "rows": 1, "n": 8192, "k": 8192, "rank": 16,
         "adapters": 8, "none": 0.0, "prompts": False, "in": "bf16", "out": "bf16"},
        # a decode batch of the fused QKV projection: every row another request, the
        # adapters in no order, one row in eight without one
        {"name": "adapters_decode", "op": "adapters", "rows": 256, "n": 10240, "k": 8192,
         "rank": 16, "adapters": 64, "none": 0.125, "prompts": False, "in": "bf16", "out": "bf16"},
        # a small batch on a narrow projection of odd sizes, fp16 with fp32 results
        {"name": "adapters_odd", "op": "adapters", "rows": 77, "n": 1001, "k": 2008, "rank": 24,
         "adapters": 13, "none": 0.25, "prompts": False, "in": "f16", "out": "f32"},
        # prompts of a few requests, each with its own adapter, of uneven lengths
        {"name": "adapters_prompts", "op": "adapters", "rows": 2050, "n": 4096, "k": 4096,
         "rank": 32, "adapters": 6, "none": 0.0, "prompts": True, "in": "f16", "out": "f16"},
        # a long prefill batch of the fused QKV projection with wide adapters
        {"name": "adapters_prefill", "op": "adapters", "rows": 8192, "n": 10240, "k": 8192,
         "rank": 64, "adapters": 12, "none": 0.1, "prompts": True, "in": "bf16", "out": "bf16"},
        # one token's query and key heads, text position (all axes alike)
        {"name": "rotary_token", "op": "rotary", "tokens": 1, "heads": 72, "dim": 128, "rot": 128,
         "sections": "16,24,24", "mixed": False, "pairs": "half", "inverse": False,
         "positions": 32768, "in": "bf16"},
        # a decode batch, the heads inside the fused QKV rows
        {"name": "rotary_decode", "op": "rotary", "tokens": 256, "heads": 72, "dim": 128,
         "rot": 128, "sections": "16,24,24", "mixed": True, "pairs": "half", "inverse": False,
         "positions": 32768, "in": "bf16"},
        # a training step's gradient through a partial rotation of odd sizes, neighbouring pairs
        {"name": "rotary_grad", "op": "rotary", "tokens": 4099, "heads": 16, "dim": 80, "rot": 72,
         "sections": "10,13,13", "mixed": False, "pairs": "neighbours", "inverse": True,
         "positions": 4096, "in": "f32"},
        # the query and key heads of a long prompt of text and video frames
        {"name": "rotary_video", "op": "rotary", "tokens": 8192, "heads": 72, "dim": 128,
         "rot": 128, "sections": "16,24,24", "mixed": False, "pairs": "half", "inverse": False,
         "positions": 32768, "in": "bf16"},
        # one request's next token, with a grammar
        {"name": "logits_token", "op": "logits", "rows": 1, "vocab": 128256, "history": 2000,
         "biases": 32, "masks": 1.0, "in": "bf16", "out": "f32"},
        # a batch over an odd vocabulary, fp16 logits, half of the rows under a grammar
        {"name": "logits_odd", "op": "logits", "rows": 37, "vocab": 50257, "history": 4096,
         "biases": 200, "masks": 0.5, "in": "f16", "out": "f16"},
        # a full decode batch with long histories
        {"name": "logits_batch", "op": "logits", "rows": 256, "vocab": 128256, "history": 8192,
         "biases": 64, "masks": 0.25, "in": "f32", "out": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapters", "rotary", "logits"])
    if op == "adapters":
        prompts = rng.random() < 0.4
        while True:
            rows = _log(rng, 257, 8192) if prompts else _log(rng, 1, 256)
            n, k = _log(rng, 500, 14336), 8 * _log(rng, 64, 1792)
            if rows * n * k <= MAX_MACS:
                break
        din = rng.choice(["bf16", "f16"])
        return {"op": op, "rows": rows, "n": n, "k": k,
                "rank": rng.choice([8, 16, 16, 24, 32, 64, 128]),
                "adapters": _log(rng, 1, 24 if prompts else 100),
                "none": rng.choice([0.0, 0.1, 0.5]), "prompts": prompts, "in": din,
                "out": rng.choice([din, din, "f32"])}
    if op == "rotary":
        while True:
            tokens, heads = _log(rng, 1, 8192), _log(rng, 1, 72)
            dim = rng.choice([64, 72, 80, 96, 128, 128, 256])
            dt = rng.choice(["bf16", "f16", "f32"])
            if tokens * heads * dim * SIZES[dt] <= MAX_ROTARY_BYTES:
                break
        half = rng.choice([dim // 2, dim // 2, dim // 4])
        axes = rng.choice([1, 2, 3, 4])
        cuts = sorted(rng.randint(0, half) for _ in range(axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [half])]
        return {"op": op, "tokens": tokens, "heads": heads, "dim": dim, "rot": 2 * half,
                "sections": ",".join(map(str, sections)), "mixed": rng.random() < 0.3,
                "pairs": rng.choice(["half", "neighbours"]), "inverse": rng.random() < 0.4,
                "positions": _log(rng, 1000, 60000), "in": dt}
    while True:
        rows, vocab = _log(rng, 1, 256), _log(rng, 8000, 160000)
        if rows * vocab <= MAX_LOGITS:
            break
    din = rng.choice(["bf16", "f16", "f32"])
    return {"op": op, "rows": rows, "vocab": vocab, "history": _log(rng, 16, 8192),
            "biases": rng.choice([0, 1, 50, 300]), "masks": rng.choice([0.0, 0.3, 1.0]),
            "in": din, "out": rng.choice([din, "f32"])}


# ------------------------------------------------------------------------- inputs --
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) % (1 << 62) + 1)
    return g


def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _integers(g, lo, hi, shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)


def _lengths(g, count, longest):
    """Ragged lengths in 0..longest, the first row's the longest."""
    n = _integers(g, 0, longest + 1, (count,)).to(torch.int64)
    n[0] = longest
    return n


def _starts(lengths):
    return torch.cat([lengths.new_zeros(1), lengths.cumsum(0)])


def _adapters(case, g):
    m, n, k, r, count = case["rows"], case["n"], case["k"], case["rank"], case["adapters"]
    dt = DTYPES[case["in"]]
    if case["prompts"]:  # contiguous runs of rows, one request each
        ends = torch.sort(_integers(g, 0, m + 1, (max(count, 2) - 1,))).values
        ids = torch.bucketize(torch.arange(m, device="cuda"), ends.long(), right=True)
        order = torch.randperm(max(count, 2), generator=g, device="cuda") % count
        ids = order[ids].to(torch.int32)
        gone = torch.rand(count, generator=g, device="cuda") < case["none"]
        ids = torch.where(gone[ids.long()], torch.full_like(ids, -1), ids)
    else:
        ids = _integers(g, 0, count, (m,))
        gone = torch.rand(m, generator=g, device="cuda") < case["none"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return {"x": _normal(g, (m, k), 1.0, dt), "w": _normal(g, (n, k), k ** -0.5, dt),
            "down": _normal(g, (count, r, k), k ** -0.5, dt),
            "up": _normal(g, (count, n, r), 0.02, dt),
            "scale": torch.rand(count, generator=g, device="cuda") + 0.5,
            "ids": ids}


def _pair_axes(case):
    """The axis whose position turns each pair: sections in a row, or dealt out in turn."""
    left = [int(s) for s in case["sections"].split(",")]
    if not case["mixed"]:
        return [a for a, s in enumerate(left) for _ in range(s)]
    axes = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                axes.append(a)
    return axes


def _rotary(case, g):
    t, h, d, half = case["tokens"], case["heads"], case["dim"], case["rot"] // 2
    axes = len(case["sections"].split(","))
    # rows as the projection leaves them: the rotated heads first, then the values' heads
    wide = _normal(g, (t, h + max(1, h // 9), d), 1.0, DTYPES[case["in"]])
    freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    angle = torch.arange(case["positions"], device="cuda", dtype=torch.float64)[:, None] * freq
    # a prompt's positions: they advance along every axis by steps of its own
    start = _integers(g, 0, max(1, case["positions"] - t), (axes, 1)).long()
    step = _integers(g, 0, 2, (axes, t)).long().cumsum(1)
    return {"x": wide[:, :h], "cos": angle.cos().float(), "sin": angle.sin().float(),
            "positions": ((start + step) % case["positions"]).to(torch.int32).contiguous(),
            "axes": _pair_axes(case)}


def _logits(case, g):
    b, v = case["rows"], case["vocab"]
    lens = _lengths(g, b, case["history"])
    total = int(lens.sum())
    # frequent tokens repeat often, as in text
    tokens = (torch.rand(total, generator=g, device="cuda") ** 4 * v).to(torch.int32).clamp_(max=v - 1)
    s = {"logits": _normal(g, (b, v), 3.0, DTYPES[case["in"]]), "tokens": tokens,
         "token_start": _starts(lens),
         "prompt_len": (lens.float() * torch.rand(b, generator=g, device="cuda")).to(torch.int32),
         "repetition": 1.0 + 0.5 * torch.rand(b, generator=g, device="cuda"),
         "frequency": 0.5 * torch.rand(b, generator=g, device="cuda"),
         "presence": 0.5 * torch.rand(b, generator=g, device="cuda")}
    if case["biases"]:
        blen = _lengths(g, b, case["biases"])
        start = _starts(blen)
        row = torch.repeat_interleave(torch.arange(b, device="cuda"), blen)
        tok = _integers(g, 0, v, (int(blen.sum()),)).long()
        key = torch.sort(row * v + tok).values  # a row's biases in the order of their tokens
        s["bias_tokens"] = (key % v).to(torch.int32)
        s["bias_values"] = 4.0 * torch.randn(key.numel(), generator=g, device="cuda")
        s["bias_start"] = start
    if case["masks"] > 0:
        words = (v + 31) // 32
        count = max(1, b // 2)  # grammars are shared by requests; the last lets nothing pass
        bits = _integers(g, -2 ** 31, 2 ** 31 - 1, (count, words))
        bits &= _integers(g, -2 ** 31, 2 ** 31 - 1, (count, words))
        if count > 1:
            bits[-1] = 0
        which = _integers(g, 0, count, (b,))
        free = torch.rand(b, generator=g, device="cuda") >= case["masks"]
        s["mask"] = bits
        s["mask_row"] = torch.where(free, torch.full_like(which, -1), which)
    return s


_INPUTS = {"adapters": _adapters, "rotary": _rotary, "logits": _logits}


def prepare(case, seed):
    s = _INPUTS[case["op"]](case, _generator(seed))
    s["case"] = case
    # the program's own output buffers
    if case["op"] == "adapters":
        s["y"] = torch.empty(case["rows"], case["n"], dtype=DTYPES[case["out"]], device="cuda")
    elif case["op"] == "rotary":
        s["y"] = torch.empty(case["tokens"], case["heads"], case["dim"],
                             dtype=DTYPES[case["in"]], device="cuda")
    else:
        s["y"] = torch.empty(case["rows"], case["vocab"], dtype=DTYPES[case["out"]], device="cuda")
    if own:
        from dense_gemm_blackwell_02_gb300 import Gemm
        s["gemm"] = Gemm()
    return s


# ---------------------------------------------------------------------- plain forms --
def _run_adapters(s):
    x = s["x"].float()
    y = x @ s["w"].float().T
    # each row's own adapter, one adapter after the other
    for a in range(s["down"].shape[0]):
        mine = (s["ids"] == a).float()[:, None]
        u = (x * mine) @ s["down"][a].float().T
        y += (u @ s["up"][a].float().T) * s["scale"][a]
    return y.to(s["y"].dtype)


def _run_rotary(s):
    case, x = s["case"], s["x"].float()
    half = case["rot"] // 2
    pos = s["positions"].long()
    axis = torch.tensor(s["axes"], device="cuda")
    row = pos[axis].T                                       # tokens x pairs
    c = torch.gather(s["cos"], 0, row)[:, None]
    sn = torch.gather(s["sin"], 0, row)[:, None]
    if case["inverse"]:
        sn = -sn
    y = x.clone()
    if case["pairs"] == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half] = a * c - b * sn
        y[..., half:2 * half] = b * c + a * sn
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2] = a * c - b * sn
        y[..., 1:2 * half:2] = b * c + a * sn
    return y.to(s["y"].dtype)


def _rows_of(start, total):
    """The row of each entry of a ragged list."""
    at = torch.arange(total, device="cuda")
    return torch.searchsorted(start, at, right=True) - 1, at


def _run_logits(s):
    z = s["logits"].float()
    b, v = z.shape
    row, at = _rows_of(s["token_start"], s["tokens"].numel())
    key = row * v + s["tokens"].long()
    said = (at - s["token_start"][row] >= s["prompt_len"][row]).float()
    count = torch.zeros(b * v, device="cuda").scatter_add_(0, key, said).view(b, v)
    seen = torch.zeros(b * v, device="cuda").scatter_add_(0, key, torch.ones_like(said)).view(b, v)
    rep = s["repetition"][:, None]
    z = torch.where(seen > 0, torch.where(z > 0, z / rep, z * rep), z)
    z = z - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0).float()
    if "bias_tokens" in s:
        row, _ = _rows_of(s["bias_start"], s["bias_tokens"].numel())
        add = torch.zeros(b * v, device="cuda")
        add.scatter_add_(0, row * v + s["bias_tokens"].long(), s["bias_values"])
        z = z + add.view(b, v)
    if "mask" in s:
        words = s["mask"][s["mask_row"].clamp(min=0).long()]
        col = torch.arange(v, device="cuda")
        allowed = (words[:, col // 32] >> (col % 32).to(torch.int32)) & 1
        banned = (allowed == 0) & (s["mask_row"] >= 0)[:, None]
        z = torch.where(banned, torch.full_like(z, -math.inf), z)
    return z.to(s["y"].dtype)


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"adapters": _run_adapters, "rotary": _run_rotary, "logits": _run_logits}[op](s)
    g = s["gemm"]
    if op == "adapters":
        return g.run_adapters(s["x"], s["w"], s["y"], s["down"], s["up"], s["ids"], scale=s["scale"])
    if op == "rotary":
        return g.rotary(s["x"], s["y"], s["cos"], s["sin"], s["positions"], pair_axis=s["axes"],
                        neighbours=s["case"]["pairs"] == "neighbours", inverse=s["case"]["inverse"])
    names = ("tokens", "token_start", "prompt_len", "repetition", "frequency", "presence",
             "bias_tokens", "bias_values", "bias_start", "mask", "mask_row")
    return g.adjust_logits(s["logits"], s["y"], **{k: s[k] for k in names if k in s})


# ------------------------------------------------------------------------ 64 bits --
def exact(case, seed):
    s = _INPUTS[case["op"]](case, _generator(seed))
    return {"adapters": _exact_adapters, "rotary": _exact_rotary,
            "logits": _exact_logits}[case["op"]](case, s)


def _exact_adapters(case, s):
    x = s["x"].double()
    out = torch.empty(case["rows"], case["n"], dtype=torch.float64, device="cuda")
    for j in range(0, case["n"], 2048):  # columns in pieces, to hold little in 64 bits
        out[:, j:j + 2048] = torch.mm(x, s["w"][j:j + 2048].double().t())
    for a in sorted(set(s["ids"].tolist()) - {-1}):
        rows = torch.nonzero(s["ids"] == a).flatten()
        low = torch.mm(x[rows], s["down"][a].double().t())
        out[rows] += s["scale"][a].double() * torch.mm(low, s["up"][a].double().t())
    return out


def _exact_rotary(case, s):
    # (a + ib) times (cos + i sin), or its conjugate for the gradient
    x = s["x"].double()
    half = case["rot"] // 2
    turn = torch.empty(case["tokens"], half, dtype=torch.complex128, device="cuda")
    for i, a in enumerate(s["axes"]):
        at = s["positions"][a].long()
        turn[:, i] = torch.complex(s["cos"][at, i].double(), s["sin"][at, i].double())
    if case["inverse"]:
        turn = turn.conj()
    if case["pairs"] == "half":
        z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous())
        z = z * turn[:, None, :]
        return torch.cat([z.real, z.imag, x[..., 2 * half:]], dim=-1)
    z = torch.view_as_complex(x[..., :2 * half].reshape(*x.shape[:2], half, 2).contiguous())
    z = torch.view_as_real(z * turn[:, None, :]).flatten(-2)
    return torch.cat([z, x[..., 2 * half:]], dim=-1)


def _exact_logits(case, s):
    b, v = case["rows"], case["vocab"]
    out = s["logits"].double()
    ts = s["token_start"].tolist()
    bs = s["bias_start"].tolist() if "bias_start" in s else None
    pl = s["prompt_len"].tolist()
    which = s["mask_row"].tolist() if "mask" in s else [-1] * b
    for i in range(b):
        z = out[i]
        history = s["tokens"][ts[i]:ts[i + 1]].long()
        rep = s["repetition"][i].double()
        before = torch.unique(history)
        z[before] = torch.where(z[before] > 0, z[before] / rep, z[before] * rep)
        said, times = torch.unique(history[pl[i]:], return_counts=True)
        z[said] -= s["frequency"][i].double() * times.double() + s["presence"][i].double()
        if bs is not None:
            t = s["bias_tokens"][bs[i]:bs[i + 1]].long()
            z.index_put_((t,), s["bias_values"][bs[i]:bs[i + 1]].double(), accumulate=True)
        if which[i] >= 0:
            bits = s["mask"][which[i]][:, None] >> torch.arange(32, device="cuda", dtype=torch.int32)
            z[(bits & 1).flatten()[:v] == 0] = -math.inf
    return out


# --------------------------------------------------------------------------- work --
def work(case):
    op = case["op"]
    if op == "adapters":
        m, n, k, r = case["rows"], case["n"], case["k"], case["rank"]
        si, so = SIZES[case["in"]], SIZES[case["out"]]
        used = min(case["adapters"], m)  # adapters no row asks for need not be read
        return {"bytes": si * (m * k + n * k + used * r * (n + k)) + so * m * n + 4 * (m + used),
                "flops": 2 * m * n * k + 2 * m * r * (n + k)}
    if op == "rotary":
        t, half = case["tokens"], case["rot"] // 2
        axes = len(case["sections"].split(","))
        data = t * case["heads"] * case["dim"] * SIZES[case["in"]]
        table = 8 * half * min(t, case["positions"])
        return {"bytes": 2 * data + table + 4 * axes * t, "flops": 6 * t * case["heads"] * half}
    b, v = case["rows"], case["vocab"]
    n = b * v
    lists = 4 * b * (case["history"] // 2) + 8 * b * (case["biases"] // 2)
    masks = max(1, b // 2) * ((v + 31) // 32) * 4 if case["masks"] > 0 else 0
    return {"bytes": n * (SIZES[case["in"]] + SIZES[case["out"]]) + lists + masks, "flops": 6 * n}
