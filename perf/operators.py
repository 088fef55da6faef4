"""The steps between the weight products of a decoded block, as measured cases.

Three operators that a transformer block needs around its compressed weights:

* ``norm``: the residual's addition and the root-mean-square norm of every
  token, written as bf16 (the input of the entropy-coded GEMV) or in 8 bits
  with one scale per token (the input of the 4-bit products);
* ``silu``: silu(gate) * up of every token, in the same output types;
* ``w4``: products of a few tokens with 4-bit weights that carry a scale for
  every group of columns, several matrices in one call.

``listed()`` names the cases, ``draw()`` makes more of the same ranges,
``prepare()`` makes one case's inputs, ``run()`` computes it (``own`` false:
plain torch operations in 32 bits; true: this package's kernels), ``exact()``
computes it in 64 bits, ``work()`` says what one pass cannot do without.
"""
import math

import torch

own = False

EPS = 1e-5
F32, BF16 = "f32", "bf16"
INT8, E4M3 = "int8", "e4m3"  # 8-bit activations
INT4, E2M1 = "int4", "e2m1"  # 4-bit weights
TORCH = {F32: torch.float32, BF16: torch.bfloat16, INT8: torch.int8, E4M3: torch.float8_e4m3fn}
BYTES = {F32: 4, BF16: 2, INT8: 1, E4M3: 1}
LARGEST = {INT8: 127.0, E4M3: 448.0}
SMALLEST_AMAX = 2.0 ** -96  # a row's largest magnitude is taken as no less than this
E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # one token's hidden state after a block's output product (fp32 from the GEMV), normed for the
        # next entropy-coded GEMV: the smallest call, latency alone
        dict(name="norm token", op="norm", tokens=1, cols=4096, x=F32, residual=BF16, out=BF16),
        # a decode batch, residual stream kept in fp32, normed for int8 products
        dict(name="norm batch int8", op="norm", tokens=48, cols=8192, x=F32, residual=F32, out=INT8),
        # a long prompt
        dict(name="norm prompt e4m3", op="norm", tokens=8192, cols=8192, x=BF16, residual=BF16, out=E4M3),
        # a norm without a residual (of queries, of a final state) at a width that divides by nothing
        dict(name="norm odd width", op="norm", tokens=1777, cols=5003, x=BF16, residual="", out=BF16),
        # one token between the gate and up products and the down product
        dict(name="silu token int8", op="silu", tokens=1, cols=28672, x=F32, out=INT8),
        # a long prompt between them
        dict(name="silu prompt e4m3", op="silu", tokens=4096, cols=11008, x=BF16, out=E4M3),
        # one token through one square projection: the smallest product
        dict(name="w4 token square", op="w4", tokens=1, rows="4096", cols=4096, w=INT4, group=128, zeros=False, x=BF16, out=F32),
        # one token through gate and up of a large block, activations in int8
        dict(name="w4 token gate+up int8", op="w4", tokens=1, rows="28672,28672", cols=8192, w=INT4, group=128, zeros=False, x=INT8, out=F32),
        # four tokens (a speculative step) through q, k and v, 4-bit floats in small groups
        dict(name="w4 four tokens qkv", op="w4", tokens=4, rows="8192,1024,1024", cols=8192, w=E2M1, group=32, zeros=False, x=BF16, out=BF16),
        # a decode batch through down, 4-bit floats with 8-bit floats
        dict(name="w4 batch down e4m3", op="w4", tokens=16, rows="8192", cols=28672, w=E2M1, group=128, zeros=False, x=E4M3, out=F32),
        # zero points, odd sizes, a ragged last group
        dict(name="w4 odd zeros", op="w4", tokens=7, rows="5001", cols=4133, w=INT4, group=64, zeros=True, x=BF16, out=F32),
        # the largest decode batch through gate and up
        dict(name="w4 large batch gate+up int8", op="w4", tokens=64, rows="28672,28672", cols=8192, w=INT4, group=128, zeros=False, x=INT8, out=F32),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm; mostly multiples of 128 where it is large, at times odd."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v >= 512 and rng.random() < 0.6:
        v = v // 128 * 128
    v = min(max(v, low), high)
    return v - 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["norm", "silu", "w4", "w4"])
    if op != "w4":
        cols = _spread(rng, 64, 28672)
        tokens = min(_spread(rng, 1, 8192), (8192 * 8192 if op == "norm" else 4096 * 11008) // cols)
        case = dict(op=op, tokens=max(1, tokens), cols=cols, x=rng.choice([F32, BF16]))
        if op == "norm":
            case["residual"] = rng.choice(["", F32, BF16])
        case["out"] = rng.choice([BF16, INT8, E4M3])
        return case
    w = rng.choice([INT4, E2M1])
    cols = _spread(rng, 64, 28672)
    n = rng.randint(1, 3)
    most = min(28672, max(16, 2 * 28672 * 8192 // cols // n))
    rows = [_spread(rng, 16, most) for _ in range(n)]
    return dict(op="w4", tokens=_spread(rng, 1, 64), rows=",".join(map(str, rows)), cols=cols, w=w, group=rng.choice([32, 64, 128]),
                zeros=w == INT4 and rng.random() < 0.4, x=rng.choice([BF16, INT8 if w == INT4 else E4M3]), out=rng.choice([F32, BF16]))


def _rows(case):
    return [int(r) for r in case["rows"].split(",")]


def work(case):
    tokens, cols = case["tokens"], case["cols"]
    if case["op"] == "norm":
        moved = BYTES[case["x"]] + (2 * BYTES[case["residual"]] if case["residual"] else 0) + BYTES[case["out"]]
        return {"bytes": tokens * cols * moved + 2 * cols + (4 * tokens if case["out"] in LARGEST else 0), "flops": 5 * tokens * cols}
    if case["op"] == "silu":
        moved = 2 * BYTES[case["x"]] + BYTES[case["out"]]
        return {"bytes": tokens * cols * moved + (4 * tokens if case["out"] in LARGEST else 0), "flops": 6 * tokens * cols}
    rows = sum(_rows(case))
    groups = -(-cols // case["group"])
    weights = rows * (-(-cols // 2) + groups * (3 if case["zeros"] else 2))
    x = tokens * cols * BYTES[case["x"]] + (4 * tokens if case["x"] in LARGEST else 0)
    return {"bytes": weights + x + tokens * rows * BYTES[case["out"]], "flops": 2 * tokens * rows * cols}


# --- inputs -------------------------------------------------------------------


def _hidden(gen, tokens, cols, dtype):
    """Hidden states: normal, a few channels far larger than the rest, one padding token of zeros in a batch."""
    x = torch.randn(tokens, cols, generator=gen, device="cuda")
    x[:, torch.randint(cols, (max(1, cols // 1000),), generator=gen, device="cuda")] *= 20
    if tokens >= 16:
        x[tokens // 2] = 0
    return x.to(dtype)


def _in_8_bits(x, dtype):
    """Codes and one scale per row of x."""
    amax = x.abs().amax(dim=1).clamp_min(SMALLEST_AMAX)
    y = (x * (LARGEST[dtype] / amax)[:, None]).clamp(-LARGEST[dtype], LARGEST[dtype])
    return (y.round() if dtype == INT8 else y).to(TORCH[dtype]), amax / LARGEST[dtype]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    tokens, cols, out = case["tokens"], case["cols"], case["out"]
    s = {"case": case}
    if case["op"] != "w4":
        s["x"] = _hidden(gen, tokens, cols, TORCH[case["x"]])
        if case["op"] == "norm":
            s["weight"] = (1 + 0.2 * torch.randn(cols, generator=gen, device="cuda")).to(torch.bfloat16)
            s["residual"] = s["residual_out"] = None
            if case["residual"]:
                s["residual"] = (4 * _hidden(gen, tokens, cols, torch.float32)).to(TORCH[case["residual"]])
                s["residual_out"] = torch.empty_like(s["residual"])
        else:
            s["up"] = _hidden(gen, tokens, cols, TORCH[case["x"]])
        s["out"] = torch.empty(tokens, cols, dtype=TORCH[out], device="cuda")
        s["scale"] = torch.empty(tokens, device="cuda") if out in LARGEST else None
        return s
    x = _hidden(gen, tokens, cols, torch.float32)
    if case["x"] in LARGEST:
        s["x"], s["x_scale"] = _in_8_bits(x, case["x"])
    else:
        s["x"], s["x_scale"] = x.to(TORCH[case["x"]]), None
    groups = -(-cols // case["group"])
    s["weights"] = []
    for rows in _rows(case):
        # two codes a byte, the lower half first; the codes of a normal weight matrix after scaling
        codes = torch.empty(rows, -(-cols // 2), dtype=torch.uint8, device="cuda")
        for at in range(0, rows, 4096):
            n = min(4096, rows - at)
            q = torch.randn(n, 2 * codes.shape[1], generator=gen, device="cuda") * 2.6
            if case["w"] == INT4:
                q = (q.round_().clamp_(-8, 7).to(torch.int16) + (8 if case["zeros"] else 16)) % 16  # offset binary or two's complement
            else:
                q = torch.bucketize(q.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")).to(torch.int16) + 8 * (q < 0)
            codes[at:at + n] = (q[:, 0::2] + 16 * q[:, 1::2]).to(torch.uint8)
        scales = (0.002 + 0.006 * torch.rand(rows, groups, generator=gen, device="cuda")).to(torch.bfloat16)
        zeros = torch.randint(5, 12, (rows, groups), generator=gen, device="cuda").to(torch.uint8) if case["zeros"] else None
        s["weights"].append((codes, scales, zeros))
    s["ys"] = [torch.empty(tokens, rows, dtype=TORCH[out], device="cuda") for rows in _rows(case)]
    if own:  # the weights in the kernels' layout, made when a model is loaded
        from rans_decode_amd import eq
        dtype = eq.EQ_DTYPE_INT4 if case["w"] == INT4 else eq.EQ_DTYPE_E2M1
        s["block"] = eq.W4Block([eq.W4Tensor(c, k, z, dtype=dtype, group=case["group"], cols=cols) for c, k, z in s["weights"]])
    return s


# --- one pass -----------------------------------------------------------------


def _answer(y, scale, residual=None):
    """The outputs: int8 codes as the values they stand for, 8-bit floats as themselves, beside their scales."""
    if y.dtype == torch.int8:
        y = torch.mul(y, scale[:, None], out=torch.empty(y.shape, dtype=torch.bfloat16, device=y.device))
    r = {"y": y}
    if scale is not None:
        r["scale"] = scale
    if residual is not None:
        r["residual"] = residual
    return r


def _plain_out(y, case):
    if case["out"] in LARGEST:
        return _in_8_bits(y, case["out"])
    return y.to(TORCH[case["out"]]), None


def _plain_norm(s):
    x, new = s["x"].float(), None
    if s["residual"] is not None:
        new = (x + s["residual"].float()).to(s["residual"].dtype)
        x = new.float()
    y = x * torch.rsqrt(x.square().mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    return _answer(*_plain_out(y, s["case"]), new)


def _plain_silu(s):
    g = s["x"].float()
    return _answer(*_plain_out(g / (1 + torch.exp(-g)) * s["up"].float(), s["case"]))


def _plain_matrix(case, codes, scales, zeros):
    """A 4-bit matrix in 32 bits."""
    q = torch.stack([codes & 15, codes >> 4], dim=2).flatten(1)[:, : case["cols"]]
    groups, size = scales.shape[1], case["group"]
    spare = groups * size - case["cols"]
    if spare:
        q = torch.nn.functional.pad(q, (0, spare))
    q = q.view(-1, groups, size)
    if case["w"] == E2M1:
        v = torch.tensor(E2M1_VALUES, device=q.device)[q.int()]
    elif zeros is not None:
        v = q.float() - zeros.float()[:, :, None]
    else:
        v = ((q ^ 8).float() - 8)
    return (v * scales.float()[:, :, None]).flatten(1)[:, : case["cols"]]


def _plain_w4(s):
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = x * s["x_scale"][:, None]
    return {"y": [(x @ _plain_matrix(s["case"], *w).t()).to(TORCH[s["case"]["out"]]) for w in s["weights"]]}


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "silu": _plain_silu, "w4": _plain_w4}[op](state)
    from rans_decode_amd import eq
    if op == "norm":
        eq.eq_add_rmsnorm(state["x"], state["weight"], EPS, state["out"], out_scale=state["scale"],
                          residual=state["residual"], residual_out=state["residual_out"])
        return _answer(state["out"], state["scale"], state["residual_out"])
    if op == "silu":
        eq.eq_silu_mul(state["x"], state["up"], state["out"], out_scale=state["scale"])
        return _answer(state["out"], state["scale"])
    n = len(state["ys"])
    eq.eq_w4_matvec(state["block"], [state["x"]] * n, state["ys"], None if state["x_scale"] is None else [state["x_scale"]] * n)
    return {"y": state["ys"]}


# --- the definition in 64 bits --------------------------------------------------


def _round_e4m3(v):
    """v to the nearest multiple of its E4M3 step (3 bits below the leading one, 2**-9 at the least), ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_out(y, case, residual=None):
    r = {"y": y}
    if case["out"] in LARGEST:
        scale = torch.maximum(y.abs().max(dim=1).values, torch.tensor(SMALLEST_AMAX, dtype=torch.float64, device=y.device)) / LARGEST[case["out"]]
        codes = y / scale[:, None]
        r = {"y": torch.round(codes) * scale[:, None] if case["out"] == INT8 else _round_e4m3(codes), "scale": scale}
    if residual is not None:
        r["residual"] = residual
    return r


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "norm":
        new = None
        if s["residual"] is not None:
            new = x + s["residual"].double()
            # the norm is of the residual as it is stored
            x = new.float().to(s["residual"].dtype).double()
        size = torch.sqrt((x * x).sum(dim=1) / case["cols"] + EPS)
        return _exact_out(x / size[:, None] * s["weight"].double()[None, :], case, new)
    if case["op"] == "silu":
        return _exact_out(x * torch.sigmoid(x) * s["up"].double(), case)
    if s["x_scale"] is not None:
        x = x * s["x_scale"].double()[:, None]
    cols, ys = case["cols"], []
    group_of = torch.arange(cols, device="cuda") // case["group"]
    for codes, scales, zeros in s["weights"]:
        parts = []
        for at in range(0, codes.shape[0], 2048):
            c = codes[at:at + 2048].to(torch.int64)
            q = torch.empty(c.shape[0], 2 * c.shape[1], dtype=torch.float64, device="cuda")
            for half in (0, 1):
                n = (c // 16 ** half) % 16
                if case["w"] == INT4:
                    q[:, half::2] = n.double() if zeros is not None else torch.where(n > 7, n - 16, n).double()
                else:
                    exponent, last = (n % 8) // 2, (n % 2).double()
                    size = torch.where(exponent == 0, 0.5 * last, (1 + 0.5 * last) * 2.0 ** (exponent.double() - 1))
                    q[:, half::2] = torch.where(n > 7, -size, size)
            q = q[:, :cols]
            if zeros is not None:
                q = q - zeros[at:at + 2048].double()[:, group_of]
            parts.append(x @ (q * scales[at:at + 2048].double()[:, group_of]).t())
        ys.append(torch.cat(parts, dim=1))
    return {"y": ys}
