"""The 8-bit and the ragged matrix products beside the routed NVFP4 layer, as they are timed.

Five kinds of call:

* ``quantize``         rows of activations to int8 codes with an FP32 scale for each row
* ``swiglu_quantize``  the same of h = SiLU(gate) * up, from rows that hold gate | up
* ``int8``             the product of int8 rows and int8 channels, with their scales
* ``grouped``          rows sorted by expert times each expert's own matrix (BF16, F16, int8)
* ``grouped_backward`` the gradients of that product for its rows and for its matrices

``own`` false: the plain forms, elementary torch operations in 32 bits (64 where a value
stands next to a rounding border). ``own`` true: the library's calls. Shapes are those of
the layers that this repository runs (hidden 2048, intermediate 768, 512 experts, top-10;
hidden 256, intermediate 128, 8 experts) and generic ones.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 64          # rows of one block of the plain grouped forms
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one decode token's activations, ahead of an int8 product
        {"name": "quantize_token", "op": "quantize", "rows": 1, "cols": 2048, "type": "bf16"},
        # the W4A8 prompt chunk: 32768 tokens of hidden 2048
        {"name": "quantize_32k", "op": "quantize", "rows": 32768, "cols": 2048, "type": "bf16"},
        # h of a shared expert, four tokens being decoded
        {"name": "swiglu_4", "op": "swiglu_quantize", "rows": 4, "cols": 768, "type": "f32"},
        # h of a shared expert over a ragged prompt chunk
        {"name": "swiglu_8191", "op": "swiglu_quantize", "rows": 8191, "cols": 768, "type": "bf16"},
        # gate and up rows of an 8-bit shared expert for one token
        {"name": "int8_token", "op": "int8", "rows": 1, "n": 1536, "k": 2048, "out": "bf16"},
        # its down projection for a small odd batch
        {"name": "int8_201", "op": "int8", "rows": 201, "n": 2048, "k": 768, "out": "f32"},
        # gate and up of the same for the 32768-token chunk
        {"name": "int8_32k", "op": "int8", "rows": 32768, "n": 1536, "k": 2048, "out": "bf16"},
        # 8 tokens x top-10 over 512 experts left in BF16: most experts empty, the rest 1 to 3 rows
        {"name": "grouped_decode", "op": "grouped", "experts": 512, "rows": 80, "n": 1536, "k": 2048, "type": "bf16",
         "out": "bf16", "skew": 0.5},
        # 8192 tokens x top-10, the same experts, Zipf popularity
        {"name": "grouped_prefill", "op": "grouped", "experts": 512, "rows": 81920, "n": 1536, "k": 2048, "type": "bf16",
         "out": "bf16", "skew": 1.1},
        # experts in 8 bits, a ragged prompt chunk
        {"name": "grouped_int8", "op": "grouped", "experts": 64, "rows": 20011, "n": 2048, "k": 768, "type": "int8",
         "out": "bf16", "skew": 0.8},
        # a training step of a tiny layer: 8 experts, 256 x 128, 128 pairs
        {"name": "backward_tiny", "op": "grouped_backward", "experts": 8, "rows": 128, "n": 256, "k": 256, "type": "bf16",
         "out": "f32", "skew": 0.5},
        # a training step of 64 experts over 16384 pairs
        {"name": "backward_16k", "op": "grouped_backward", "experts": 64, "rows": 16384, "n": 1536, "k": 2048,
         "type": "bf16", "out": "bf16", "skew": 0.8},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; odd as often as not."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "swiglu_quantize", "int8", "grouped", "grouped", "grouped_backward"])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 32768), "cols": _log(rng, 16, 4096), "type": rng.choice(["bf16", "f16", "f32"])}
    if op == "swiglu_quantize":
        return {"op": op, "rows": _log(rng, 1, 32768), "cols": _log(rng, 16, 2048), "type": rng.choice(["bf16", "f16", "f32"])}
    if op == "int8":
        return {"op": op, "rows": _log(rng, 1, 32768), "n": _log(rng, 64, 2560), "k": _log(rng, 64, 2560),
                "out": rng.choice(["bf16", "f16", "f32"])}
    if op == "grouped":
        kind = rng.choice(["bf16", "f16", "int8"])
        return {"op": op, "experts": _log(rng, 1, 128), "rows": _log(rng, 1, 32768), "n": _log(rng, 32, 2048),
                "k": _log(rng, 32, 2048), "type": kind, "out": rng.choice(["f32", "bf16" if kind == "int8" else kind]),
                "skew": round(rng.uniform(0.0, 1.2), 3)}
    kind = rng.choice(["bf16", "f16"])
    return {"op": op, "experts": _log(rng, 1, 64), "rows": _log(rng, 1, 16384), "n": _log(rng, 32, 2048),
            "k": _log(rng, 32, 2048), "type": kind, "out": rng.choice(["f32", kind]), "skew": round(rng.uniform(0.0, 1.2), 3)}


# ------------------------------------------------------------------ inputs

def _padded(shape, dtype):
    """An empty tensor whose rows start every whole number of 16 bytes, as the products read them."""
    unit = 16 // torch.empty(0, dtype=dtype).element_size()
    cols = shape[-1]
    return torch.empty(*shape[:-1], -(-cols // unit) * unit, dtype=dtype, device=DEV)[..., :cols]


def _normal(g, shape, dtype, std=1.0, outliers=False):
    v = torch.randn(*shape, generator=g, device=DEV) * std
    if outliers:    # a thousandth of the channels twenty times as large, at least one
        n = max(1, round(0.001 * shape[-1]))
        v[:, torch.randint(0, shape[-1], (n,), generator=g, device=DEV)] *= 20.0
    out = _padded(shape, dtype)
    out.copy_(v)
    return out


def _codes(g, shape):
    out = _padded(shape, torch.int8)
    out.copy_((torch.randn(*shape, generator=g, device=DEV) * 32.0).round_().clamp_(-127, 127))
    return out


def _scales(g, shape, about):
    return (torch.rand(*shape, generator=g, device=DEV) + 0.5) * about


def _offsets(g, experts, rows, skew):
    """Where each expert's rows begin and end: popularity r^-skew over the experts in a random order."""
    p = torch.arange(1, experts + 1, device=DEV, dtype=torch.float32) ** -skew
    p = p[torch.randperm(experts, generator=g, device=DEV)]
    ids = torch.multinomial(p, rows, replacement=True, generator=g)
    off = torch.zeros(experts + 1, dtype=torch.int64, device=DEV)
    off[1:] = torch.bincount(ids, minlength=experts).cumsum(0)
    return off.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, rows = case["op"], case["rows"]
    s = {"case": case, "op": op}
    if op == "quantize":
        s["x"] = _normal(g, (rows, case["cols"]), TYPES[case["type"]], outliers=True)
    elif op == "swiglu_quantize":
        s["x"] = _normal(g, (rows, 2 * case["cols"]), TYPES[case["type"]])
    elif op == "int8":
        s["x"], s["xs"] = _codes(g, (rows, case["k"])), _scales(g, (rows,), 0.03)
        s["w"], s["ws"] = _codes(g, (case["n"], case["k"])), _scales(g, (case["n"],), 0.0006)
    else:
        e, n, k = case["experts"], case["n"], case["k"]
        s["offsets"] = _offsets(g, e, rows, case["skew"])
        if case["type"] == "int8":
            s["x"], s["xs"] = _codes(g, (rows, k)), _scales(g, (rows,), 0.03)
            s["w"], s["ws"] = _codes(g, (e, n, k)), _scales(g, (e, n), 0.0006)
        else:
            t = TYPES[case["type"]]
            s["x"] = _normal(g, (rows, k), t)
            s["w"] = _padded((e, n, k), t)
            for i in range(e):
                s["w"][i].copy_(torch.randn(n, k, generator=g, device=DEV) * 0.02)
            if op == "grouped_backward":
                s["dy"] = _normal(g, (rows, n), t, 0.1)
    return s


# ------------------------------------------------------------- plain forms

def _swiglu(x, cols):
    gate, up = x[:, :cols], x[:, cols:]
    return gate / (1 + torch.exp(-gate)) * up


def _quantize(v):
    """Codes as whole numbers in 64 bits, and scales: the quotient is taken in 64 bits, for it may stand next to a half."""
    scale = (v.abs().amax(1).double() / 127.0).float()
    safe = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
    return (v.double() / safe[:, None]).round().clamp(-127, 127), scale


def _blocks(offsets, rows):
    """Blocks of up to BLOCK rows of one expert: the expert and the rows of each, and each row's place among them."""
    off = offsets.long()
    experts = off.numel() - 1
    count = off[1:] - off[:-1]
    each = (count + BLOCK - 1) // BLOCK
    upto = each.cumsum(0)
    b = torch.arange(rows // BLOCK + experts, device=DEV)
    e = torch.searchsorted(upto, b, right=True)
    real = e < experts
    e = e.clamp(max=experts - 1)
    at = off[e][:, None] + ((b - (upto - each)[e]) * BLOCK)[:, None] + torch.arange(BLOCK, device=DEV)
    ok = real[:, None] & (at < off[e + 1][:, None])
    p = torch.arange(rows, device=DEV)
    pe = torch.searchsorted(off[1:].contiguous(), p, right=True)
    inside = p - off[pe]
    return e, at.clamp(0, rows - 1), ok, ((upto - each)[pe] + inside // BLOCK) * BLOCK + inside % BLOCK


def _gather(v, at, ok):
    return torch.where(ok[:, :, None], v[at].float(), 0.0)


def _plain(s):
    case, op = s["case"], s["op"]
    if op == "quantize":
        q, scale = _quantize(s["x"].float())
        return {"values": q.float() * scale[:, None], "scale": scale}
    if op == "swiglu_quantize":
        q, scale = _quantize(_swiglu(s["x"].float(), case["cols"]))
        return {"values": (q.float() * scale[:, None]).to(torch.bfloat16), "scale": scale}
    out = TYPES[case["out"]]
    if op == "int8":
        return (s["x"].float() @ s["w"].float().t() * s["xs"][:, None] * s["ws"]).to(out)
    e, at, ok, place = _blocks(s["offsets"], case["rows"])
    if op == "grouped":
        y = torch.bmm(_gather(s["x"], at, ok), s["w"][e].float().transpose(1, 2))
        if case["type"] == "int8":
            y *= s["ws"][e][:, None, :]
        y = y.reshape(-1, case["n"])[place]
        if case["type"] == "int8":
            y *= s["xs"][:, None]
        return y.to(out)
    dy, x = _gather(s["dy"], at, ok), _gather(s["x"], at, ok)
    dx = torch.bmm(dy, s["w"][e].float()).reshape(-1, case["k"])[place].to(TYPES[case["type"]])
    dw = torch.zeros(s["w"].shape, device=DEV).index_add_(0, e, torch.bmm(dy.transpose(1, 2), x))
    return {"dx": dx, "dw": dw.to(out)}


# ------------------------------------------------------------ the library's

def _library(s):
    import nvfp4_mixture_experts_03_b200 as nv
    case, op = s["case"], s["op"]
    if op == "quantize":
        q, scale = nv.quantize_int8(s["x"])
        return {"values": q * scale[:, None], "scale": scale}
    if op == "swiglu_quantize":
        q, scale = nv.quantize_int8(s["x"], swiglu=True)
        values = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        return {"values": torch.mul(q, scale[:, None], out=values), "scale": scale}
    out = TYPES[case["out"]]
    if op == "int8":
        return nv.gemm_int8(s["x"], s["w"], s["xs"], s["ws"], out_dtype=out)
    if op == "grouped":
        return nv.grouped_gemm(s["x"], s["w"], s["offsets"], x_scale=s.get("xs"), w_scale=s.get("ws"), out_dtype=out)
    return {"dx": nv.grouped_gemm_dx(s["dy"], s["w"], s["offsets"]),
            "dw": nv.grouped_gemm_dw(s["dy"], s["x"], s["offsets"], out_dtype=out)}


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------- what it takes

def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4, "int8": 1}
    op, rows = case["op"], case["rows"]
    if op in ("quantize", "swiglu_quantize"):
        wide = 1 if op == "quantize" else 2
        cols = case["cols"]
        return {"bytes": rows * cols * (wide * size[case["type"]] + 1) + 4 * rows, "flops": 6 * rows * cols}
    n, k = case["n"], case["k"]
    if op == "int8":
        return {"bytes": rows * k + n * k + 4 * (rows + n) + rows * n * size[case["out"]], "flops": 2 * rows * n * k}
    # an expert without rows is not read: no more of them are than there are rows
    one, used = size[case["type"]], min(case["experts"], rows)
    if op == "grouped":
        scales = 4 * (rows + used * n) if case["type"] == "int8" else 0
        return {"bytes": one * (rows * k + used * n * k) + scales + rows * n * size[case["out"]], "flops": 2 * rows * n * k}
    # dy, x and the matrices in; dx and every expert's dw, zeros among them, out
    return {"bytes": one * (rows * n + 2 * rows * k + used * n * k) + case["experts"] * n * k * size[case["out"]],
            "flops": 4 * rows * n * k}


# ------------------------------------------------------- the definition, 64 bits

def _codes_of(v, amax):
    """scale: the FP32 number nearest to amax / 127; code: the whole number nearest to v / scale, ties to the even one."""
    scale = (amax / 127.0).to(torch.float32).to(torch.float64)
    code = torch.zeros_like(v)
    some = scale > 0
    code[some] = torch.clamp(torch.round(v[some] / scale[some].unsqueeze(1)), -127, 127)
    return {"values": code * scale.unsqueeze(1), "scale": scale}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        v = s["x"].to(torch.float64)
        return _codes_of(v, v.abs().max(dim=1).values)
    if op == "swiglu_quantize":
        gate, up = s["x"].to(torch.float64).split(case["cols"], dim=1)
        h = gate * torch.sigmoid(gate) * up
        return _codes_of(h, h.abs().max(dim=1).values)
    if op == "int8":
        a = s["x"].to(torch.float64) * s["xs"].to(torch.float64).unsqueeze(1)
        b = s["w"].to(torch.float64) * s["ws"].to(torch.float64).unsqueeze(1)
        return torch.mm(a, b.T)
    off = s["offsets"].tolist()
    rows, n, k = case["rows"], case["n"], case["k"]
    if op == "grouped":
        y = torch.zeros(rows, n, dtype=torch.float64, device=DEV)
        for e in range(case["experts"]):
            lo, hi = off[e], off[e + 1]
            if hi > lo:
                a, b = s["x"][lo:hi].to(torch.float64), s["w"][e].to(torch.float64)
                if case["type"] == "int8":
                    a, b = a * s["xs"][lo:hi, None].to(torch.float64), b * s["ws"][e][:, None].to(torch.float64)
                y[lo:hi] = a @ b.T
        return y
    dx = torch.zeros(rows, k, dtype=torch.float64, device=DEV)
    dw = torch.zeros(case["experts"], n, k, dtype=torch.float64, device=DEV)
    for e in range(case["experts"]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            d = s["dy"][lo:hi].to(torch.float64)
            dx[lo:hi] = d @ s["w"][e].to(torch.float64)
            dw[e] = d.T @ s["x"][lo:hi].to(torch.float64)
    return {"dx": dx, "dw": dw}
