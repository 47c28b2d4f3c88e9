"""Products of rows that are quantised on both sides, dense and grouped by expert, and the norm that makes such rows, case by case.

`own` chooses between the plain form (elementary torch operations in fp32) and the library's calls.  Widths 4096, 12288, 11008 and
2048 tokens are those of the library's workloads; expert counts are generic.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SDT = {"f16": torch.float16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEV = "cuda"
BITS = {"int4": 4, "nvfp4": 4, "mxfp4": 4, "int8": 8, "mxfp8": 8}
FIXED = {"nvfp4": (16, "e4m3"), "mxfp4": (32, "e8m0"), "mxfp8": (32, "e8m0")}
MOST_WORK = 8192 * 12288 * 4096
EPS = 1e-5


# ---------------------------------------------------------------------------------------------------------- cases

def _mm(name, n, rows, tokens, a, ag, w, wg, scale, out):
    return {"name": name, "op": "matmul", "n": n, "rows": rows, "tokens": tokens, "a": a, "ag": ag, "w": w, "wg": wg, "scale": scale, "out": out}


def _gm(name, n, rows, tokens, top, experts, uneven, a, ag, w, wg, scale, out):
    return {"name": name, "op": "grouped", "n": n, "rows": rows, "tokens": tokens, "top": top, "experts": experts, "uneven": uneven,
            "a": a, "ag": ag, "w": w, "wg": wg, "scale": scale, "out": out}


def _no(name, n, tokens, dtype, residual, weight, block, fmt, group, scale):
    return {"name": name, "op": "norm", "n": n, "tokens": tokens, "dtype": dtype, "residual": residual, "weight": weight, "block": block,
            "a": fmt, "ag": group, "scale": scale}


def _bl(name, n, rows, tokens, dtype, block, a, ag, w, wg, scale):
    return {"name": name, "op": "block", "n": n, "rows": rows, "tokens": tokens, "dtype": dtype, "residual": True, "weight": False,
            "block": block, "a": a, "ag": ag, "w": w, "wg": wg, "scale": scale, "out": dtype}


def listed():
    return [
        # one token through an attention projection, one scale a token, weights in groups of 128: latency counts
        _mm("mm_int4_1", 4096, 4096, 1, "int4", 0, "int4", 128, "f16", "bf16"),
        # sixteen running sequences through the up projection
        _mm("mm_nvfp4_16", 4096, 12288, 16, "nvfp4", 16, "nvfp4", 16, "e4m3", "bf16"),
        # a prompt of 2048 tokens through the up projection: per-token and per-row scales
        _mm("mm_int4_2048", 4096, 12288, 2048, "int4", 0, "int4", 0, "f32", "bf16"),
        # the same prompt through the down projection, both sides in groups of 128
        _mm("mm_int4g_down_2048", 12288, 4096, 2048, "int4", 128, "int4", 128, "f16", "f16"),
        # a ragged batch of prompts through the 172 x 64 width
        _mm("mm_nvfp4_11008", 11008, 4096, 2047, "nvfp4", 16, "nvfp4", 16, "e4m3", "f16"),
        # a large batch of prompts, the largest call
        _mm("mm_mxfp4_8192", 4096, 12288, 8192, "mxfp4", 32, "mxfp4", 32, "e8m0", "bf16"),
        # 8-bit activations where 4 bits cost too much quality; odd numbers of tokens and rows, fp32 sums
        _mm("mm_mxfp8_333", 11008, 4001, 333, "mxfp8", 32, "mxfp4", 32, "e8m0", "f32"),
        # eight sequences' next tokens, four experts of 64 each: the weights of whichever are called
        _gm("gm_decode_8", 2048, 4096, 8, 4, 64, 3, "int4", 0, "int4", 128, "f16", "bf16"),
        # a prompt's tokens, two experts of eight each, unevenly, one of them without any
        _gm("gm_prompt_2048", 4096, 4096, 2048, 2, 8, 5, "mxfp4", 32, "mxfp4", 32, "e8m0", "bf16"),
        # one sequence's next token: norm with weights, 8 bits with one scale, latency counts
        _no("norm_int8_1", 4096, 1, "bf16", True, True, 0, "int8", 0, "f32"),
        # a prompt's tokens: residual, norm (its weights folded into the projections), rotation, 8-bit blocks
        _no("norm_mxfp8_8192", 4096, 8192, "bf16", True, False, 4096, "mxfp8", 32, "e8m0"),
        # residual, norm, rotation and INT4 rows, and the projection that they are for
        _bl("norm_then_mm_512", 4096, 4096, 512, "bf16", 4096, "int4", 0, "int4", 128, "f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _pair(rng, n):
    """Formats, groups and scale type of both sides of a product of width n."""
    kind = rng.choice(["int4", "int4", "int8", "nvfp4", "mxfp4", "mxfp8"])
    if kind in FIXED:
        w = "nvfp4" if kind == "nvfp4" else "mxfp4"
        return kind, FIXED[kind][0], w, FIXED[w][0], FIXED[kind][1]
    fits = [0, 0] + [g for g in (32, 64, 128, 128, 256) if n % g == 0]
    return kind, rng.choice(fits), "int4", rng.choice(fits), rng.choice(["f16", "f32"])


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul", "grouped", "grouped", "norm", "norm", "block"])
    if op == "norm":
        n = rng.choice([1024, 2048, 4096, 8192, 32 * rng.randint(8, 400)])
        fmt = rng.choice(["int8", "mxfp8", "mxfp8"])
        tokens = max(1, min(_log(rng, 1, 8192), 8192 * 4096 // n))
        block = rng.choice([0, 0, n if n & (n - 1) == 0 else n & -n])
        c = _no("", n, tokens, rng.choice(["bf16", "f16", "f32"]), rng.random() < 0.7, rng.random() < 0.5, block,
                fmt, *FIXED.get(fmt, (0 if n % 128 else rng.choice([0, 128]), rng.choice(["f16", "f32"]))))
    else:
        n = rng.choice([1024, 2048, 4096, 4096, 5504, 8192, 11008, 12288, 32 * rng.randint(4, 300)])
        rows = _log(rng, 60, 12288)
        dtype = rng.choice(["bf16", "f16"])
        if op == "matmul":
            tokens = min(_log(rng, 1, 8192), MOST_WORK // (rows * n))
            c = _mm("", n, rows, max(1, tokens), *_pair(rng, n), rng.choice(["bf16", "f16", "f32"]))
        elif op == "grouped":
            experts = _log(rng, 2, 64)
            rows = max(16, min(rows, 64 * 4096 * 2048 // (experts * n)))
            top = rng.randint(1, min(8, experts))
            tokens = min(_log(rng, 1, 2048), MOST_WORK // (8 * top * rows * n))
            c = _gm("", n, rows, max(1, tokens), top, experts, rng.randint(1, 9999), *_pair(rng, n), rng.choice(["bf16", "f16", "f32"]))
        else:
            n = rng.choice([1024, 2048, 4096])
            a, ag, w, wg, scale = _pair(rng, n)
            while a == "nvfp4":
                a, ag, w, wg, scale = _pair(rng, n)
            c = _bl("", n, rows, _log(rng, 1, 2048), dtype, rng.choice([0, n, 128]), a, ag, w, wg, scale)
    del c["name"]
    return c


def _plan(case):
    """The experts (without repeats) that each token of a grouped case calls: whole numbers, from the case alone.  Popularity falls off,
    and the last expert in line is called by none where there are enough others."""
    r = np.random.RandomState(case["uneven"])
    experts, top = case["experts"], case["top"]
    p = 1.0 / (1.0 + np.arange(experts)) ** 0.5
    if experts > top:
        p[-1] = 0.0
    p = p[r.permutation(experts)]
    # the `top` largest of perturbed log weights are a draw without replacement
    noise = -np.log(-np.log(r.uniform(1e-12, 1.0, (case["tokens"], experts))))
    with np.errstate(divide="ignore"):
        return np.argsort(-(np.log(p)[None] + noise), axis=1)[:, :top]


def _counts(case):
    return np.bincount(_plan(case).reshape(-1), minlength=case["experts"])


def _row_bytes(n, fmt, group, scale):
    return n * BITS[fmt] / 8 + (n // (group or n)) * {"f32": 4, "f16": 2}.get(scale, 1)


def work(case):
    n, t, op = case["n"], case["tokens"], case["op"]
    a = _row_bytes(n, case["a"], case["ag"], case["scale"])
    total = {"bytes": 0.0, "flops": 0.0}
    if op in ("norm", "block"):
        size = DT[case["dtype"]].itemsize
        total["bytes"] += t * n * size * (3 if case["residual"] else 1) + (n * size if case["weight"] else 0) + (n if case["block"] else 0)
        total["flops"] += t * n * (8.0 + (math.log2(case["block"]) if case["block"] else 0))
        if op == "norm":
            total["bytes"] += t * a
    if op == "matmul" or op == "block":
        w = _row_bytes(n, case["w"], case["wg"], case["scale"])
        total["bytes"] += (t * a if op == "matmul" else 0) + case["rows"] * w + t * case["rows"] * DT[case["out"]].itemsize
        total["flops"] += 2.0 * t * case["rows"] * n
    elif op == "grouped":
        w = _row_bytes(n, case["w"], case["wg"], case["scale"])
        slots, called = t * case["top"], int((_counts(case) > 0).sum())
        total["bytes"] += t * a + called * case["rows"] * w + slots * (case["rows"] * DT[case["out"]].itemsize + 4)
        total["flops"] += 2.0 * slots * case["rows"] * n
    return total


# ----------------------------------------------------------------------------------------------- what is in hand

def _pack(c):
    return ((c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)).contiguous()


def _to_e2m1(v):
    edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    return (torch.bucketize(v.abs(), edge) + 8 * (v < 0)).to(torch.uint8)


def _quantised(y, fmt, group, scale):
    """Rows of y (last axis) in one of the formats: codes, scales, tensor scale (one for all of the leading axis' entry)."""
    n = y.shape[-1]
    b = y.reshape(*y.shape[:-1], n // (group or n), group or n)
    top = b.abs().amax(-1, keepdim=True)
    ts = None
    if fmt in ("int4", "int8"):
        m = 7 if fmt == "int4" else 127
        s = (top / m).to(SDT[scale])
        c = torch.round(b / s.float().clamp(min=1e-30)).clamp_(-m - 1, m).to(torch.int8).reshape(y.shape)
        c = _pack(c.view(torch.uint8)) if fmt == "int4" else c
    elif fmt == "nvfp4":
        ts = (y.abs().amax((-1, -2)) / 2688).reshape(-1)
        g = ts.reshape(ts.shape[0], 1, 1, 1) if y.dim() == 3 else ts
        s = (top / (6 * g)).to(torch.float8_e4m3fn)
        c = _pack(_to_e2m1(b / (s.float() * g).clamp(min=1e-30)).reshape(y.shape))
        s = s.view(torch.uint8)
    else:
        e = torch.floor(torch.log2(top.clamp(min=1e-30))) - (2 if fmt == "mxfp4" else 8)
        v = (b / torch.exp2(e)).reshape(y.shape)
        c = _pack(_to_e2m1(v)) if fmt == "mxfp4" else v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s = (e + 127).to(torch.uint8)
    return c, s.squeeze(-1).contiguous(), ts


def _weights(case, g, *lead):
    w = torch.randn(*lead, case["rows"], case["n"], generator=g, device=DEV) * 0.02
    return _quantised(w, case["w"], case["wg"], case["scale"])


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n, t = case["n"], case["tokens"]
    state = {"case": dict(case)}
    if case["op"] in ("norm", "block"):
        # a residual stream: log-normal channels, a few far larger ones; its update is smaller
        channel = torch.exp(0.5 * torch.randn(n, generator=g, device=DEV))
        h = torch.randn(t, n, generator=g, device=DEV) * channel
        h[:, torch.randperm(n, generator=g, device=DEV)[:4]] *= 20
        state["x"] = (h if not case["residual"] else 0.3 * torch.randn(t, n, generator=g, device=DEV) * channel).to(DT[case["dtype"]])
        state["residual"] = h.to(DT[case["dtype"]]) if case["residual"] else None
        state["weight"] = (1 + 0.2 * torch.randn(n, generator=g, device=DEV)).to(DT[case["dtype"]]) if case["weight"] else None
        state["signs"] = (torch.randint(0, 2, (n,), generator=g, device=DEV) * 2 - 1).to(torch.int8) if case["block"] else None
    else:
        # rotated activations: near Gaussian, tokens of different size
        x = torch.randn(t, n, generator=g, device=DEV) * torch.exp(0.3 * torch.randn(t, 1, generator=g, device=DEV))
        state["a"] = _quantised(x, case["a"], case["ag"], case["scale"])
    if case["op"] in ("matmul", "block"):
        state["w"] = _weights(case, g)
    elif case["op"] == "grouped":
        state["w"] = _weights(case, g, case["experts"])
        plan = _plan(case).reshape(-1)
        order = np.argsort(plan, kind="stable")
        state["starts"] = torch.tensor(np.concatenate([[0], np.cumsum(_counts(case))]), dtype=torch.int32, device=DEV)
        state["index"] = torch.tensor(order // case["top"], dtype=torch.int32, device=DEV)
    return state


# ------------------------------------------------------------------------------------------------ the plain forms

def _nibbles(p):
    return torch.stack((p & 15, p >> 4), -1).flatten(-2)


def _values(rows, fmt, group):
    """Rows as fp32."""
    c, s, ts = rows
    if fmt == "int4":
        v = _nibbles(c).to(torch.int8)
        v, s = (v - 16 * (v > 7)).float(), s.float()
    elif fmt == "int8":
        v, s = c.float(), s.float()
    elif fmt == "mxfp8":
        v, s = c.view(torch.float8_e4m3fn).float(), torch.exp2(s.float() - 127)
    else:
        v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=c.device)[_nibbles(c).int()]
        s = torch.exp2(s.float() - 127) if fmt == "mxfp4" else s.view(torch.float8_e4m3fn).float() * ts.reshape((-1,) + (1,) * (s.dim() - 1))
    n = v.shape[-1]
    return (v.view(*v.shape[:-1], n // (group or n), group or n) * s[..., None]).view(v.shape)


def _plain_matmul(s):
    case = s["case"]
    return (_values(s["a"], case["a"], case["ag"]) @ _values(s["w"], case["w"], case["wg"]).t()).to(DT[case["out"]])


def _plain_grouped(s):
    """Every expert's slots padded to the longest list, one batched product, and back to their places."""
    case, starts, index = s["case"], s["starts"].long(), s["index"].long()
    slots, most = index.shape[0], int(_counts(case).max())
    at = torch.arange(slots, device=index.device)
    e = torch.searchsorted(starts, at, right=True) - 1
    place = e * most + at - starts[e]
    a = torch.zeros(case["experts"] * most, case["n"], device=index.device)
    a[place] = _values(s["a"], case["a"], case["ag"])[index]
    y = a.view(case["experts"], most, case["n"]) @ _values(s["w"], case["w"], case["wg"]).transpose(1, 2).contiguous()
    return y.view(-1, case["rows"])[place].to(DT[case["out"]])


def _sylvester(n):
    i = torch.arange(n, device=DEV)
    p = i[:, None] & i[None, :]
    p = p ^ (p >> 8)
    p = p ^ (p >> 4)
    p = p ^ (p >> 2)
    p = p ^ (p >> 1)
    return (1 - 2 * (p & 1)).float()


def _plain_rows(s):
    """The normalised, rotated rows in fp32, and the new residual."""
    case, x = s["case"], s["x"].float()
    h = None
    if case["residual"]:
        h = (x + s["residual"].float()).to(s["x"].dtype)
        x = h.float()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    if case["weight"]:
        y = y * s["weight"].float()
    if case["block"]:
        b = case["block"]
        u = 1 << (b.bit_length() - 1) // 2
        y = (_sylvester(u) @ (y * s["signs"].float()).view(-1, u, b // u) @ _sylvester(b // u)).view(y.shape) / math.sqrt(b)
    return y, h


def _plain_norm(s):
    case = s["case"]
    y, h = _plain_rows(s)
    c, sc, _ = _quantised(y, case["a"], case["ag"], case["scale"])
    return _told(c, sc, h, s)


def _told(c, scales, h, s):
    """What a norm case returns: 8-bit codes as the values they stand for, or those before the scale beside the scales' values."""
    case = s["case"]
    out = {} if h is None else {"residual": h}
    if case["a"] == "mxfp8":
        return out | {"codes": c.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}
    n = c.shape[1]
    y = c.view(-1, n // (case["ag"] or n), case["ag"] or n) * scales[..., None].to(torch.bfloat16)
    return out | {"y": y.view(-1, n)}


def _plain_block(s):
    case = s["case"]
    y, h = _plain_rows(s)
    a = _values(_quantised(y, case["a"], case["ag"], case["scale"]), case["a"], case["ag"])
    return {"residual": h, "y": (a @ _values(s["w"], case["w"], case["wg"]).t()).to(DT[case["out"]])}


# ------------------------------------------------------------------------------------------------- one pass of each

def _rows(R, rows, fmt, group):
    return R.RhtqRows(*rows, fmt=fmt, group=group)


def _own_matmul(R, s):
    c = s["case"]
    return R.rhtq_matmul(_rows(R, s["a"], c["a"], c["ag"]), _rows(R, s["w"], c["w"], c["wg"]), out_dtype=DT[c["out"]])


def _own_grouped(R, s):
    c = s["case"]
    return R.rhtq_grouped_matmul(_rows(R, s["a"], c["a"], c["ag"]), _rows(R, s["w"], c["w"], c["wg"]), s["starts"], s["index"],
                                 out_dtype=DT[c["out"]])


def _own_rows(R, s):
    c = s["case"]
    return R.rhtq_norm_forward(s["x"], s["weight"], s["residual"], eps=EPS, signs=s["signs"], block=c["block"], fmt=c["a"], group=c["ag"],
                               scale_dtype=c["scale"])


def _own_norm(R, s):
    rows, h = _own_rows(R, s)
    return _told(rows.codes, rows.scales, h, s)


def _own_block(R, s):
    c = s["case"]
    rows, h = _own_rows(R, s)
    return {"residual": h, "y": R.rhtq_matmul(rows, _rows(R, s["w"], c["w"], c["wg"]), out_dtype=DT[c["out"]])}


def run(state):
    op = state["case"]["op"]
    if own:
        import randomized_hadamard_rotation_amd as R
        return {"matmul": _own_matmul, "grouped": _own_grouped, "norm": _own_norm, "block": _own_block}[op](R, state)
    return {"matmul": _plain_matmul, "grouped": _plain_grouped, "norm": _plain_norm, "block": _plain_block}[op](state)


# ------------------------------------------------------------------------------------- the definition, in 64 bits

def _exact_e2m1(c):
    mag = torch.zeros(c.shape, dtype=torch.float64, device=c.device)
    for i, v in enumerate(E2M1):
        mag[c % 8 == i] = v
    return torch.where(c >= 8, -mag, mag)


def _exact_e4m3(b):
    """E4M3 bytes by their bits."""
    b = b.to(torch.int32)
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m / 512, (8 + m) * torch.pow(2.0, (e - 10).double()))
    return torch.where(b >= 128, -v, v)


def _exact_values(rows, fmt, group):
    c, s, ts = rows
    if BITS[fmt] == 4:
        c = torch.stack((c % 16, c // 16), -1).reshape(*c.shape[:-1], 2 * c.shape[-1])
        v = torch.where(c < 8, c.double(), c.double() - 16) if fmt == "int4" else _exact_e2m1(c)
    else:
        v = c.double() if fmt == "int8" else _exact_e4m3(c)
    if fmt == "nvfp4":
        sc = _exact_e4m3(s) * ts.double().reshape((-1,) + (1,) * (s.dim() - 1))
    else:
        sc = torch.pow(2.0, s.double() - 127) if fmt in FIXED else s.double()
    return v * sc.repeat_interleave(v.shape[-1] // sc.shape[-1], -1)


def _exact_rows(s):
    """The normalised, rotated rows in 64 bits (butterflies), and the new residual."""
    case, x = s["case"], s["x"].double()
    n, h = case["n"], None
    if case["residual"]:
        # two 16- or 32-bit values: their sum in 64 bits rounds once on the way to fp32 and, where the type is shorter, is exact there
        h = (x + s["residual"].double()).float().to(s["x"].dtype)
        x = h.double()
    y = x * (x.square().sum(-1, keepdim=True) / n + EPS).rsqrt()
    if case["weight"]:
        y = y * s["weight"].double()
    if case["block"]:
        b, step = case["block"], 1
        y = y * s["signs"].double()
        while step < b:
            y = y.reshape(-1, n // (2 * step), 2, step)
            y = torch.stack((y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]), 2).reshape(-1, n)
            step *= 2
        y = y / math.sqrt(b)
    return y, h


def _exact_codes(y, fmt, group, scale):
    """(codes' values, scales' values) of rows in 64 bits: each scale from its group's largest value, each value to the nearest code."""
    n = y.shape[1]
    b = y.reshape(y.shape[0], -1, group or n)
    top = b.abs().amax(-1, keepdim=True)
    if fmt in ("int4", "int8"):
        m = 7 if fmt == "int4" else 127
        s = (top / m).to(SDT[scale]).double()
        c = torch.round(b / torch.where(s > 0, s, 1.0)).clamp(-m - 1, m)
    else:
        e = torch.frexp(top)[1].double() - 1 - (2 if fmt == "mxfp4" else 8)
        s = torch.pow(2.0, e)
        v = (b / s).abs().clamp(max=6.0 if fmt == "mxfp4" else 448.0)
        # spacing of the codes at a value's binade, not below that of the smallest normal number
        least, bits = (0.0, 1) if fmt == "mxfp4" else (-6.0, 3)
        step = torch.pow(2.0, (torch.frexp(v)[1].double() - 1).clamp(min=least) - bits)
        c = torch.copysign(torch.round(v / step) * step, b)
    return c, s


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matmul":
        return _exact_values(s["a"], case["a"], case["ag"]) @ _exact_values(s["w"], case["w"], case["wg"]).t()
    if case["op"] == "grouped":
        a, starts = _exact_values(s["a"], case["a"], case["ag"]), s["starts"].tolist()
        y = torch.empty(s["index"].shape[0], case["rows"], dtype=torch.float64, device=DEV)
        for e in range(case["experts"]):
            i, j = starts[e], starts[e + 1]
            w = tuple(None if x is None else x[e:e + 1] for x in s["w"])
            if j > i:
                y[i:j] = a[s["index"][i:j].long()] @ _exact_values(w, case["w"], case["wg"])[0].t()
        return y
    y, h = _exact_rows(s)
    c, sc = _exact_codes(y, case["a"], case["ag"], case["scale"])
    out = {} if h is None else {"residual": h.double()}
    v = (c * sc).reshape(y.shape)
    if case["op"] == "block":
        return out | {"y": v @ _exact_values(s["w"], case["w"], case["wg"]).t()}
    if case["a"] == "mxfp8":
        return out | {"codes": c.reshape(y.shape), "scales": sc.squeeze(-1)}
    return out | {"y": v}
