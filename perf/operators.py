"""The serving operators on 4-bit rows, case by case: products with quantised weights, the paged 4-bit key-value cache
(store and load), one new token's attention over it, and the handling of its pages.

`own` chooses between the plain form (elementary torch operations in fp32) and the library's calls.
Head size 128, 32 heads (8 key-value heads when grouped), widths 4096, 12288 and 11008 and 2048/4096-token windows are
those of the library's workloads.
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


# ---------------------------------------------------------------------------------------------------------- cases

def _mv(name, n, rows, tokens, dtype, fmt, group, scale):
    return {"name": name, "op": "matvec", "n": n, "rows": rows, "tokens": tokens, "dtype": dtype, "fmt": fmt,
            "group": group, "scale": scale}


def _at(name, seqs, heads, kv, dim, longest, ragged, page, dtype, scale, window=0, sinks=0):
    return {"name": name, "op": "attention", "seqs": seqs, "heads": heads, "kv": kv, "dim": dim, "longest": longest,
            "ragged": ragged, "page": page, "dtype": dtype, "scale": scale, "window": window, "sinks": sinks}


def _ca(name, seqs, kv, dim, new, held, ragged, page, dtype, scale):
    return {"name": name, "op": "cache", "seqs": seqs, "kv": kv, "dim": dim, "new": new, "held": held,
            "ragged": ragged, "page": page, "dtype": dtype, "scale": scale}


def _pg(name, kind, layers, seqs, kv, dim, longest, page, many, spread):
    return {"name": name, "op": "pages", "kind": kind, "layers": layers, "seqs": seqs, "kv": kv, "dim": dim,
            "longest": longest, "page": page, "many": many, "spread": spread}


def listed():
    return [
        # one token through an attention projection of a 4096-wide model: latency counts
        _mv("mv_4096_1", 4096, 4096, 1, "bf16", "int4", 128, "f16"),
        # four sequences' next tokens through the up projection, NVFP4 weights
        _mv("mv_up_nvfp4_4", 4096, 12288, 4, "f16", "nvfp4", 16, "e4m3"),
        # sixteen sequences through the down projection (12 x 1024), one scale per output row
        _mv("mv_down_12288_16", 12288, 4096, 16, "bf16", "int4", 0, "f32"),
        # a large batch on the 172 x 64 width, MXFP4 weights, an odd number of rows and tokens, fp32 in and out
        _mv("mv_11008_mx_61", 11008, 4001, 61, "f32", "mxfp4", 32, "e8m0"),
        # one short conversation, every head with keys of its own: latency counts
        _at("at_one_short", 1, 32, 32, 128, 515, 0, 16, "bf16", "f16"),
        # the KV workload: 32 sequences x 32 heads x 4096 tokens
        _at("at_batch_4096", 32, 32, 32, 128, 4096, 0, 16, "bf16", "f16"),
        # one long context, grouped heads: only a split over the length fills the chip
        _at("at_long_131072", 1, 32, 8, 128, 131072, 0, 64, "bf16", "f16"),
        # ragged batch with an empty and a one-token sequence, sliding window and four first tokens
        _at("at_window_ragged", 48, 32, 8, 128, 32768, 11, 32, "f16", "f32", 2048, 4),
        # each running sequence stores its new token and the row is read back: latency counts
        _ca("ca_decode_32", 32, 8, 128, 1, 2048, 3, 16, "bf16", "f16"),
        # prompts of uneven lengths are stored and read back for the next chunk
        _ca("ca_prompts", 12, 32, 128, 4096, 777, 5, 16, "bf16", "f16"),
        # parallel sampling: finished samples are freed, a prompt is forked, room for the next tokens is made
        _pg("pg_fork", "fork", 36, 64, 8, 128, 2048, 16, 16, 7),
        # half the sequences have ended: their pages are freed and the live ones moved together
        _pg("pg_compact", "compact", 36, 32, 8, 128, 1024, 16, 16, 9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matvec", "matvec", "attention", "attention", "cache", "pages"])
    if op == "matvec":
        fmt = rng.choice(["int4", "int4", "nvfp4", "mxfp4"])
        n = rng.choice([1024, 2048, 4096, 8192, 12288, 11008, 5504])
        group = {"nvfp4": 16, "mxfp4": 32}.get(fmt) or rng.choice([0, 16, 32, 64, 128, 128])
        scale = {"nvfp4": "e4m3", "mxfp4": "e8m0"}.get(fmt) or rng.choice(["f16", "f32"])
        c = _mv("", n, _log(rng, 200, 12000), _log(rng, 1, 61), rng.choice(["bf16", "f16", "f32"]), fmt, group, scale)
    elif op == "attention":
        kv = rng.choice([1, 2, 4, 8, 8, 32])
        longest = _log(rng, 1, 60000)
        seqs = max(1, min(_log(rng, 1, 48), 4000000 // (longest * kv) or 1))
        c = _at("", seqs, kv * rng.choice([1, 2, 4, 7, 8] if kv < 32 else [1]), kv, rng.choice([64, 128, 128, 256]), longest,
                rng.choice([0, rng.randint(1, 9999)]), rng.choice([16, 32, 64]), rng.choice(["bf16", "f16"]),
                rng.choice(["f16", "f32"]))
        if rng.random() < 0.4:
            c["window"], c["sinks"] = _log(rng, 1, 5000), rng.choice([0, 1, 4, 21])
    elif op == "cache":
        kv = rng.choice([1, 2, 8, 32])
        seqs = _log(rng, 1, 48)
        new = max(1, min(_log(rng, 1, 4000), 1500000 // (kv * seqs)))
        c = _ca("", seqs, kv, rng.choice([64, 128, 128, 256]), new, _log(rng, 1, 3000), rng.randint(1, 9999),
                rng.choice([16, 32, 64]), rng.choice(["bf16", "f16"]), rng.choice(["f16", "f32"]))
    else:
        seqs = 2 * _log(rng, 4, 32)
        c = _pg("", rng.choice(["fork", "compact"]), _log(rng, 1, 36), seqs, rng.choice([1, 2, 8]), rng.choice([64, 128]),
                _log(rng, 20, 1024), rng.choice([16, 32]), rng.randint(1, seqs // 2), rng.randint(1, 9999))
    del c["name"]
    return c


def _spread(case):
    """Lengths of a case's sequences: all `longest`, or spread from empty over one token to the longest."""
    n, most = case["seqs"], case["longest"]
    if not case["ragged"]:
        return [most] * n
    r = random.Random(case["ragged"])
    return ([most, 0, 1] + [max(1, _log(r, 1, most)) for _ in range(n)])[:n]


def _news(case):
    """(lengths after the new tokens, new tokens of each sequence) of a cache case."""
    r = random.Random(case["ragged"])
    new = [case["new"] if case["new"] == 1 or i == 0 else r.randint(1, case["new"]) for i in range(case["seqs"])]
    return [r.randint(0, case["held"]) + k for k in new], new


def _plan(case):
    """Lengths, dropped sequences, fork sources and targets of a pages case (whole numbers, from the case alone)."""
    r = random.Random(case["spread"])
    n, m = case["seqs"], case["many"]
    lens = [r.randint(1, case["longest"]) for _ in range(n)]
    drop = sorted(r.sample(range(n), m))
    kept = [i for i in range(n) if i not in drop]
    src = [r.choice(kept[:max(1, len(kept) // 4)]) for _ in drop]
    return lens, drop, src


def _visible(case):
    w, k = case["window"], case["sinks"]
    return [x if not w else min(x, w + min(k, max(0, x - w))) for x in _spread(case)]


def work(case):
    op = case["op"]
    if op == "matvec":
        n, rows, t = case["n"], case["rows"], case["tokens"]
        size = DT[case["dtype"]].itemsize
        sb = {"f32": 4, "f16": 2}.get(case["scale"], 1)
        return {"bytes": rows * n / 2 + rows * (n // (case["group"] or n)) * sb + t * (n + rows) * size + n,
                "flops": 2.0 * rows * n * t}
    if op == "attention":
        d, vis = case["dim"], sum(_visible(case))
        sb = SDT[case["scale"]].itemsize
        return {"bytes": vis * case["kv"] * 2.0 * (d / 2 + sb) + 4.0 * case["seqs"] * case["heads"] * d
                + 4.0 * sum(-(-x // case["page"]) for x in _visible(case)), "flops": 4.0 * vis * case["heads"] * d}
    if op == "cache":
        rows = 2 * sum(_news(case)[1]) * case["kv"]
        d, sb = case["dim"], SDT[case["scale"]].itemsize
        return {"bytes": rows * (2.0 * d + 2 * (d / 2 + sb) + 2.0 * d), "flops": 2.0 * rows * d * math.log2(d)}
    lens, drop, src = _plan(case)
    slot = case["layers"] * case["kv"] * 2 * (case["dim"] / 2 + 2)
    width = -(-(case["longest"] + 8) // case["page"]) + 1
    small = 4.0 * 2 * (case["seqs"] * width + case["seqs"] + _pool(case))
    if case["kind"] == "fork":
        return {"bytes": small + 2 * slot * sum(lens[s] % case["page"] for s in src), "flops": 0}
    need = [-(-x // case["page"]) for x in lens]
    live = sum(need) - sum(need[i] for i in drop)
    order = _order(case)
    at = np.cumsum([0] + need)
    held = np.concatenate([order[at[i]:at[i + 1]] for i in range(len(need)) if i not in drop])
    return {"bytes": small + 2 * slot * case["page"] * int((held >= live).sum()), "flops": 0}


def _pool(case):
    return sum(-(-x // case["page"]) for x in _plan(case)[0]) + 2 * case["seqs"] + 8


def _order(case):
    return np.random.RandomState(case["spread"]).permutation(_pool(case))


# ----------------------------------------------------------------------------------------------- what is in hand

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _signs(n, g):
    return (torch.randint(0, 2, (n,), generator=g, device=DEV) * 2 - 1).to(torch.int8)


def _pack(c):
    return (c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)


def _codes(shape, scale, g):
    """Packed INT4 rows (last axis: one row) of near-Gaussian values, as rotated rows are, with their scales."""
    y = torch.randn(shape, generator=g, device=DEV) * (0.5 + torch.rand(shape[:-1] + (1,), generator=g, device=DEV) * 1.5)
    s = (y.abs().amax(-1, keepdim=True) / 7).to(SDT[scale])
    c = torch.round(y / s.float()).clamp_(-8, 7).to(torch.int8).view(torch.uint8)
    return _pack(c).contiguous(), s.squeeze(-1).contiguous()


def _rows_to_e2m1(v):
    edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    return (torch.bucketize(v.abs(), edge) + 8 * (v < 0)).to(torch.uint8)


def _prepare_matvec(case, g):
    n, rows, t = case["n"], case["rows"], case["tokens"]
    w = torch.randn(rows, n, generator=g, device=DEV) * 0.02
    state = {"signs": _signs(n, g), "tensor_scale": None}
    group = case["group"] or n
    b = w.view(rows, n // group, group)
    top = b.abs().amax(-1, keepdim=True)
    if case["fmt"] == "int4":
        s = (top / 7).to(SDT[case["scale"]])
        c = torch.round(b / s.float()).clamp_(-8, 7).to(torch.int8).view(torch.uint8)
    elif case["fmt"] == "nvfp4":
        ts = (w.abs().max() / 2688).reshape(1)
        s = (top / (6 * ts)).to(torch.float8_e4m3fn)
        c = _rows_to_e2m1(b / (s.float() * ts))
        s, state["tensor_scale"] = s.view(torch.uint8), ts
    else:
        e = torch.floor(torch.log2(top)) - 2
        c = _rows_to_e2m1(b / torch.exp2(e))
        s = (e + 127).to(torch.uint8)
    state["packed"], state["scales"] = _pack(c.view(rows, n)).contiguous(), s.squeeze(-1).contiguous()
    # activations: log-normal channels and a few far larger ones
    x = torch.randn(t, n, generator=g, device=DEV) * torch.exp(0.5 * torch.randn(n, generator=g, device=DEV))
    x[:, torch.randperm(n, generator=g, device=DEV)[:8]] *= 30
    state["x"] = x.to(DT[case["dtype"]])
    return state


def _prepare_pool(pages, case, g, layers=None):
    shape = (() if layers is None else (layers,)) + (pages, case["kv"], case["page"], case["dim"])
    k, ks = _codes(shape, case.get("scale", "f16"), g)
    v, vs = _codes(shape, case.get("scale", "f16"), g)
    return {"k": k, "ks": ks, "v": v, "vs": vs}


def _table(lens, page, order, width):
    t = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for i, x in enumerate(lens):
        k = -(-x // page)
        t[i, :k] = order[at:at + k]
        at += k
    return t


def _prepare_attention(case, g, rs):
    lens, page = _spread(case), case["page"]
    pages = sum(-(-x // page) for x in lens) + 5
    width = -(-max(lens) // page) + 1
    state = _prepare_pool(pages, case, g)
    state["table"] = torch.from_numpy(_table(lens, page, rs.permutation(pages), width)).to(DEV)
    state["lengths"] = _ints(lens)
    state["k_signs"], state["v_signs"] = _signs(case["dim"], g), _signs(case["dim"], g)
    state["q"] = torch.randn(case["seqs"], case["heads"], case["dim"], generator=g, device=DEV).to(DT[case["dtype"]])
    return state


def _prepare_cache(case, g, rs):
    lens, new = _news(case)
    page = case["page"]
    pages = sum(-(-x // page) for x in lens) + 3
    state = _prepare_pool(pages, case, g)
    state["table"] = torch.from_numpy(_table(lens, page, rs.permutation(pages), -(-max(lens) // page) + 1)).to(DEV)
    state["lengths"], state["starts"] = _ints(lens), _ints([0] + list(np.cumsum(new)))
    state["k_signs"], state["v_signs"] = _signs(case["dim"], g), _signs(case["dim"], g)
    # keys and values lie side by side, as a fused projection leaves them; 1% of the values are ten times larger
    kv = torch.randn(sum(new), 2, case["kv"], case["dim"], generator=g, device=DEV)
    kv = torch.where(torch.rand(kv.shape, generator=g, device=DEV) < 0.01, kv * 10, kv).to(DT[case["dtype"]])
    state["new_k"], state["new_v"] = kv[:, 0], kv[:, 1]
    return state


def _prepare_pages(case, g):
    lens, drop, src = _plan(case)
    page = case["page"]
    pages = _pool(case)
    state = _prepare_pool(pages, case, g, case["layers"])
    t = _table(lens, page, _order(case), -(-(case["longest"] + 8) // page) + 1)
    refs = np.zeros(pages, dtype=np.int32)
    refs[t[t >= 0]] = 1
    state["table"], state["refs"] = torch.from_numpy(t).to(DEV), torch.from_numpy(refs).to(DEV)
    state["lengths"], state["drop"], state["src"] = _ints(lens), _ints(drop), _ints(src)
    state["add"] = _ints([1 + i % 8 for i in range(case["seqs"])])
    return state


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 31))
    op = case["op"]
    state = (_prepare_matvec(case, g) if op == "matvec" else _prepare_attention(case, g, rs) if op == "attention"
             else _prepare_cache(case, g, rs) if op == "cache" else _prepare_pages(case, g))
    return state | {"case": dict(case)}


# ------------------------------------------------------------------------------------------------ the plain forms

def _sylvester(n):
    i = torch.arange(n, device=DEV)
    p = i[:, None] & i[None, :]
    p = p ^ (p >> 8)
    p = p ^ (p >> 4)
    p = p ^ (p >> 2)
    p = p ^ (p >> 1)
    return (1 - 2 * (p & 1)).float()


def _blocks(a, b, c, d, pattern):
    m = {"a": a, "b": b, "c": c, "d": d, "A": -a, "B": -b, "C": -c, "D": -d}
    return np.block([[m[x] for x in row] for row in pattern.split()])


def _odd_factor(n):
    """The order-12 or order-172 factor of a width, or the order-1 one."""
    if n % 43 == 0:
        sub = [1, 6, 7, 36, 37, 42]
        i = np.arange(43)
        first = lambda cosets: np.where(np.isin(i, [pow(3, c, 43) * u % 43 for c in cosets for u in sub]), -1.0, 1.0)  # noqa: E731
        turn = lambda cosets: first(cosets)[(i[None, :] - i[:, None]) % 43]  # noqa: E731
        return _blocks(turn([4, 5, 6]), turn([0, 3, 4, 6]), turn([0, 2, 6]), turn([0, 1, 4]), "abcd BaDc CdaB DCba")
    if n % 3 == 0:
        a, b = np.ones((3, 3)), np.ones((3, 3)) - 2 * np.eye(3)
        return _blocks(a, b, b, b, "abbb BaBb BbaB BBba")
    return np.ones((1, 1))


def _rotated(x, signs, back=False):
    """H diag(signs) x / sqrt(n) along the last axis in fp32 (back: diag(signs) H^T x / sqrt(n))."""
    n = x.shape[-1]
    f = torch.from_numpy(_odd_factor(n)).to(x.device, torch.float32)
    m = n // f.shape[0]
    a = 1 << (m.bit_length() - 1) // 2
    s = signs.float() / math.sqrt(n)
    y = (x if back else x * s).reshape(-1, f.shape[0], a, m // a)
    y = _sylvester(a) @ y @ _sylvester(m // a)
    y = ((f.t() if back else f) @ y.reshape(-1, f.shape[0], m)).reshape(x.shape)
    return y * s if back else y


def _nibbles(p):
    return torch.stack((p & 15, p >> 4), -1).flatten(-2)


def _int4(p):
    c = _nibbles(p).to(torch.int8)
    return (c - 16 * (c > 7)).float()


def _weights(s):
    """Dequantised weight rows in the rotated basis, fp32."""
    case, p = s["case"], s["packed"]
    rows, n = p.shape[0], 2 * p.shape[1]
    group = case["group"] or n
    if case["fmt"] == "int4":
        c, scale = _int4(p), s["scales"].float()
    else:
        c = _nibbles(p).long()
        c = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=p.device)[c]
        scale = (torch.exp2(s["scales"].float() - 127) if case["fmt"] == "mxfp4"
                 else s["scales"].view(torch.float8_e4m3fn).float() * s["tensor_scale"])
    return (c.view(rows, n // group, group) * scale[..., None]).view(rows, n)


def _plain_matvec(s):
    return (_rotated(s["x"].float(), s["signs"]) @ _weights(s).t()).to(s["x"].dtype)


def _plain_attention(s):
    case, table, lens, q = s["case"], s["table"], s["lengths"].long(), s["q"]
    seqs, heads, d = q.shape
    kv, page = case["kv"], case["page"]
    most = table.shape[1] * page
    t = table.clamp(min=0).long()
    k = (_int4(s["k"][t]) * s["ks"][t].float()[..., None]).transpose(1, 2).reshape(seqs, kv, most, d)
    v = (_int4(s["v"][t]) * s["vs"][t].float()[..., None]).transpose(1, 2).reshape(seqs, kv, most, d)
    at = torch.arange(most, device=q.device)[None]
    seen = at < lens[:, None]
    if case["window"]:
        seen = seen & ((at >= lens[:, None] - case["window"]) | (at < case["sinks"]))
    seen = seen[:, None, None]
    qr = _rotated(q.float(), s["k_signs"]).reshape(seqs, kv, heads // kv, d)
    x = (qr @ k.transpose(2, 3)) / math.sqrt(d)
    x = torch.where(seen, x, torch.full_like(x, -1e30))
    p = torch.where(seen, torch.exp(x - x.amax(-1, keepdim=True)), torch.zeros_like(x))
    o = (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return _rotated(o.reshape(seqs, heads, d), s["v_signs"], back=True).to(q.dtype)


def _places(s):
    """(page, slot) of every new token."""
    page, starts, lens = s["case"]["page"], s["starts"].long(), s["lengths"].long()
    t = torch.arange(s["new_k"].shape[0], device=lens.device)
    i = torch.searchsorted(starts, t, right=True) - 1
    pos = lens[i] - starts[i + 1] + t
    return s["table"].long()[i, pos // page], pos % page


def _store(x, signs, codes, scales, at):
    y = _rotated(x.float(), signs)
    sc = (y.abs().amax(-1, keepdim=True) / 7).to(scales.dtype)
    c = torch.round(y / sc.float().clamp(min=1e-30)).clamp(-8, 7).to(torch.int8).view(torch.uint8)
    codes[at[0], :, at[1]] = _pack(c)
    scales[at[0], :, at[1]] = sc.squeeze(-1)


def _load(codes, scales, signs, at, dtype):
    y = _int4(codes[at[0], :, at[1]]) * scales[at[0], :, at[1]].float()[..., None]
    return _rotated(y, signs, back=True).to(dtype)


def _plain_cache(s):
    at = _places(s)
    _store(s["new_k"], s["k_signs"], s["k"], s["ks"], at)
    _store(s["new_v"], s["v_signs"], s["v"], s["vs"], at)
    dtype = s["new_k"].dtype
    return _load(s["k"], s["ks"], s["k_signs"], at, dtype), _load(s["v"], s["vs"], s["v_signs"], at, dtype)


def _plain_free(table, lens, refs, drop):
    held = table[drop.long()].flatten().long()
    refs -= torch.bincount(held[held >= 0], minlength=refs.shape[0]).to(refs.dtype)
    table[drop.long()] = -1
    lens[drop.long()] = 0


def _free_pages(refs):
    return torch.nonzero(refs == 0).flatten()


def _plain_fork(s, table, lens, refs, src, dst):
    page, src, dst = s["case"]["page"], src.long(), dst.long()
    n = lens[src].long()
    full, rest = n // page, n % page
    rows = table[src].clone()
    at = torch.arange(table.shape[1], device=table.device)[None]
    whole = rows[(at < full[:, None]) & (rows >= 0)].long()
    part = torch.nonzero(rest).flatten()
    old = rows[part, full[part]].long()
    fresh = _free_pages(refs)[:part.shape[0]]
    refs += torch.bincount(whole, minlength=refs.shape[0]).to(refs.dtype)
    refs[fresh] = 1
    rows = torch.where(at < full[:, None], rows, torch.full_like(rows, -1))
    rows[part, full[part]] = fresh.to(rows.dtype)
    table[dst], lens[dst] = rows, lens[src]
    slot = torch.arange(page, device=table.device)[None] < rest[part][:, None]
    i, j = torch.nonzero(slot, as_tuple=True)
    for name in ("k", "ks", "v", "vs"):
        s[name][:, fresh[i], :, j] = s[name][:, old[i], :, j]
    return torch.zeros(1, dtype=torch.int32, device=table.device)


def _plain_reserve(table, lens, refs, add, page):
    after = lens + add
    at = torch.arange(table.shape[1], device=table.device)[None]
    need = (at >= -(-lens // page)[:, None]) & (at < -(-after // page)[:, None]) & (table < 0)
    i, j = torch.nonzero(need, as_tuple=True)
    fresh = _free_pages(refs)[:i.shape[0]]
    table[i, j] = fresh.to(table.dtype)
    refs[fresh] = 1
    lens.copy_(after)
    return torch.zeros(1, dtype=torch.int32, device=table.device)


def _plain_compact(s, table, refs):
    live = (refs > 0).sum()
    at = torch.arange(refs.shape[0], device=refs.device)
    old = torch.nonzero((refs > 0) & (at >= live)).flatten()
    new = torch.nonzero((refs == 0) & (at < live)).flatten()
    for name in ("k", "ks", "v", "vs"):
        s[name][:, new] = s[name][:, old]
    to = at.to(table.dtype)
    to[old] = new.to(table.dtype)
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))
    refs[new] = refs[old]
    refs[old] = 0
    return live.to(torch.int32).reshape(1)


def _plain_pages(s):
    table, lens, refs = s["table"].clone(), s["lengths"].clone(), s["refs"].clone()
    _plain_free(table, lens, refs, s["drop"])
    if s["case"]["kind"] == "fork":
        said = [_plain_fork(s, table, lens, refs, s["src"], s["drop"]), _plain_reserve(table, lens, refs, s["add"], s["case"]["page"])]
    else:
        said = [_plain_compact(s, table, refs)]
    return [table, lens, refs, said, s["k"], s["ks"], s["v"], s["vs"]]


# ------------------------------------------------------------------------------------------------- one pass of each

def _own_matvec(R, s):
    c = s["case"]
    return R.rhtq_matvec(s["packed"], s["scales"], s["x"], s["signs"], fmt=c["fmt"], group=c["group"], scale_dtype=c["scale"],
                         tensor_scale=s["tensor_scale"])


def _own_cache(R, s):
    return R.RhtqCache(s["k"], s["ks"], s["v"], s["vs"])


def _own_attention(R, s):
    c = s["case"]
    return R.rhtq_paged_attention(s["q"], _own_cache(R, s), s["table"], s["lengths"], s["k_signs"], s["v_signs"],
                                  window=c["window"], sinks=c["sinks"])


def _own_store_load(R, s):
    cache = _own_cache(R, s)
    R.rhtq_cache_append(cache, s["new_k"], s["new_v"], s["table"], s["lengths"], s["starts"], s["k_signs"], s["v_signs"])
    return R.rhtq_cache_read(cache, s["table"], s["lengths"], s["starts"], s["new_k"].shape[0], s["k_signs"], s["v_signs"],
                             dtype=s["new_k"].dtype)


def _own_pages(R, s):
    table, lens, refs, cache = s["table"].clone(), s["lengths"].clone(), s["refs"].clone(), _own_cache(R, s)
    R.rhtq_pages_free(table, lens, refs, s["drop"])
    if s["case"]["kind"] == "fork":
        said = [R.rhtq_pages_fork(cache, table, lens, refs, s["src"], s["drop"]),
                R.rhtq_pages_reserve(table, lens, refs, s["add"], s["case"]["page"])]
    else:
        said = [R.rhtq_pages_compact(cache, table, refs)]
    return [table, lens, refs, said, s["k"], s["ks"], s["v"], s["vs"]]


def run(state):
    op = state["case"]["op"]
    if own:
        import randomized_hadamard_rotation_amd as R
        return {"matvec": _own_matvec, "attention": _own_attention, "cache": _own_store_load, "pages": _own_pages}[op](R, state)
    return {"matvec": _plain_matvec, "attention": _plain_attention, "cache": _plain_cache, "pages": _plain_pages}[op](state)


# ------------------------------------------------------------------------------------- the definition, in 64 bits

def _exact_rotation(x, signs, back=False):
    """Butterflies in 64 bits over the power of two, then the dense odd factor."""
    n = x.shape[-1]
    f = torch.from_numpy(_odd_factor(n)).to(x.device)
    m = n // f.shape[0]
    y = (x if back else x * signs.double()).reshape(-1, m)
    h = 1
    while h < m:
        y = y.reshape(-1, m // (2 * h), 2, h)
        y = torch.stack((y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]), 2).reshape(-1, m)
        h *= 2
    y = y.reshape(-1, f.shape[0], m).transpose(1, 2) @ (f if back else f.t())
    y = y.transpose(1, 2).reshape(x.shape) / math.sqrt(n)
    return y * signs.double() if back else y


def _exact_codes(p):
    lo, hi = (p & 15).to(torch.int16), (p >> 4).to(torch.int16)
    c = torch.empty(p.shape[:-1] + (2 * p.shape[-1],), dtype=torch.float64, device=p.device)
    c[..., 0::2] = torch.where(lo < 8, lo, lo - 16).double()
    c[..., 1::2] = torch.where(hi < 8, hi, hi - 16).double()
    return c


def _exact_matvec(s):
    case, n = s["case"], s["x"].shape[1]
    if case["fmt"] == "int4":
        w, sc = _exact_codes(s["packed"]), s["scales"].double()
    else:
        c = torch.stack((s["packed"] % 16, s["packed"] // 16), 2).reshape(-1, n)
        mag = torch.zeros(c.shape, dtype=torch.float64, device=c.device)
        for i, v in enumerate(E2M1):
            mag[c % 8 == i] = v
        w = torch.where(c >= 8, -mag, mag)
        b = s["scales"].double()
        if case["fmt"] == "mxfp4":
            sc = torch.pow(2.0, b - 127)
        else:
            e, m = torch.floor(b / 8), b % 8
            sc = torch.where(e == 0, m / 512, (8 + m) * torch.pow(2.0, e - 10)) * s["tensor_scale"].double()
    w = w * sc.repeat_interleave(n // sc.shape[1], 1)
    return _exact_rotation(s["x"].double(), s["signs"]) @ w.t()


def _exact_attention(s):
    case, q = s["case"], s["q"].double()
    heads, d = q.shape[1:]
    each = heads // case["kv"]
    out = torch.zeros_like(q)
    for i, n in enumerate(_spread(case)):
        pos = [j for j in range(n) if not case["window"] or j >= n - case["window"] or j < case["sinks"]]
        if not pos:
            continue
        pos = torch.tensor(pos, device=q.device)
        pg, sl = s["table"][i].long()[pos // case["page"]], pos % case["page"]
        for h in range(case["kv"]):
            k = _exact_rotation(_exact_codes(s["k"][pg, h, sl]) * s["ks"][pg, h, sl].double()[:, None], s["k_signs"], back=True)
            v = _exact_rotation(_exact_codes(s["v"][pg, h, sl]) * s["vs"][pg, h, sl].double()[:, None], s["v_signs"], back=True)
            p = torch.softmax(q[i, h * each:(h + 1) * each] @ k.t() / math.sqrt(d), -1)
            out[i, h * each:(h + 1) * each] = p @ v
    return out


def _exact_row(x, signs, scale):
    y = _exact_rotation(x.double(), signs)
    sc = (y.abs().amax(-1, keepdim=True) / 7).to(SDT[scale]).double()
    c = torch.round(torch.where(sc > 0, y / torch.where(sc > 0, sc, 1.0), 0.0)).clamp(-8, 7)
    return _exact_rotation(c * sc, signs, back=True)


def exact(case, seed):
    if case["op"] == "pages":
        return None
    if case["op"] == "attention" and sum(_visible(case)) * case["kv"] > 5e6:
        return None
    s = prepare(case, seed)
    if case["op"] == "matvec":
        return _exact_matvec(s)
    if case["op"] == "attention":
        return _exact_attention(s)
    return _exact_row(s["new_k"], s["k_signs"], case["scale"]), _exact_row(s["new_v"], s["v_signs"], case["scale"])
