"""GPU: the serving calls against plain 64-bit forms.

Tolerances count roundings: u = eps / 2 of the output type for its one rounding, 2^-24 for each fp32 rounding of a sum, and 2^-16
(2^-22 for fp32 output) of the largest value for an operand that a kernel carries in fixed point or in two halves.
"""
import math
import os
import sys

import numpy as np
import pytest

import oracle as O
from oracle import check as C

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def say(*msg):
    print("[case]", *msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    import randomized_hadamard_rotation_amd as R
    return R


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def signs_of(n, seed):
    return np.where(np.random.RandomState(seed).rand(n) < 0.5, -1, 1).astype(np.int8)


# --------------------------------------------------------------------------------------------------------- matvec

def weights(rows, n, fmt, group, scale, seed, spread=1.0):
    """Packed rows, scales, tensor scale (numpy, as rhtq_forward lays them out) and the dequantised matrix in 64 bits."""
    w = np.random.RandomState(seed).randn(rows, n) * spread
    w[:, ::37] *= 4
    ts = None
    if rows > 2:
        w[1] = 0
        w[2, : n // 2] = 0
    if fmt == "int4":
        p, s = int4_rows(w, group, scale)
    elif fmt == "nvfp4":
        ts = O.nvfp4_tensor_scale(w)
        top = np.abs(w).reshape(rows, n // 16, 16).max(-1)
        s = O.e4m3_encode(top / (6.0 * np.float64(ts)))
        p = O.pack_nibbles(O.nvfp4_codes_from_scales(w, s, ts)[0])
    else:
        e = O.mxfp4_scale_exponent(np.abs(w).reshape(rows, n // 32, 32).max(-1))
        s = (np.asarray(e, dtype=np.int64) + 127).astype(np.uint8)
        c = O.mxfp4_codes_from_scales(w, s)[0]
        p = O.pack_nibbles(c)
    p, s = np.ascontiguousarray(p).astype(np.uint8), np.ascontiguousarray(s)
    return p, s, ts, O.dequantize(p, s, fmt, group, ts)


def int4_rows(w, group, scale):
    rows, n = w.shape
    g = group or n
    s = O.int4_scale_store(np.abs(w).reshape(rows, n // g, g).max(-1), scale)
    s = np.asarray(s).astype(np.float32 if scale == "f32" else np.float16)
    f = s.astype(np.float64)[..., None]
    q = np.clip(np.rint(np.divide(w.reshape(rows, n // g, g), f, out=np.zeros((rows, n // g, g)), where=f > 0)), -8, 7)
    return O.pack_nibbles(q.reshape(rows, n).astype(np.int64)), s


def device_weights(p, s, ts):
    return (torch.from_numpy(p).cuda(), torch.from_numpy(s).cuda(),
            None if ts is None else torch.tensor([float(ts)], dtype=torch.float32, device="cuda"))


def matvec_bound(x, w, out, rot=0.0):
    """Allowed |error| of y = x w^T elementwise: what the operand carries, fp32 sums, one rounding of the output."""
    t, n = x.shape
    b = math.gcd(n, 128)
    top = np.repeat(np.abs(x).reshape(t, n // b, b).max(-1), b, axis=1)
    if b < 128:
        top = np.abs(x).max(-1, keepdims=True) + 0 * x
    carried = 2.0 ** (-22 if out == torch.float32 else -16)
    a = np.abs(x) @ np.abs(w).T
    return (carried * top + rot * np.abs(x).max(-1, keepdims=True)) @ np.abs(w).T + (n / 16 + 64) * 2.0 ** -24 * a


def check_matvec(y, x, w, rot=0.0):
    y64 = y.double().cpu().numpy()
    ref = x @ w.T
    assert y64.shape == ref.shape
    u = half_step(y.dtype)
    tiny = 2.0 ** -25 if y.dtype == torch.float16 else 0.0     # half a step of its subnormals
    allowed = matvec_bound(x, w, y.dtype, rot) * (1 + u) + u * np.abs(ref) + tiny
    bad = ~(np.abs(y64 - ref) <= allowed)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(y64 - ref) / (allowed + 1e-300)):.3g} x allowed"


MATVEC = [
    # n, rows, tokens, fmt, group, scale, x type, out type
    (32, 1, 1, "int4", 0, "f32", "bf16", "bf16"), (32, 5, 3, "int4", 16, "f16", "f32", "f32"), (64, 16, 1, "int4", 32, "f16", "f16", "f16"),
    (96, 17, 2, "int4", 32, "f32", "bf16", "f32"), (160, 15, 2, "int4", 16, "f32", "f32", "bf16"), (128, 33, 8, "int4", 128, "f16", "bf16", "bf16"),
    (256, 31, 9, "int4", 64, "f16", "f16", "f16"), (1024, 100, 1, "int4", 128, "f16", "bf16", "bf16"),
    (4096, 130, 2, "int4", 128, "f16", "bf16", "bf16"), (4096, 65, 1, "int4", 0, "f32", "f32", "f32"), (4096, 64, 7, "int4", 512, "f16", "f16", "f16"),
    (4096, 48, 17, "int4", 16, "f32", "bf16", "bf16"), (2048, 257, 33, "int4", 256, "f16", "f32", "f32"), (12288, 19, 4, "int4", 4096, "f32", "bf16", "bf16"),
    (11008, 40, 61, "int4", 64, "f16", "bf16", "bf16"), (5504, 16, 5, "int4", 32, "f16", "f32", "f32"), (1376, 34, 6, "int4", 0, "f16", "bf16", "bf16"),
    (32, 3, 1, "nvfp4", 16, "e4m3", "bf16", "bf16"), (512, 21, 2, "nvfp4", 16, "e4m3", "f16", "f16"), (4096, 70, 5, "nvfp4", 16, "e4m3", "f32", "f32"),
    (11008, 18, 16, "nvfp4", 16, "e4m3", "bf16", "f32"), (96, 50, 65, "nvfp4", 16, "e4m3", "bf16", "bf16"),
    (32, 2, 2, "mxfp4", 32, "e8m0", "f32", "f32"), (4096, 66, 1, "mxfp4", 32, "e8m0", "bf16", "bf16"), (12288, 33, 10, "mxfp4", 32, "e8m0", "f16", "f16"),
    (2752, 129, 64, "mxfp4", 32, "e8m0", "f32", "f32"), (224, 20, 130, "mxfp4", 32, "e8m0", "bf16", "bf16"),
]


@pytest.mark.parametrize("n,rows,tokens,fmt,group,scale,xt,yt", MATVEC)
def test_matvec_of_rotated_rows(R, n, rows, tokens, fmt, group, scale, xt, yt):
    say("matvec", n, rows, tokens, fmt, group, scale, xt, yt)
    p, s, ts, w = weights(rows, n, fmt, group, scale, seed=n + rows)
    x = torch.from_numpy(np.random.RandomState(tokens).randn(tokens, n) * np.exp(np.random.RandomState(1).randn(n))).to(DT[xt])
    if tokens > 2:
        x[1] = 0
    dp, ds, dts = device_weights(p, s, ts)
    y = R.rhtq_matvec(dp, ds, x.cuda(), fmt=fmt, group=group, scale_dtype=scale, tensor_scale=dts, rotated=True, out_dtype=DT[yt])
    assert y.dtype == DT[yt]
    check_matvec(y, x.double().numpy(), w)


@pytest.mark.parametrize("n,block,fmt,group,scale,xt", [(4096, None, "int4", 128, "f16", "bf16"), (12288, None, "nvfp4", 16, "e4m3", "f16"),
                                                        (11008, None, "mxfp4", 32, "e8m0", "f32"), (1408, 128, "int4", 64, "f16", "bf16"),
                                                        (64, None, "int4", 0, "f32", "bf16")])
def test_matvec_rotates_its_rows(R, n, block, fmt, group, scale, xt):
    """y = x (rhtq_inverse(packed))^T, the rotation taken by the call."""
    say("matvec with rotation", n, block, fmt, group)
    p, s, ts, w = weights(37, n, fmt, group, scale, seed=n)
    sg = signs_of(n, 5)
    x = torch.from_numpy(np.random.RandomState(3).randn(3, n)).to(DT[xt])
    dp, ds, dts = device_weights(p, s, ts)
    xr = O.rotate(x.double().numpy(), sg) if block is None else O.rotate_blocked(x.double().numpy(), sg, block)
    y = R.rhtq_matvec(dp, ds, x.cuda(), sg, fmt=fmt, group=group, scale_dtype=scale, tensor_scale=dts, block=block)
    check_matvec(y, xr, w, rot=C.ROT_REL)
    back = R.rhtq_inverse(dp, ds, n, sg, fmt=fmt, group=group, scale_dtype=scale, tensor_scale=dts, block=block)
    plain = x.double().numpy() @ back.double().cpu().numpy().T
    assert np.linalg.norm(y.double().cpu().numpy() - plain) <= (half_step(y.dtype) + 1e-4) * np.linalg.norm(plain)


def test_matvec_extremes(R):
    """Values near the ends of the types: a row of x far larger than its neighbours, fp32 rows near 1e30 and 1e-30, scales near fp16's
    largest and among its subnormals, codes -8."""
    n = 512
    rs = np.random.RandomState(0)
    q = rs.randint(-8, 8, (20, n))
    for scale, val in (("f16", 65504.0), ("f16", 2.0 ** -24), ("f32", 1e-20)):
        s = np.full((20, n // 128), val).astype(np.float16 if scale == "f16" else np.float32)
        p = O.pack_nibbles(q).astype(np.uint8)
        w = O.dequantize(p, s, "int4", 128, None)
        for size in (1e30, 1e-30, 1.0):
            if not 1e-33 < size * val < 1e33:         # the product itself stays a normal fp32 number
                continue
            x = torch.from_numpy(rs.randn(3, n) * np.array([[size], [size * 1e-3], [0.0]])).float()
            say("matvec extremes", scale, val, size)
            y = R.rhtq_matvec(*device_weights(p, s, None)[:2], x.cuda(), group=128, scale_dtype=scale, rotated=True)
            check_matvec(y, x.double().numpy(), w)


def test_matvec_views_and_buffers(R):
    """Rows and columns cut from larger tensors, an out of the caller's, no rows, no tokens, another stream."""
    p, s, ts, w = weights(40, 256, "int4", 32, "f16", 9)
    dp, ds, _ = device_weights(p, s, ts)
    big = torch.randn(6, 512, device="cuda", dtype=torch.bfloat16)
    x = big[::2, 128:384]
    kw = dict(group=32, scale_dtype="f16", rotated=True)
    ref = R.rhtq_matvec(dp, ds, x.contiguous(), **kw)
    assert torch.equal(R.rhtq_matvec(dp, ds, x, **kw), ref)
    assert torch.equal(R.rhtq_matvec(dp[::2], ds[::2], x, **kw), ref[:, ::2])
    out = torch.full((3, 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert R.rhtq_matvec(dp, ds, x, out=out, **kw) is out and torch.equal(out, ref)
    st = torch.cuda.Stream()
    y = R.rhtq_matvec(dp, ds, x, stream=st, **kw)
    st.synchronize()
    assert torch.equal(y, ref)
    assert R.rhtq_matvec(dp[:0], ds[:0], x, **kw).shape == (3, 0)
    assert R.rhtq_matvec(dp, ds, x[:0], **kw).shape == (0, 40)
    with pytest.raises(R.RhtqError):
        R.rhtq_matvec(dp[:, :24].contiguous(), ds[:, :1].contiguous(), x[:, :48], group=48, scale_dtype="f16", rotated=True)
    with pytest.raises(R.RhtqError):                       # no Hadamard of order 160
        R.rhtq_matvec(dp[:, :80].contiguous(), ds[:, :5].contiguous(), x[:, :160], group=32, scale_dtype="f16")


# ---------------------------------------------------------------------------------------------------------- cache

def paged(R, lens, kv, dim, page, scale, seed, spare=3, fill=True, width=None):
    """A cache with the given lengths: (cache, table, lengths) on the device; random rows everywhere if `fill`."""
    rs = np.random.RandomState(seed)
    need = [-(-x // page) for x in lens]
    pages = sum(need) + spare
    width = max(need + [1]) + 1 if width is None else width
    order, at = rs.permutation(pages), 0
    table = np.full((len(lens), width), -1, dtype=np.int32)
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    cache = R.rhtq_cache_new(pages, kv, page, dim, scale_dtype=scale)
    if fill:
        for c in (cache.k_codes, cache.v_codes):
            c.copy_(torch.from_numpy(rs.randint(0, 256, tuple(c.shape)).astype(np.uint8)))
        for s in (cache.k_scales, cache.v_scales):
            s.copy_(torch.from_numpy(np.exp(rs.randn(*s.shape)) * 0.1))
    return cache, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def host(cache):
    return [t.cpu().numpy() for t in cache]


def place(table, s, pos, page):
    t = table[s, pos // page] if 0 <= pos < table.shape[1] * page else -1
    return t, pos % page


CACHE = [(64, 1, 16, "f16", "bf16"), (128, 8, 16, "f16", "bf16"), (128, 3, 32, "f32", "f16"), (256, 2, 64, "f16", "f32"), (64, 5, 256, "f32", "f32"),
         (128, 32, 128, "f16", "f16")]


@pytest.mark.parametrize("dim,kv,page,scale,xt", CACHE)
@pytest.mark.parametrize("ragged", [False, True])
def test_cache_append_and_read(R, dim, kv, page, scale, xt, ragged):
    say("cache", dim, kv, page, scale, xt, ragged)
    rs = np.random.RandomState(dim + kv)
    old = [0, 5, page - 1, page, 3 * page + 7, 1]
    new = [1] * 6 if not ragged else [page + 3, 0, 1, 2 * page, 37, 2]
    lens = [a + b for a, b in zip(old, new)]
    cache, table, lengths = paged(R, lens, kv, dim, page, scale, seed=1)
    before = host(cache)
    tokens = sum(new)
    x = torch.from_numpy(rs.randn(tokens + 1, 2, kv, dim) * np.exp(rs.randn(tokens + 1, 2, kv, 1))).to(DT[xt])
    x[0, 0, 0] = 0                                                     # a zero row: scale and codes 0
    xd = x.cuda()
    starts = None if not ragged else torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
    extra = 1 if ragged else 0                                          # a row that belongs to no sequence
    ks, vs = signs_of(dim, 1), signs_of(dim, 2)
    R.rhtq_cache_append(cache, xd[:tokens + extra, 0], xd[:tokens + extra, 1], table, lengths, starts, ks, vs)
    after, tb = host(cache), table.cpu().numpy()
    written = set()
    rows = [(s, old[s] + i) for s in range(6) for i in range(new[s])]
    for w, sg in ((0, ks), (1, vs)):
        y = O.rotate(x[:tokens, w].double().numpy().reshape(-1, dim), sg).reshape(tokens, kv, dim)
        codes, scales = [], []
        for s, pos in rows:
            p, sl = place(tb, s, pos, page)
            written.add((p, sl))
            codes.append(after[2 * w][p, :, sl])
            scales.append(after[2 * w + 1][p, :, sl])
        codes, scales = np.stack(codes).reshape(-1, dim // 2), np.stack(scales).reshape(-1, 1)
        C.check_int4(codes, scales, y.reshape(-1, dim), 0, scale, enforce_fraction=False)
        forward = R.rhtq_forward(xd[:tokens, w].reshape(-1, dim), sg, scale_dtype=scale)
        same = (forward[0].cpu().numpy() == codes).mean()
        assert same >= 1 - 2e-3, f"{1 - same} of the bytes are not rhtq_forward's"   # only ties of a rounding may differ
    for a, b in zip(before, after):                                     # every other slot is as it was
        keep = np.ones(a.shape[:1] + a.shape[2:3], dtype=bool)
        for p, sl in written:
            keep[p, sl] = False
        a, b = np.moveaxis(a, 2, 1), np.moveaxis(b, 2, 1)
        assert np.array_equal(a[keep], b[keep])
    for out in (torch.float32, DT[xt]):
        k, v = R.rhtq_cache_read(cache, table, lengths, starts, tokens + extra, ks, vs, dtype=out)
        assert k.dtype == out and k.shape == (tokens + extra, kv, dim)
        for got, w, sg in ((k, 0, ks), (v, 1, vs)):
            c = np.stack([after[2 * w][place(tb, s, pos, page)[0], :, place(tb, s, pos, page)[1]] for s, pos in rows]).reshape(-1, dim // 2)
            sc = np.stack([after[2 * w + 1][place(tb, s, pos, page)[0], :, place(tb, s, pos, page)[1]] for s, pos in rows]).reshape(-1, 1)
            ref = O.inverse(c, sc, sg, "int4").reshape(tokens, kv, dim)
            g = got.double().cpu().numpy()
            tiny = 2.0 ** -25 if out == torch.float16 else 0.0
            # whole-number transform exact; two fp32 products, then the output's rounding
            assert (np.abs(g[:tokens] - ref) <= (half_step(out) + 3 * 2.0 ** -24) * np.abs(ref) + tiny).all()
            if extra:
                assert (g[tokens:] == 0).all()


def test_cache_rows_without_a_place(R):
    """Rows whose page is missing or outside the pool, whose position is below 0 or beyond the table: nothing is stored, zeros are read."""
    cache, table, _ = paged(R, [40, 40, 40], 2, 64, 16, "f16", 3)
    table[0, 1], table[1, 0] = 1 << 20, -7
    lengths = torch.tensor([20, 3, 4000], dtype=torch.int32, device="cuda")
    before = host(cache)
    x = torch.randn(3, 2, 64, device="cuda", dtype=torch.float16)
    say("cache rows without a place")
    R.rhtq_cache_append(cache, x, x, table, lengths)
    starts = torch.tensor([0, 0, 0, 3], dtype=torch.int32, device="cuda")
    R.rhtq_cache_append(cache, x, x, table, torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda"), starts)
    for a, b in zip(before, host(cache)):
        assert np.array_equal(a, b)
    k, v = R.rhtq_cache_read(cache, table, lengths, None, 3, dtype=torch.float32)
    assert (k == 0).all() and (v == 0).all()
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    R.rhtq_cache_append(cache, x[:0], x[:0], table[:0], none)
    k, v = R.rhtq_cache_read(cache, table, lengths, starts, 0)
    assert k.shape == (0, 2, 64)


def test_cache_strided_rows(R):
    """Keys and values inside a fused projection, heads in another order of strides, and rows that do not start on 16 bytes."""
    cache, table, lengths = paged(R, [7, 9], 4, 128, 16, "f16", 5)
    qkv = torch.randn(2, 12 * 128 + 4, device="cuda", dtype=torch.bfloat16)
    sets = [qkv[:, :1536].unflatten(1, (12, 128))[:, 4:8],
            qkv[:, 4:1540].unflatten(1, (12, 128))[:, 4:8], torch.randn(4, 2, 128, device="cuda", dtype=torch.bfloat16).transpose(0, 1),
            torch.randn(2, 128, 4, device="cuda", dtype=torch.bfloat16).transpose(1, 2)]
    for x in sets:
        R.rhtq_cache_append(cache, x, x.flip(0), table, lengths)
        got = host(cache)
        R.rhtq_cache_append(cache, x.contiguous(), x.flip(0).contiguous(), table, lengths)
        for a, b in zip(got, host(cache)):
            assert np.array_equal(a, b)


# ------------------------------------------------------------------------------------------------------ attention

def attention_ref(q, cache, table, lens, ks, vs, scale, window, sinks):
    """64-bit attention per (sequence, head), and the allowed 2-norm of each head's error besides the output's rounding."""
    kc, ksc, vc, vsc = host(cache)
    seqs, heads, dim = q.shape
    kv, page = kc.shape[1], kc.shape[2]
    each = heads // kv
    out, allowed = np.zeros(q.shape), np.zeros(q.shape[:2])
    qr = O.rotate(q.reshape(-1, dim), ks).reshape(q.shape)
    for s in range(seqs):
        n = max(0, min(int(lens[s]), table.shape[1] * page))
        pos = [p for p in range(n) if (not window or p >= n - window or p < sinks) and 0 <= table[s, p // page] < kc.shape[0]]
        if not pos:
            continue
        pg, sl = np.array([table[s, p // page] for p in pos]), np.array([p % page for p in pos])
        for h in range(kv):
            kq = O.unpack_nibbles(kc[pg, h, sl], signed=True).astype(np.float64)
            vq = O.unpack_nibbles(vc[pg, h, sl], signed=True).astype(np.float64)
            sk, sv = ksc[pg, h, sl].astype(np.float64), vsc[pg, h, sl].astype(np.float64)
            for j in range(h * each, (h + 1) * each):
                x = scale * sk * (kq @ qr[s, j])
                p = np.exp(x - x.max())
                l = p.sum()
                p = p / l
                o = (p * sv) @ vq
                out[s, j] = O.inverse_rotate(o[None], vs)[0]
                # score error: q carried to 2^-16 of its largest value, its fp32 rotation, the fp32 products and exponential
                dx = abs(scale) * sk * (2.0 ** -16 + 16 * 2.0 ** -24) * np.abs(qr[s, j]).max() * np.abs(kq).sum(1) + 2.0 ** -20 * (1 + np.abs(x))
                rel = np.expm1(2 * np.minimum(dx, 20))
                m = (p * sv).max()
                allowed[s, j] = np.linalg.norm((p * rel * sv) @ np.abs(vq)) + math.sqrt(dim) * 8 * (
                    len(pos) * 2.0 ** -16 * m + 2.0 ** -20 * (p * sv).sum())
    return out, allowed


def check_attention(o, ref, allowed):
    g = o.double().cpu().numpy()
    assert np.isfinite(g).all()
    norm = np.linalg.norm(ref, axis=-1)
    tiny = 2.0 ** -25 * math.sqrt(ref.shape[-1]) if o.dtype == torch.float16 else 0.0
    off = np.linalg.norm(g - ref, axis=-1)
    bad = ~(off <= half_step(o.dtype) * (norm + allowed) + allowed + tiny)
    assert not bad.any(), f"{bad.sum()} of {bad.size} heads off; worst {np.max(off / (half_step(o.dtype) * norm + allowed + 1e-30)):.3g} x allowed"


ATTENTION = [
    # lengths, q heads, kv heads, dim, page, scale, type, window, sinks
    ([1], 1, 1, 128, 16, "f16", "bf16", 0, 0), ([0, 1, 2, 15, 16, 17], 4, 4, 128, 16, "f16", "bf16", 0, 0),
    ([63, 64, 65, 255, 256, 257], 8, 2, 128, 32, "f32", "f16", 0, 0), ([515], 32, 32, 128, 16, "f16", "bf16", 0, 0),
    ([1023, 0, 77], 14, 2, 64, 16, "f16", "f16", 0, 0), ([130, 300], 6, 2, 256, 64, "f32", "bf16", 0, 0),
    ([4097], 8, 1, 128, 256, "f16", "bf16", 0, 0), ([900, 33], 24, 2, 128, 16, "f16", "f16", 0, 0), ([70], 40, 1, 64, 16, "f16", "bf16", 0, 0),
    ([17, 400, 1000, 0, 5], 8, 2, 128, 16, "f16", "bf16", 100, 4), ([500, 260, 16], 4, 4, 64, 32, "f32", "f16", 1, 0),
    ([500, 261, 40], 4, 1, 128, 16, "f16", "bf16", 37, 21), ([333], 9, 3, 256, 16, "f16", "f16", 64, 64), ([2000, 1], 5, 1, 128, 32, "f16", "bf16", 1999, 0),
    ([2000], 8, 8, 128, 64, "f16", "f16", 5000, 3), ([12000, 3], 16, 2, 128, 64, "f16", "bf16", 0, 0), ([9000], 2, 1, 64, 128, "f32", "f16", 0, 0),
]


@pytest.mark.parametrize("lens,heads,kv,dim,page,sd,qt,window,sinks", ATTENTION)
def test_attention(R, lens, heads, kv, dim, page, sd, qt, window, sinks):
    say("attention", lens, heads, kv, dim, page, sd, qt, window, sinks)
    cache, table, lengths = paged(R, lens, kv, dim, page, sd, seed=heads + dim)
    q = torch.from_numpy(np.random.RandomState(7).randn(len(lens), heads, dim)).to(DT[qt])
    ks, vs = signs_of(dim, 3), signs_of(dim, 4)
    o = R.rhtq_paged_attention(q.cuda(), cache, table, lengths, ks, vs, window=window, sinks=sinks)
    ref, allowed = attention_ref(q.double().numpy(), cache, table.cpu().numpy(), lens, ks, vs, 1 / math.sqrt(dim), window, sinks)
    check_attention(o, ref, allowed)
    for s, n in enumerate(lens):
        if n == 0:
            assert (o[s] == 0).all()


@pytest.mark.parametrize("peak", [0.0, 30.0, 300.0, -300.0])
def test_attention_scores_of_any_size(R, peak):
    """Flat, sharp and huge scores: the largest position last, first or in the middle; scales among fp16's subnormals and zeros."""
    say("attention scores", peak)
    dim, n = 128, 700
    cache, table, lengths = paged(R, [n], 2, dim, 16, "f16", seed=11)
    cache.k_scales.zero_()
    cache.v_scales.mul_(2.0 ** -18)
    tb = table.cpu().numpy()
    for i, pos in enumerate((0, 350, n - 1)):
        p, sl = place(tb, 0, pos, 16)
        cache.k_scales[p, :, sl] = abs(peak) * (1 + 0.01 * i)
    q = torch.from_numpy(np.random.RandomState(2).randn(1, 4, dim)).half()
    if peak < 0:
        q = -q
    o = R.rhtq_paged_attention(q.cuda(), cache, table, lengths, None, None, scale=0.05)
    ref, allowed = attention_ref(q.double().numpy(), cache, tb, [n], None, None, 0.05, 0, 0)
    check_attention(o, ref, allowed)


@pytest.mark.parametrize("size", [1e4, 1e7])
def test_attention_huge_scores_stay_finite(R, size):
    """Scores so large that neighbouring fp32 numbers are whole units apart: the largest one still has weight 1, none overflows."""
    say("attention huge scores", size)
    cache, table, lengths = paged(R, [130], 1, 128, 16, "f32", seed=13)
    cache.k_scales.fill_(size)
    q = (torch.randn(1, 4, 128, device="cuda") * 1e4).bfloat16()
    o = R.rhtq_paged_attention(q, cache, table, lengths, None, None)
    kc, ksc, vc, vsc = host(cache)
    tb = table.cpu().numpy()
    pg, sl = np.array([tb[0, p // 16] for p in range(130)]), np.arange(130) % 16
    x = O.rotate(q[0].double().cpu().numpy(), None) @ O.unpack_nibbles(kc[pg, 0, sl], signed=True).astype(np.float64).T
    top = x.argmax(1)
    gap = np.sort(x, axis=1)
    # the two largest are further apart than q's fixed point can move them
    clear = (gap[:, -1] - gap[:, -2]) > 2 * 8 * 128 * 2.0 ** -16 * np.abs(q.double().cpu().numpy()).max() * 11.4
    v = O.inverse(vc[pg, 0, sl], vsc[pg, 0, sl][:, None], None, "int4")[top]
    g = o[0].double().cpu().numpy()
    assert np.isfinite(g).all() and clear.any()
    assert np.allclose(g[clear], v[clear], rtol=2.0 ** -7, atol=2.0 ** -14 * np.abs(v).max())


@pytest.mark.parametrize("sd", ["f16", "f32"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
def test_attention_sees_nothing_of_masked_places(R, sd, window, sinks):
    """NaN, infinities and any bytes behind the last position, between the first positions and the window, and on unused pages."""
    say("attention masked places", sd, window, sinks)
    lens = [1, 15, 130, 700, 0]
    cache, table, lengths = paged(R, lens, 2, 128, 16, sd, seed=17)
    q = torch.randn(5, 8, 128, device="cuda", dtype=torch.float16)
    ref = R.rhtq_paged_attention(q, cache, table, lengths, window=window, sinks=sinks)
    tb = table.cpu().numpy()
    seen = np.zeros((cache.k_codes.shape[0], 16), dtype=bool)
    for s, n in enumerate(lens):
        for p in range(n):
            if not window or p >= n - window or p < sinks:
                seen[tb[s, p // 16], p % 16] = True
    hidden = torch.from_numpy(~seen).cuda()[:, None, :].expand(-1, 2, -1)
    for bad in (float("nan"), float("inf"), -float("inf")):
        for t in (cache.k_scales, cache.v_scales):
            t[hidden] = bad
        for t in (cache.k_codes, cache.v_codes):
            t[hidden] = 0x87
        assert torch.equal(R.rhtq_paged_attention(q, cache, table, lengths, window=window, sinks=sinks), ref)


def test_offsets_beyond_32_bits(R):
    """Pages whose bytes start beyond 4 GiB: stored, read, attended to, copied, moved."""
    say("offsets beyond 32 bits")
    pages, kv, page, dim = 34000, 4, 256, 256                 # 131 KB a page and tensor: 4.4 GB of keys
    cache = R.rhtq_cache_new(pages, kv, page, dim)
    small, _, _ = paged(R, [1], kv, dim, page, "f16", seed=1, spare=7)
    n = 300
    far = torch.tensor([[33999, 33001]], dtype=torch.int32, device="cuda")
    near = torch.tensor([[3, 5]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    x = torch.randn(2, n, kv, dim, device="cuda", dtype=torch.bfloat16)
    q = torch.randn(1, 8, dim, device="cuda", dtype=torch.bfloat16)
    out = []
    for c, t in ((cache, far), (small, near)):
        R.rhtq_cache_append(c, x[0], x[1], t, lengths, starts)
        out.append(R.rhtq_cache_read(c, t, lengths, starts, n) + (R.rhtq_paged_attention(q, c, t, lengths),))
    assert all(torch.equal(a, b) for a, b in zip(*out))
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    R.rhtq_pages_copy(cache, ints(33999, 33001), ints(33500, 40))
    t = torch.tensor([[33500, 40]], dtype=torch.int32, device="cuda")
    assert torch.equal(R.rhtq_paged_attention(q, cache, t, lengths), out[0][2])
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[far[0].long()] = 1
    assert R.rhtq_pages_compact(cache, far, refs).item() == 2
    assert sorted(far[0].tolist()) == [0, 1] and torch.equal(R.rhtq_paged_attention(q, cache, far, lengths), out[0][2])


def test_cache_without_pages(R):
    """No page, or a table without columns: rows are passed over, zeros come back."""
    say("cache without pages")
    empty = R.rhtq_cache_new(0, 2, 16, 128)
    lengths = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    x = torch.randn(2, 2, 128, device="cuda", dtype=torch.float16)
    full, table, _ = paged(R, [5, 9], 2, 128, 16, "f16", seed=2)
    for c, t in ((empty, table), (empty, table[:, :0].contiguous()), (full, table[:, :0].contiguous())):
        R.rhtq_cache_append(c, x, x, t, lengths)
        k, v = R.rhtq_cache_read(c, t, lengths, None, 2, dtype=torch.float16)
        assert (k == 0).all() and (v == 0).all()
        assert (R.rhtq_paged_attention(x, c, t, lengths) == 0).all()


def test_calls_from_many_threads(R):
    """Eight threads on streams of their own, all calls at once, against the calls one after another."""
    import threading
    say("calls from many threads")
    cache, table, lengths = paged(R, [700, 90, 33], 2, 128, 16, "f16", seed=41)
    p, s, ts, w = weights(300, 1024, "int4", 64, "f16", 5)
    dp, ds, _ = device_weights(p, s, ts)
    qs = [torch.randn(3, 8, 128, device="cuda", dtype=torch.bfloat16) for _ in range(8)]
    xs = [torch.randn(1 + 3 * i, 1024, device="cuda", dtype=torch.bfloat16) for i in range(8)]
    sg = torch.from_numpy(signs_of(1024, 3)).cuda()

    def calls(i):
        return (R.rhtq_paged_attention(qs[i], cache, table, lengths), R.rhtq_matvec(dp, ds, xs[i], sg, group=64, scale_dtype="f16"),
                R.rhtq_cache_read(cache, table, lengths, None, 3)[0])
    one = [calls(i) for i in range(8)]
    torch.cuda.synchronize()
    got, errors = [None] * 8, []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[i] = calls(i)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(one, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_attention_missing_pages(R):
    """Entries that name no page are seen by no query; a sequence with none left gets zeros.  Lengths beyond the table end with it."""
    say("attention missing pages")
    lens = [200, 90, 64, 40]
    cache, table, _ = paged(R, lens, 2, 128, 16, "f16", seed=21)
    table[0, 3], table[0, 0], table[1, :] = -1, 1 << 25, -3
    table[3, 0] = -(1 << 31)
    given = [200, 90, 4000, -5]
    lengths = torch.tensor(given, dtype=torch.int32, device="cuda")
    q = torch.randn(4, 4, 128, device="cuda", dtype=torch.bfloat16)
    for window, sinks in ((0, 0), (30, 20)):
        o = R.rhtq_paged_attention(q, cache, table, lengths, window=window, sinks=sinks)
        tb = table.cpu().numpy()
        tb[2, tb.shape[1] - 1 - (tb[2] >= 0)[::-1].argmax() + 1:] = -1
        ref, allowed = attention_ref(q.double().cpu().numpy(), cache, tb, given, None, None, 1 / math.sqrt(128), window, sinks)
        check_attention(o, ref, allowed)
        assert (o[1] == 0).all() and (o[3] == 0).all()


def test_attention_views_streams_and_buffers(R):
    cache, table, lengths = paged(R, [300, 20, 1000], 2, 128, 16, "f16", seed=31)
    qkv = torch.randn(3, 13 * 128, device="cuda", dtype=torch.bfloat16)
    q = qkv[:, 128:128 * 9].unflatten(1, (8, 128))
    ref = R.rhtq_paged_attention(q.contiguous(), cache, table, lengths)
    assert torch.equal(R.rhtq_paged_attention(q, cache, table, lengths), ref)
    assert torch.equal(R.rhtq_paged_attention(q.transpose(1, 2).contiguous().transpose(1, 2), cache, table, lengths), ref)
    out = torch.empty_like(ref)
    assert R.rhtq_paged_attention(q, cache, table, lengths, out=out) is out and torch.equal(out, ref)
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [R.rhtq_paged_attention(q, cache, table, lengths, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    again = [R.rhtq_paged_attention(q, cache, table, lengths) for _ in range(5)]
    assert all(torch.equal(o, ref) for o in again)                     # the same bits in every run
    none = R.rhtq_paged_attention(q[:0], cache, table[:0], lengths[:0])
    assert none.shape == (0, 8, 128)
    empty = R.rhtq_paged_attention(q, cache, table[:, :0].contiguous(), lengths)
    assert (empty == 0).all()


# ---------------------------------------------------------------------------------------------------------- pages

class Pool:
    """The same state on the device and as plain lists, moved on by a plain model."""

    def __init__(self, R, seqs, pages, page, width, layers=None, kv=2, dim=64, seed=0):
        rs = np.random.RandomState(seed)
        self.R, self.page = R, page
        self.cache = R.rhtq_cache_new(pages, kv, page, dim, layers=layers)
        for t in self.cache:
            t.copy_(torch.from_numpy(rs.randint(0, 200, tuple(t.shape))))
        self.table = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.t, self.n, self.r = self.table.cpu().numpy(), self.lengths.cpu().numpy(), self.refs.cpu().numpy()
        self.data = [t.cpu().numpy().copy() for t in self.cache]

    def ints(self, v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def fresh(self, count):
        return np.nonzero(self.r <= 0)[0][:count]

    def check(self):
        assert np.array_equal(self.table.cpu().numpy(), self.t)
        assert np.array_equal(self.lengths.cpu().numpy(), self.n)
        assert np.array_equal(self.refs.cpu().numpy(), self.r)
        for a, b in zip(self.cache, self.data):
            assert np.array_equal(a.cpu().numpy(), b)
        held = self.t[self.t >= 0]
        assert np.array_equal(np.bincount(held, minlength=len(self.r)), self.r)

    def reserve(self, add):
        st = self.R.rhtq_pages_reserve(self.table, self.lengths, self.refs, self.ints(add), self.page).item()
        slots, over = [], 0
        for s, a in enumerate(add):
            if a < 0:
                assert st == -1
                return st
            need = -(-(int(self.n[s]) + a) // self.page)
            over += max(0, need - self.t.shape[1])
            slots += [(s, i) for i in range(-(-int(self.n[s]) // self.page), min(need, self.t.shape[1])) if self.t[s, i] < 0]
        have = int((self.r <= 0).sum())
        assert st == over + max(0, len(slots) - have)
        if st == 0:
            for (s, i), p in zip(slots, self.fresh(len(slots))):
                self.t[s, i], self.r[p] = p, 1
            self.n += np.array(add, dtype=np.int32)
        return st

    def free(self, seqs):
        self.R.rhtq_pages_free(self.table, self.lengths, self.refs, self.ints(seqs))
        for s in set(seqs):
            if 0 <= s < len(self.n):
                for p in self.t[s]:
                    if p >= 0:
                        self.r[p] -= 1
                self.t[s], self.n[s] = -1, 0

    def fork(self, src, dst):
        st = self.R.rhtq_pages_fork(self.cache, self.table, self.lengths, self.refs, self.ints(src), self.ints(dst)).item()
        ok = all(0 <= i < len(self.n) for i in src + dst) and len(set(dst)) == len(dst) and not set(src) & set(dst) and \
            all(self.n[d] == 0 and (self.t[d] < 0).all() for d in dst)
        if not ok:
            assert st == -1
            return st
        part = [i for i, s in enumerate(src) if self.n[s] % self.page and self.t[s, self.n[s] // self.page] >= 0]
        have = int((self.r <= 0).sum())
        assert st == max(0, len(part) - have)
        if st == 0:
            new = dict(zip(part, self.fresh(len(part))))
            for i, (s, d) in enumerate(zip(src, dst)):
                full, rest = divmod(int(self.n[s]), self.page)
                self.t[d, :full] = self.t[s, :full]
                for p in self.t[s, :full]:
                    if p >= 0:
                        self.r[p] += 1
                if i in new:
                    self.t[d, full], self.r[new[i]] = new[i], 1
                    for a in self.data:
                        ax = a.ndim - (4 if a.dtype == np.uint8 else 3)
                        m = np.moveaxis(a, ax, 0)
                        slots = m.ndim - (2 if a.dtype == np.uint8 else 1)
                        np.moveaxis(m[new[i]], slots - 1, 0)[:rest] = np.moveaxis(m[self.t[s, full]], slots - 1, 0)[:rest]
                self.n[d] = self.n[s]
        return st

    def compact(self):
        live = self.R.rhtq_pages_compact(self.cache, self.table, self.refs).item()
        assert live == int((self.r > 0).sum())
        old = [p for p in range(live, len(self.r)) if self.r[p] > 0]
        new = [p for p in range(live) if self.r[p] <= 0]
        for o, w in zip(old, new):
            for a in self.data:
                m = np.moveaxis(a, a.ndim - (4 if a.dtype == np.uint8 else 3), 0)
                m[w] = m[o]
            self.t[self.t == o] = w
            self.r[w], self.r[o] = self.r[o], 0
        return live


@pytest.mark.parametrize("seqs,pages,page,width,layers", [(3, 8, 16, 4, None), (40, 300, 16, 12, 3), (70, 3000, 32, 9, 1), (1, 1, 16, 1, 2)])
def test_pages_as_they_are_used(R, seqs, pages, page, width, layers):
    say("pages", seqs, pages, page, width, layers)
    rs = np.random.RandomState(seqs)
    P = Pool(R, seqs, pages, page, width, layers)
    done = []
    for step in range(30):
        op = rs.choice(["reserve", "reserve", "free", "fork", "compact"])
        if op == "reserve":
            st = P.reserve([int(v) for v in rs.randint(0, page + 9, seqs) * (rs.rand(seqs) < 0.6)])
        elif op == "free":
            st = P.free([int(v) for v in rs.randint(-1, seqs + 1, max(1, seqs // 4))])
        elif op == "fork":
            empty = [i for i in range(seqs) if P.n[i] == 0 and (P.t[i] < 0).all()]
            full = [i for i in range(seqs) if P.n[i] > 0]
            if not empty or not full:
                continue
            dst = empty[: max(1, len(empty) // 2)]
            st = P.fork([int(rs.choice(full)) for _ in dst], dst)
        else:
            st = P.compact()
        done.append((op, st))
        P.check()
    print(done)


def test_pages_all_or_nothing(R):
    say("pages all or nothing")
    P = Pool(R, 4, 5, 16, 3, 2)
    assert P.reserve([20, 0, 16, 1]) == 0 and (P.check() or True)
    assert P.reserve([16, 0, 1, 0]) == 1 and (P.check() or True)         # two pages wanted, one free
    assert P.reserve([-1, 0, 0, 0]) == -1 and (P.check() or True)
    assert P.reserve([40, 0, 0, 0]) > 0 and (P.check() or True)          # beyond the table
    assert P.reserve([2**31 - 1] * 4) > 0 and (P.check() or True)
    assert P.fork([0], [2]) == -1 and (P.check() or True)                # not empty
    assert P.fork([0, 3], [1, 1]) == -1 and (P.check() or True)          # twice
    assert P.fork([1], [1]) == -1 and (P.check() or True)
    assert P.fork([4], [1]) == -1 and (P.check() or True)
    assert P.fork([0], [-1]) == -1 and (P.check() or True)
    assert P.fork([2], [1]) == 0 and (P.check() or True)                 # a full page: shared, none taken
    assert P.r.max() == 2
    P.free([1, 1, 7, -2])
    P.check()
    assert P.fork([0], [1]) == 0 and (P.check() or True)                 # takes the last page
    P.free([3])
    assert P.reserve([0, 0, 0, 32]) == 1 and (P.check() or True)
    assert P.fork([], []) == 0
    assert P.compact() == 4 and (P.check() or True)


def test_pages_copy_and_trim(R):
    say("pages copy and trim")
    P = Pool(R, 2, 9, 16, 6, 3)
    P.R.rhtq_pages_copy(P.cache, P.ints([0, 5, 7, -1, 3]), P.ints([2, 6, 99, 1, 3]))
    for a in P.data:
        m = np.moveaxis(a, 1, 0)
        m[2], m[6] = m[0].copy(), m[5].copy()
    P.check()
    assert P.reserve([90, 20]) == 0
    R.rhtq_pages_trim(P.table, P.lengths, P.refs, 16, window=20, sinks=4)
    for s, i in ((0, 1), (0, 2), (0, 3)):                                 # pages 1..3 hold positions 16..63 < 90 - 20
        P.r[P.t[s, i]] -= 1
        P.t[s, i] = -1
    P.check()
    R.rhtq_pages_trim(P.table, P.lengths, P.refs, 16, window=20, sinks=4)
    P.check()


# --------------------------------------------------------------------------------------------- a run of them together

def decode_parts(R, layers=2, seqs=5, kv=2, each=4, dim=128, page=16, seed=0):
    rs = np.random.RandomState(seed)
    hidden, heads = 512, kv * each
    ws = []
    for i in range(layers):
        def quant(rows, n, k):
            w = torch.from_numpy(rs.randn(rows, n) / math.sqrt(n)).to(torch.bfloat16).cuda()
            sg = signs_of(n, k)
            return R.rhtq_forward(w, sg, group=64, scale_dtype="f16")[:2] + (torch.from_numpy(sg).cuda(),)
        ws.append((quant((heads + 2 * kv) * dim, hidden, 10 + i), quant(hidden, heads * dim, 20 + i)))
    ks, vs = (torch.from_numpy(signs_of(dim, k)).cuda() for k in (1, 2))
    return ws, ks, vs, hidden, heads


def decode_step(R, ws, ks, vs, cache, table, lengths, x, heads, kv, dim, **kw):
    for i, (wqkv, wo) in enumerate(ws):
        layer = cache.layer(i)
        h = (x.float() * torch.rsqrt(x.float().square().mean(1, keepdim=True) + 1e-6)).to(x.dtype)
        qkv = R.rhtq_matvec(wqkv[0], wqkv[1], h, wqkv[2], group=64, scale_dtype="f16").unflatten(1, (heads + 2 * kv, dim))
        R.rhtq_cache_append(layer, qkv[:, heads:heads + kv], qkv[:, heads + kv:], table, lengths, None, ks, vs)
        o = R.rhtq_paged_attention(qkv[:, :heads], layer, table, lengths, ks, vs, **kw)
        x = x + R.rhtq_matvec(wo[0], wo[1], o.flatten(1), wo[2], group=64, scale_dtype="f16")
    return x


def test_decode_steps_with_forks(R):
    """Steps of a small two-layer decoder: room for the token, projection, store, attention, projection; then a fork, whose copies go on from
    the same cache, and a compaction, which changes no result."""
    say("decode steps")
    kv, dim, page, seqs = 2, 128, 16, 5
    ws, ks, vs, hidden, heads = decode_parts(R)
    cache = R.rhtq_cache_new(60, kv, page, dim, layers=2)
    table = torch.full((seqs, 8), -1, dtype=torch.int32, device="cuda")
    lengths, refs = torch.zeros(seqs, dtype=torch.int32, device="cuda"), torch.zeros(60, dtype=torch.int32, device="cuda")
    live = torch.tensor([1, 1, 1, 0, 0], dtype=torch.int32, device="cuda")
    x = torch.randn(seqs, hidden, device="cuda", dtype=torch.bfloat16)
    for step in range(21):
        assert R.rhtq_pages_reserve(table, lengths, refs, live, page).item() == 0
        x = decode_step(R, ws, ks, vs, cache, table, lengths, x, heads, kv, dim, window=17, sinks=2)
        assert torch.isfinite(x).all()
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    assert R.rhtq_pages_fork(cache, table, lengths, refs, ints(0, 2), ints(3, 4)).item() == 0
    x[3], x[4] = x[0], x[2]
    R.rhtq_pages_free(table, lengths, refs, ints(1))
    before = [t.clone() for t in (*cache, table, lengths, refs)]
    results = []
    for compacted in (False, True):
        for t, b in zip((*cache, table, lengths, refs), before):
            t.copy_(b)
        if compacted:
            n = R.rhtq_pages_compact(cache, table, refs).item()
            assert (refs[:n] > 0).all() and (refs[n:] == 0).all()
        assert R.rhtq_pages_reserve(table, lengths, refs, ints(1, 0, 1, 1, 1), page).item() == 0
        results.append(decode_step(R, ws, ks, vs, cache, table, lengths, x, heads, kv, dim))
    assert torch.equal(results[0], results[1])
    assert torch.equal(results[0][0], results[0][3]) and torch.equal(results[0][2], results[0][4])
    k, v = R.rhtq_cache_read(cache.layer(1), table, lengths, torch.cat([ints(0), lengths.cumsum(0).int()]), int(lengths.sum()), ks, vs)
    n = lengths.tolist()
    at = np.cumsum([0] + n)
    assert torch.equal(k[at[0]:at[1]], k[at[3]:at[4]]) and torch.equal(v[at[2]:at[3]], v[at[4]:at[5]])


def test_captured_steps_replay_as_eager(R):
    """A whole step captured twice into graphs of their own (first calls included), replayed in turn with eager work between."""
    say("captured steps")
    kv, dim, page, seqs = 2, 128, 16, 5
    ws, ks, vs, hidden, heads = decode_parts(R, seed=3)

    def state():
        g = torch.Generator(device="cuda").manual_seed(1)
        cache = R.rhtq_cache_new(80, kv, page, dim, layers=2)
        table = torch.full((seqs, 40), -1, dtype=torch.int32, device="cuda")
        lengths, refs = torch.zeros(seqs, dtype=torch.int32, device="cuda"), torch.zeros(80, dtype=torch.int32, device="cuda")
        add = torch.tensor([100, 0, 30, 15, 1], dtype=torch.int32, device="cuda")
        R.rhtq_pages_reserve(table, lengths, refs, add, page)
        total = int(add.sum())
        starts = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), add.cumsum(0).int()])
        for i in range(2):
            kvs = torch.randn(2, total, kv, dim, generator=g, device="cuda", dtype=torch.bfloat16)
            R.rhtq_cache_append(cache.layer(i), kvs[0], kvs[1], table, lengths, starts, ks, vs)
        return cache, table, lengths, refs, torch.randn(seqs, hidden, generator=g, device="cuda", dtype=torch.bfloat16)

    one = torch.ones(seqs, dtype=torch.int32, device="cuda")

    def step(s):
        cache, table, lengths, refs, x = s
        R.rhtq_pages_reserve(table, lengths, refs, one, page)
        x.copy_(decode_step(R, ws, ks, vs, cache, table, lengths, x, heads, kv, dim))

    eager, sets = state(), [state(), state()]
    graphs = []
    torch.cuda.synchronize()
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s)
        graphs.append(g)
    for k in range(4):
        step(eager)
        for g, s in zip(graphs, sets):
            g.replay()
        torch.cuda.synchronize()
        for s in sets:
            for a, b in zip(s[0] + s[1:], eager[0] + eager[1:]):
                assert torch.equal(a, b), f"replay {k}"
