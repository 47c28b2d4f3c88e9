"""Paged attention on 4-bit rows in 64 bits, with a bound on what fp32 arithmetic may add; shared by the GPU tests and the CPU test that
the bound notices lost positions."""
import math

import numpy as np

import oracle as O

STEP = 2.0 ** -24          # half a step of fp32, relative
FIXED = 2.0 ** -22         # q and the weights as whole numbers of 22 bits: half a step, relative to the largest


def make(lens, kv, dim, page, scale, seed, spare=3):
    """(k codes, k scales, v codes, v scales, table) of random rows, as numpy arrays in the cache's layout."""
    rs = np.random.RandomState(seed)
    need = [-(-x // page) for x in lens]
    pages = sum(need) + spare
    order, at = rs.permutation(pages), 0
    table = np.full((len(lens), max(need + [1]) + 1), -1, dtype=np.int32)
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    codes = [rs.randint(0, 256, (pages, kv, page, dim // 2)).astype(np.uint8) for _ in range(2)]
    # scores of about 1, so that no position outweighs the others
    scales = [(0.1 + 0.2 * rs.rand(pages, kv, page)).astype(np.float16 if scale == "f16" else np.float32) for _ in range(2)]
    return codes[0], scales[0], codes[1], scales[1], table


def seen_positions(n, table_row, page, pages, window, sinks):
    n = max(0, min(int(n), len(table_row) * page))
    return [p for p in range(n) if (not window or p >= n - window or p < sinks) and 0 <= table_row[p // page] < pages]


def rows_of(codes, scales, table_row, head, pos, page):
    pos = np.asarray(pos)
    pg, sl = table_row[pos // page], pos % page
    return O.unpack_nibbles(codes[pg, head, sl], signed=True).astype(np.float64), scales[pg, head, sl].astype(np.float64)


def head_output(qr, k, sk, v, sv, scale):
    """(rotated output, bound on its 2-norm's error before the output's rounding) of one head's rotated q."""
    n, dim = k.shape
    x = scale * sk * (k @ qr)
    p = np.exp(x - x.max())
    p /= p.sum()
    out = (p * sv) @ v
    # q: the rotation's log2(dim) stages in fp32, then the fixed point; the score's products and sums; exp
    dq = math.log2(dim) * STEP * np.linalg.norm(qr) + math.sqrt(dim) * FIXED * np.abs(qr).max()
    dx = abs(scale) * sk * np.linalg.norm(k, axis=1) * dq + STEP * (8 * np.abs(x) + np.abs(x - x.max())) + 4 * STEP
    size = p * sv * np.linalg.norm(v, axis=1)
    sums = 2 * n / 64 + 64             # additions one after another: a lane's weights, chunks, waves, parts
    bound = 2 * (np.expm1(dx) * size).sum() + FIXED * (p * sv).max() * np.linalg.norm(v, axis=1).sum() + sums * STEP * size.sum()
    return out, bound + 16 * STEP * np.linalg.norm(out)


def reference(q, cache, lens, k_signs, v_signs, scale, window=0, sinks=0, hidden=()):
    """(outputs, bounds [seqs][heads]) in 64 bits; `hidden` positions are left out (for the test of the bound)."""
    kc, ks, vc, vs, table = cache
    seqs, heads, dim = q.shape
    pages, kv, page = kc.shape[:3]
    each = heads // kv
    out, bound = np.zeros(q.shape), np.zeros((seqs, heads))
    qr = O.rotate(q.reshape(-1, dim), k_signs).reshape(q.shape)
    for s in range(seqs):
        pos = [p for p in seen_positions(lens[s], table[s], page, pages, window, sinks) if p not in hidden]
        if not pos:
            continue
        for h in range(kv):
            k, sk = rows_of(kc, ks, table[s], h, pos, page)
            v, sv = rows_of(vc, vs, table[s], h, pos, page)
            for j in range(h * each, (h + 1) * each):
                o, bound[s, j] = head_output(qr[s, j], k, sk, v, sv, scale)
                out[s, j] = O.inverse_rotate(o[None], v_signs)[0]
    return out, bound


def off(got, ref, bound, half_step, subnormal=0.0):
    """Which heads are further off than the bound and one rounding of each value allow, value by value and as a whole."""
    d = np.abs(got - ref)
    each = (d > half_step * (np.abs(ref) + bound[..., None]) + bound[..., None] + subnormal).any(-1)
    norm = np.linalg.norm(d, axis=-1) > half_step * (np.linalg.norm(ref, axis=-1) + bound) + bound + subnormal * math.sqrt(ref.shape[-1])
    return each | norm | ~np.isfinite(got).all(-1)


# lengths, q heads, kv heads, dim, page, scale type, q type, window, sinks: several chunks, waves and parts, and the join
LONG = [
    ([515], 4, 4, 128, 16, "f16", "bf16", 0, 0), ([2000], 8, 2, 64, 16, "f16", "f16", 0, 0), ([4097], 4, 1, 128, 256, "f16", "bf16", 0, 0),
    ([9000], 2, 1, 64, 128, "f32", "f16", 0, 0), ([12000, 3], 4, 2, 128, 64, "f16", "bf16", 0, 0), ([6000], 5, 1, 256, 16, "f32", "f16", 0, 0),
    ([20000], 2, 1, 128, 32, "f16", "f16", 5000, 40),
]
