"""GPU: calls at the edges of what the serving header allows."""
import sys

import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def say(*msg):
    print("[case]", *msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    import randomized_hadamard_rotation_amd as R
    return R


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def filled(R, pages, kv, page, dim, seed, **kw):
    """A cache of random rows."""
    rs = np.random.RandomState(seed)
    cache = R.rhtq_cache_new(pages, kv, page, dim, **kw)
    for c in (cache.k_codes, cache.v_codes):
        c.copy_(torch.from_numpy(rs.randint(0, 256, tuple(c.shape)).astype(np.uint8)))
    for s in (cache.k_scales, cache.v_scales):
        s.copy_(torch.from_numpy(0.1 + 0.2 * rs.rand(*s.shape)))
    return cache


# ------------------------------------------------------------------------------------------------------------ cache

@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_without_sequences(R, dim):
    """No sequence at all: rows belong to none, so nothing is stored and zeros are read."""
    say("rows without sequences", dim)
    cache = filled(R, 3, 2, 16, dim, 1)
    before = [t.clone() for t in cache]
    table, none = torch.zeros((0, 4), dtype=torch.int32, device="cuda"), ints()
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(5, 2, dim, device="cuda", dtype=dtype)
        R.rhtq_cache_append(cache, x, x, table, none, ints(0))
        out = [torch.full((5, 2, dim), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
        R.rhtq_cache_read(cache, table, none, ints(0), 5, dtype=dtype, k_out=out[0], v_out=out[1])
        assert all((o == 0).all() for o in out)
    assert all(torch.equal(a, b) for a, b in zip(before, cache))


# ------------------------------------------------------------------------------------------------------------ pages

def held(table, pages):
    t = table.cpu().numpy()
    return np.bincount(t[(t >= 0) & (t < pages)], minlength=pages)


@pytest.mark.parametrize("given", [64, 65, 1000, 2 ** 31 - 1])
def test_trim_keeps_what_attention_sees(R, given):
    """A length beyond the table's end counts as its end, for the window that attention takes and for the one that trim takes."""
    say("trim, length", given)
    page, window, sinks = 16, 20, 3
    cache = filled(R, 8, 2, page, 64, 3)
    table, lengths, refs = torch.tensor([[5, 2, 7, 0]], dtype=torch.int32, device="cuda"), ints(given), ints(1, 0, 1, 0, 0, 1, 0, 1)
    q = torch.randn(1, 4, 64, device="cuda", dtype=torch.float16)
    before = R.rhtq_paged_attention(q, cache, table, lengths, window=window, sinks=sinks)
    R.rhtq_pages_trim(table, lengths, refs, page, window, sinks)
    assert table.tolist() == [[5, -1, 7, 0]] and refs.tolist() == [1, 0, 0, 0, 0, 1, 0, 1]      # positions 16 .. 31 alone are behind it
    assert torch.equal(R.rhtq_paged_attention(q, cache, table, lengths, window=window, sinks=sinks), before)


@pytest.mark.parametrize("entry", [6, 7, 1 << 20, 2 ** 31 - 1, -1, -7, -2 ** 31])
def test_entries_that_name_no_page(R, entry):
    """Whatever an entry outside [0, pages) holds: reserve supplies the page, its rows are stored, and a fork's target counts as empty."""
    say("entries that name no page", entry)
    page, dim = 16, 64
    cache = filled(R, 6, 2, page, dim, 5)
    table = torch.full((3, 3), entry, dtype=torch.int32, device="cuda")
    table[0, 0] = 4
    lengths, refs = ints(16, 0, 0), ints(0, 0, 0, 0, 1, 0)
    assert R.rhtq_pages_reserve(table, lengths, refs, ints(3, 17, 0), page).item() == 0
    assert table.tolist() == [[4, 0, entry], [1, 2, entry], [entry] * 3]
    assert lengths.tolist() == [19, 17, 0] and refs.tolist() == [1, 1, 1, 0, 1, 0]
    x = torch.randn(20, 2, dim, device="cuda", dtype=torch.float16)
    starts = ints(0, 3, 20, 20)
    R.rhtq_cache_append(cache, x, x, table, lengths, starts)
    k, v = R.rhtq_cache_read(cache, table, lengths, starts, 20, dtype=torch.float16)
    # stored, not zero: a row is off by at most half a step, 1/14 of its largest rotated value, in each of 64 directions, and that value is
    # below 5 of the row's deviations: 8 * 5 / 14 of the norm's 8
    assert (k.float().norm(dim=-1) > 0.5 * x.float().norm(dim=-1)).all() and torch.equal(k, v)
    assert R.rhtq_pages_fork(cache, table, lengths, refs, ints(0), ints(2)).item() == 0
    assert table.tolist() == [[4, 0, entry], [1, 2, entry], [4, 3, -1]] and refs.tolist() == [1, 1, 1, 1, 2, 0]
    assert R.rhtq_pages_fork(cache, table, lengths, refs, ints(0), ints(1)).item() == -1       # not empty
    R.rhtq_pages_free(table, lengths, refs, ints(0, 1, 2))
    assert refs.tolist() == [0] * 6


def test_reserve_under_a_partly_filled_slot(R):
    """The page of the slot that the first new position falls into is missing: it is supplied.  A sequence that asks for nothing gets
    nothing."""
    say("reserve, partly filled slot")
    page = 16
    table = torch.tensor([[2, -1, -1, -1], [-1, -1, -1, -1], [-1, 3, -1, -1]], dtype=torch.int32, device="cuda")
    lengths, refs = ints(21, 5, 20), ints(0, 0, 1, 1, 0, 0)
    assert R.rhtq_pages_reserve(table, lengths, refs, ints(2, 0, 1), page).item() == 0
    assert table.tolist() == [[2, 0, -1, -1], [-1, -1, -1, -1], [-1, 3, -1, -1]] and lengths.tolist() == [23, 5, 21]
    assert refs.tolist() == [1, 0, 1, 1, 0, 0]
    assert R.rhtq_pages_reserve(table, lengths, refs, ints(0, 30, 0), page).item() == 0
    assert table.tolist()[1] == [1, 4, 5, -1] and lengths.tolist() == [23, 35, 21] and refs.tolist() == [1] * 6
    assert R.rhtq_pages_reserve(table, lengths, refs, ints(9, 0, 0), page).item() == 0       # up to the slot's last position
    assert R.rhtq_pages_reserve(table, lengths, refs, ints(1, 0, 0), page).item() == 1 and lengths.tolist() == [32, 35, 21]


def test_reserve_refuses_shared_pages(R):
    """A draft is taken back after a fork, so that the next position lies on a page the other sequence still reads: no room there.  Forked at
    its new length the sequence goes on, and the other one's rows stay."""
    say("reserve, shared pages")
    page, dim = 16, 64
    cache = filled(R, 9, 2, page, dim, 7)
    table = torch.full((3, 3), -1, dtype=torch.int32, device="cuda")
    lengths, refs = ints(0, 0, 0), torch.zeros(9, dtype=torch.int32, device="cuda")
    assert R.rhtq_pages_reserve(table, lengths, refs, ints(40, 0, 0), page).item() == 0
    assert R.rhtq_pages_fork(cache, table, lengths, refs, ints(0), ints(1)).item() == 0
    assert refs.tolist() == [2, 2, 1, 1] + [0] * 5
    for cut in (20, 16, 31, 0):                          # inside a shared page, at its start, at its last position, everything
        lengths[0] = cut
        state = [t.clone() for t in (table, lengths, refs)]
        assert R.rhtq_pages_reserve(table, lengths, refs, ints(1, 0, 0), page).item() == -1
        assert all(torch.equal(a, b) for a, b in zip(state, (table, lengths, refs)))
    lengths[0] = 32                                       # the third page is its own
    assert R.rhtq_pages_reserve(table, lengths, refs, ints(1, 1, 0), page).item() == 0
    lengths[0] = 20
    assert R.rhtq_pages_fork(cache, table, lengths, refs, ints(0), ints(2)).item() == 0
    R.rhtq_pages_free(table, lengths, refs, ints(0))
    assert R.rhtq_pages_reserve(table, lengths, refs, ints(0, 0, 1), page).item() == 0
    rows = [t[table[1, :2].long()].clone() for t in cache]
    x = torch.randn(3, 2, dim, device="cuda", dtype=torch.float16)
    R.rhtq_cache_append(cache, x, x, table, lengths)
    assert all(torch.equal(a, t[table[1, :2].long()]) for a, t in zip(rows, cache))
    assert lengths.tolist() == [0, 41, 21] and refs.tolist() == held(table, 9).tolist()


# ----------------------------------------------------------------------------------------------------------- matvec

def product_bound(x, w, n):
    """Allowed |error| before the output's rounding, of x as carried: 2^-22 of each value and, where it is not 0, 2^-35 of the row's largest;
    and of fp32 sums: n / 16 + 64 additions one after another."""
    carried = 2.0 ** -22 * np.abs(x) + 2.0 ** -35 * np.abs(x).max(-1, keepdims=True) * (x != 0)
    return carried @ np.abs(w).T + (n / 16 + 64) * 2.0 ** -24 * (np.abs(x) @ np.abs(w).T)


@pytest.mark.parametrize("tokens", [1, 2, 3, 7, 16, 30, 61])
@pytest.mark.parametrize("n,rows", [(32, 3), (96, 18), (512, 40), (1376, 300)])
def test_mxfp4_blocks_far_apart(R, n, rows, tokens):
    """Block scales of a row up to 2^60 apart, x zero in the larger blocks of every other token: the smaller blocks' sum is an ordinary
    number and is returned.  Some rows have scales close together, some all-zero blocks with the smallest scale, as rhtq_forward leaves
    them."""
    say("mxfp4 blocks far apart", n, rows, tokens)
    rs = np.random.RandomState(n + tokens)
    blocks = n // 32
    codes = rs.randint(0, 16, (rows, n))
    e = rs.randint(-3, 4, (rows, blocks))
    large = rs.rand(rows, blocks) < 0.3
    large[:, 1::5] = True
    distance = rs.choice([15, 22, 23, 24, 30, 60], (rows, 1))
    distance[::3] = 0
    e = e + np.where(large, distance, 0)
    if blocks > 3:
        codes.reshape(rows, blocks, 32)[:, 3], e[:, 3] = 0, -127
    p, s = O.pack_nibbles(codes).astype(np.uint8), (e + 127).astype(np.uint8)
    w = O.dequantize(p, s, "mxfp4", 32, None)
    x = rs.randn(tokens, n)
    x.reshape(tokens, blocks, 32)[::2, large.any(0)] = 0
    if large.any(0).all():
        x[::2, :5] = 1.0
    x = torch.from_numpy(x).float()
    y = R.rhtq_matvec(torch.from_numpy(p).cuda(), torch.from_numpy(s).cuda(), x.cuda(), fmt="mxfp4", rotated=True).double().cpu().numpy()
    x = x.double().numpy()
    ref = x @ w.T
    allowed = product_bound(x, w, n) * (1 + 2.0 ** -24) + 2.0 ** -24 * np.abs(ref)
    bad = ~(np.abs(y - ref) <= allowed)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.max(np.abs(y - ref) / (allowed + 1e-300)):.3g} x allowed"


@pytest.mark.parametrize("tokens", [1, 4, 9])
@pytest.mark.parametrize("size,tensor_scale", [(1e35, 1e-4), (1e37, 1e-5), (1e-34, 1e4), (1.0, 1e-30)])
def test_nvfp4_tensor_scale_keeps_the_range(R, tokens, size, tensor_scale):
    """x near the ends of fp32 with a tensor scale that brings the result back: nothing overflows or vanishes on the way."""
    say("nvfp4 tensor scale", tokens, size, tensor_scale)
    n, rows = 512, 24
    rs = np.random.RandomState(tokens)
    p = O.pack_nibbles(rs.randint(0, 16, (rows, n))).astype(np.uint8)
    s = O.e4m3_encode(np.exp(2 * rs.rand(rows, n // 16) - 1)).astype(np.uint8)
    ts = np.float32(tensor_scale)
    w = O.dequantize(p, s, "nvfp4", 16, ts)
    x = torch.from_numpy(rs.randn(tokens, n) * size).float()
    y = R.rhtq_matvec(torch.from_numpy(p).cuda(), torch.from_numpy(s).cuda(), x.cuda(), fmt="nvfp4", rotated=True,
                      tensor_scale=torch.tensor([float(ts)], device="cuda")).double().cpu().numpy()
    x = x.double().numpy()
    ref = x @ w.T
    # as above, the tensor scale's product and the output besides: 2^-24 each; results are normal fp32 numbers
    allowed = product_bound(x, w, n) * (1 + 2.0 ** -23) + 2.0 ** -23 * np.abs(ref)
    assert np.abs(ref).max() < 1e38 and (np.abs(y - ref) <= allowed).all(), f"{np.max(np.abs(y - ref) / allowed):.3g} x allowed"


@pytest.mark.parametrize("tokens", [1, 3, 5])
def test_rows_beyond_one_grid_row(R, tokens):
    """More row tiles than a grid's x takes at 512 threads each (2^27 rows)."""
    say("matvec rows", tokens)
    rows, n = 2 ** 27 + 2 ** 20 + 5, 32
    g = torch.Generator(device="cuda").manual_seed(tokens)
    p = torch.randint(0, 256, (rows, n // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.ones((rows, 1), dtype=torch.float16, device="cuda")
    x = torch.randint(-3, 4, (tokens, n), device="cuda", generator=g).to(torch.bfloat16)
    y = R.rhtq_matvec(p, s, x, scale_dtype="f16", rotated=True, out_dtype=torch.float32)
    for from_ in (0, 2 ** 26 - 40, 2 ** 27 - 40, 2 ** 27 + 77, rows - 100):
        c = O.unpack_nibbles(p[from_:from_ + 100].cpu().numpy(), signed=True).astype(np.float64)
        # whole numbers, exact in fp32
        assert np.array_equal(y[:, from_:from_ + 100].double().cpu().numpy(), x.double().cpu().numpy() @ c.T), from_
    del p, s, y
    torch.cuda.empty_cache()


def test_more_sequences_than_workgroups(R):
    """Free and trim over more sequences than a grid has workgroups, the last ones included."""
    say("more sequences than workgroups")
    seqs, pages, page = 2 ** 24 + 3, 9, 16
    table = torch.full((seqs, 2), -1, dtype=torch.int32, device="cuda")
    lengths, refs = torch.zeros(seqs, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    for i, s in enumerate((0, 2 ** 20 + 1, 2 ** 24, seqs - 1)):
        table[s, 0], table[s, 1], lengths[s] = 2 * i, 2 * i + 1, 32
    refs[:8] = 1
    R.rhtq_pages_trim(table, lengths, refs, page, window=16)
    assert refs.tolist() == [0, 1] * 4 + [0] and held(table, pages).tolist() == refs.tolist()
    every = torch.arange(seqs, dtype=torch.int32, device="cuda")
    R.rhtq_pages_free(table, lengths, refs, every)
    assert refs.tolist() == [0] * 9 and (table == -1).all() and (lengths == 0).all()


# ------------------------------------------------------------------------------------------------------------- views

def test_one_token_of_a_wider_row(R):
    """One sequence's token inside a fused projection whose rows are no multiple of 16 bytes apart, and one head alone."""
    say("one token of a wider row")
    cache = filled(R, 6, 4, 16, 128, 11)
    one = filled(R, 6, 1, 16, 128, 12)
    table, lengths = torch.tensor([[3, 1, 5]], dtype=torch.int32, device="cuda"), ints(37)
    qkv = torch.randn(2, 16 * 128 + 4, device="cuda", dtype=torch.bfloat16)[:, :2048].unflatten(1, (16, 128))[:1]
    assert qkv.stride(0) % 8
    ref = [t.clone() for t in cache]
    R.rhtq_cache_append(R.RhtqCache(*ref), qkv[:, 8:12].clone(), qkv[:, 12:].clone(), table, lengths)
    R.rhtq_cache_append(cache, qkv[:, 8:12], qkv[:, 12:], table, lengths)
    assert all(torch.equal(a, b) for a, b in zip(ref, cache))
    o = R.rhtq_paged_attention(qkv[:, :8], cache, table, lengths)
    assert torch.equal(o, R.rhtq_paged_attention(qkv[:, :8].clone(), cache, table, lengths))
    heads = torch.randn(1, 128, 2, device="cuda", dtype=torch.float16).transpose(1, 2)[:, :1]      # elements two apart
    R.rhtq_cache_append(one, heads, heads, table, lengths)
    assert torch.equal(R.rhtq_paged_attention(heads, one, table, lengths), R.rhtq_paged_attention(heads.clone(), one, table, lengths))


def test_views_that_start_anywhere(R):
    """x, weights' rows, scales and signs that begin off 16 bytes, as slices of larger buffers do."""
    say("views that start anywhere")
    n, rows = 256, 19

    def shifted(t, by):
        """The same values from element `by` of a buffer on."""
        buf = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
        buf[by:] = t.flatten()
        return buf[by:].view(t.shape)
    sg = torch.from_numpy(np.where(np.random.RandomState(1).rand(n) < 0.5, -1, 1).astype(np.int8)).cuda()
    w, x = torch.randn(rows, n, device="cuda").bfloat16(), torch.randn(3, n, device="cuda").bfloat16()
    for fmt, kw in (("int4", dict(group=32, scale_dtype="f16")), ("nvfp4", {}), ("mxfp4", {})):
        p, s, ts = R.rhtq_forward(w, sg, fmt=fmt, **kw)
        ref = R.rhtq_matvec(p, s, x, sg, fmt=fmt, tensor_scale=ts, **kw)
        got = R.rhtq_matvec(shifted(p, 1), shifted(s, 1), shifted(x, 3), shifted(sg, 5), fmt=fmt, tensor_scale=ts, **kw)
        assert torch.equal(got, ref), fmt
    a, b = (filled(R, 3, 2, 16, 128, 4) for _ in range(2))
    table, lengths, sg = torch.tensor([[2, 0], [1, -1]], dtype=torch.int32, device="cuda"), ints(20, 7), sg[:128]
    kv = torch.randn(2, 2, 128, device="cuda").half()
    R.rhtq_cache_append(a, kv, kv, table, lengths, None, sg, sg)
    R.rhtq_cache_append(b, shifted(kv, 1), shifted(kv, 9), table, lengths, None, shifted(sg, 1), shifted(sg, 2))
    assert all(torch.equal(t, u) for t, u in zip(a, b))
    for u, v in zip(R.rhtq_cache_read(a, table, lengths, None, 2, sg, sg), R.rhtq_cache_read(a, table, lengths, None, 2, shifted(sg, 3), shifted(sg, 1))):
        assert torch.equal(u, v)
    q = torch.randn(2, 4, 128, device="cuda").half()
    assert torch.equal(R.rhtq_paged_attention(shifted(q, 2), a, table, lengths, shifted(sg, 1), shifted(sg, 7)),
                       R.rhtq_paged_attention(q, a, table, lengths, sg, sg))


# ----------------------------------------------------------------------------------------------------------- numbers

@pytest.mark.parametrize("huge", [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 40])
def test_windows_beyond_32_bits(R, huge):
    """A window or a count of first positions larger than any sequence leaves everything visible."""
    say("windows beyond 32 bits", huge)
    cache = filled(R, 8, 1, 16, 64, 9)
    table, lengths, refs = torch.tensor([[4, 7, 1, 2]], dtype=torch.int32, device="cuda"), ints(60), ints(0, 1, 1, 0, 1, 0, 0, 1)
    q = torch.randn(1, 2, 64, device="cuda", dtype=torch.float16)
    every = R.rhtq_paged_attention(q, cache, table, lengths)
    assert torch.equal(R.rhtq_paged_attention(q, cache, table, lengths, window=huge), every)
    assert torch.equal(R.rhtq_paged_attention(q, cache, table, lengths, window=5, sinks=huge), every)
    R.rhtq_pages_trim(table, lengths, refs, 16, window=huge)
    R.rhtq_pages_trim(table, lengths, refs, 16, window=5, sinks=huge)
    assert table.tolist() == [[4, 7, 1, 2]] and refs.tolist() == [0, 1, 1, 0, 1, 0, 0, 1]
    with pytest.raises(R.RhtqError):
        R.rhtq_pages_trim(table, lengths, refs, 2 ** 32 + 16, window=5)
    with pytest.raises(R.RhtqError):
        R.rhtq_pages_trim(table, lengths, refs, 16, window=-2 ** 32 + 5)
    with pytest.raises(R.RhtqError):
        R.rhtq_pages_reserve(table, lengths, refs, ints(1), 2 ** 32 + 16)


@pytest.mark.parametrize("tokens", [1, 2, 3, 9, 61])
@pytest.mark.parametrize("fmt,group", [("int4", 64), ("nvfp4", 16), ("mxfp4", 32)])
def test_products_with_what_is_not_finite(R, fmt, group, tokens):
    """A rotated value that is not finite gives NaN for its token, and for no other."""
    say("matvec, not finite", fmt, tokens)
    w = torch.randn(40, 512, device="cuda").bfloat16()
    p, s, ts = R.rhtq_forward(w, None, fmt=fmt, group=group)
    x = torch.randn(tokens, 512, device="cuda")
    kw = dict(fmt=fmt, group=group, tensor_scale=ts, rotated=True)
    ref = R.rhtq_matvec(p, s, x, **kw)
    for bad, t, k in ((float("nan"), 0, 0), (float("inf"), tokens - 1, 511), (-float("inf"), tokens // 2, 100)):
        b = x.clone()
        b[t, k] = bad
        y = R.rhtq_matvec(p, s, b, **kw)
        assert torch.isnan(y[t]).all()
        y[t] = ref[t]
        assert torch.equal(y, ref)


def test_page_calls_without_sequences(R):
    """No sequence: nothing to do, and the calls say so."""
    say("page calls without sequences")
    cache = filled(R, 5, 2, 16, 64, 8)
    before = [t.clone() for t in cache]
    table, none, refs = torch.zeros((0, 3), dtype=torch.int32, device="cuda"), ints(), ints(0, 0, 2, 0, 0)
    assert R.rhtq_pages_reserve(table, none, refs, none, 16).item() == 0
    assert R.rhtq_pages_fork(cache, table, none, refs, none, none).item() == 0
    R.rhtq_pages_free(table, none, refs, ints(0, 1))
    R.rhtq_pages_trim(table, none, refs, 16, 4)
    assert refs.tolist() == [0, 0, 2, 0, 0] and all(torch.equal(a, b) for a, b in zip(before, cache))
    assert R.rhtq_pages_compact(cache, table, refs).item() == 1 and refs.tolist() == [2, 0, 0, 0, 0]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("sd", ["f16", "f32"])
def test_rows_that_are_not_finite(R, dim, dtype, sd):
    """A NaN or an infinity anywhere in a row: the row's scale is NaN, and it is read as NaN; the other rows are as they were."""
    say("rows that are not finite", dim, dtype, sd)
    x = torch.randn(40, 2, dim, device="cuda").to(dtype)
    table, lengths, starts = torch.tensor([[3, 0, 5]], dtype=torch.int32, device="cuda"), ints(40), ints(0, 40)
    good, bad = (filled(R, 6, 2, 16, dim, 6, scale_dtype=sd) for _ in range(2))
    R.rhtq_cache_append(good, x, x, table, lengths, starts)
    broken = x.clone()
    rows = [(0, 0, 0, float("nan")), (17, 1, dim - 1, float("inf")), (39, 0, dim // 2 + 3, -float("inf")), (39, 1, 5, float("nan"))]
    for t, h, e, value in rows:
        broken[t, h, e] = value
    R.rhtq_cache_append(bad, broken, x, table, lengths, starts)
    k, v = R.rhtq_cache_read(bad, table, lengths, starts, 40, dtype=dtype)
    ref = R.rhtq_cache_read(good, table, lengths, starts, 40, dtype=dtype)
    for t, h, _, _ in rows:
        assert torch.isnan(k[t, h]).all(), (t, h)
        k[t, h] = ref[0][t, h]
    assert torch.equal(k, ref[0]) and torch.equal(v, ref[1])


def test_lengths_near_31_bits(R):
    """The longest sequence there can be, every page of it the same one but for the last: attention, with and without a window, is that of
    a few pages; rows are stored and read at its end."""
    say("lengths near 31 bits")
    page, dim, width = 256, 64, 2 ** 23 - 1               # 2^31 - 256 positions
    cache = filled(R, 5, 1, page, dim, 14)
    table = torch.full((1, width), 3, dtype=torch.int32, device="cuda")
    n = width * page
    lengths = torch.tensor([n], dtype=torch.int64).to(torch.int32).cuda()
    with pytest.raises(R.RhtqError):                      # width * page = 2^31 - 256 is one too many
        R.rhtq_paged_attention(torch.zeros(1, 2, dim, device="cuda", dtype=torch.bfloat16), cache, table, lengths)
    table, n = table[:, :-1].contiguous(), n - page
    lengths = ints(n)
    q = torch.randn(1, 2, dim, device="cuda", dtype=torch.bfloat16)
    one = torch.tensor([[3]], dtype=torch.int32, device="cuda")
    o, ref = R.rhtq_paged_attention(q, cache, table, lengths).float(), R.rhtq_paged_attention(q, cache, one, ints(page)).float()
    # a wave adds up 4096 equal chunks in fp32: 2^-12 of the result's size before the rounding of both to bf16
    assert ((o - ref).abs() <= 2.0 ** -7 * ref.abs() + 2.0 ** -10 * ref.norm(dim=-1, keepdim=True)).all()
    table[0, -1] = 1
    x = torch.randn(2, 1, 1, dim, device="cuda", dtype=torch.bfloat16)
    R.rhtq_cache_append(cache, x[0], x[1], table, lengths)
    near = torch.tensor([[3, 3, 1]], dtype=torch.int32, device="cuda")
    for got, want in zip(R.rhtq_cache_read(cache, table, lengths, None, 1), R.rhtq_cache_read(cache, near, ints(3 * page), None, 1)):
        assert (got != 0).any() and torch.equal(got, want)
    for window, sinks in ((300, 0), (17, 40), (513, 256)):
        o = R.rhtq_paged_attention(q, cache, table, lengths, window=window, sinks=sinks)
        few = torch.tensor([[3, 3, 3, 3, 1]], dtype=torch.int32, device="cuda")
        want = R.rhtq_paged_attention(q, cache, few, ints(5 * page), window=window, sinks=sinks)
        # the same positions in other chunks: one bf16 step at most, and 2^-14 where a value cancels to next to nothing
        assert ((o - want).float().abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -14).all(), (window, sinks)


def test_most_sequences_of_a_query_call(R):
    say("65535 sequences")
    cache = filled(R, 4, 1, 16, 64, 15)
    seqs = 65535
    table = torch.randint(0, 4, (seqs, 1), dtype=torch.int32, device="cuda")
    lengths = torch.randint(0, 17, (seqs,), dtype=torch.int32, device="cuda")
    q = torch.randn(3, 64, device="cuda", dtype=torch.float16).expand(seqs, 3, 64)
    o = R.rhtq_paged_attention(q, cache, table, lengths)
    t, n = (torch.arange(68, device="cuda") // 17).int(), (torch.arange(68, device="cuda") % 17).int()
    every = R.rhtq_paged_attention(q[:68], cache, t[:, None].contiguous(), n)
    assert torch.equal(o, every[(table[:, 0] * 17 + lengths).long()])
    with pytest.raises(R.RhtqError):
        R.rhtq_paged_attention(q[:1].expand(seqs + 1, 3, 64), cache, table[:1].expand(seqs + 1, 1).contiguous(), lengths[:1].expand(seqs + 1).contiguous())


@pytest.mark.parametrize("tokens", [1, 4, 9])
@pytest.mark.parametrize("fmt,group", [("int4", 0), ("nvfp4", 16), ("mxfp4", 32)])
def test_widest_rows(R, fmt, group, tokens):
    """n = 2^20, taken rotated."""
    say("widest rows", fmt, tokens)
    n, rows = 2 ** 20, 3
    rs = np.random.RandomState(tokens)
    p = O.pack_nibbles(rs.randint(0, 16, (rows, n))).astype(np.uint8)
    ts = np.float32(0.5) if fmt == "nvfp4" else None
    s = {"int4": lambda: np.array([[0.5], [2.0], [0.125]], dtype=np.float32), "nvfp4": lambda: O.e4m3_encode(1 + rs.rand(rows, n // 16)).astype(np.uint8),
         "mxfp4": lambda: rs.randint(120, 132, (rows, n // 32)).astype(np.uint8)}[fmt]()
    w = O.dequantize(p, s, fmt, group, ts)
    x = torch.from_numpy(rs.randn(tokens, n)).float()
    y = R.rhtq_matvec(torch.from_numpy(p).cuda(), torch.from_numpy(s).cuda(), x.cuda(), fmt=fmt, rotated=True,
                      tensor_scale=None if ts is None else torch.tensor([float(ts)], device="cuda")).double().cpu().numpy()
    x = x.double().numpy()
    ref = x @ w.T
    allowed = product_bound(x, w, n) * (1 + 2.0 ** -23) + 2.0 ** -23 * np.abs(ref)
    # that bound grows with n; the roundings of up to 2^13 steps add up as a random walk does: 2^-24 * 2^6.5, with a factor of 3 for chance
    assert (np.abs(y - ref) <= allowed).all() and np.linalg.norm(y - ref) <= 2.0 ** -16 * np.linalg.norm(ref)
