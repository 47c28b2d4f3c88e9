"""GPU: products of rows quantised on both sides and the norm in front of them, against plain 64-bit forms."""
import math

import pytest
import torch

import products_model as M
import randomized_hadamard_rotation_amd as R

pytestmark = pytest.mark.gpu
OUT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def to_rows(rows, fmt, group=0):
    return R.RhtqRows(*(None if t is None else t.cuda() for t in rows), fmt=fmt, group=group)


def expect(y, av, wv, out, extra=0.0):
    """y against av @ wv.T: half a step of its type, and fp32 sums of n products, each sum and scaling off by 2^-24 of what it has summed up
    to, which the sum of magnitudes bounds.  Products of one instruction are summed in an order of its own, so n + 8 roundings bound it."""
    want, mags = av @ wv.transpose(-1, -2), av.abs() @ wv.abs().transpose(-1, -2)
    step = {"bf16": 2.0 ** -9, "f16": 2.0 ** -12, "f32": 2.0 ** -25}[out] * 2           # eps / 2
    least = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -149}[out]
    bound = step * want.abs() + (1 + step) * mags * (av.shape[-1] + 8) * 2.0 ** -24 + least + 2.0 ** -126 + extra
    got = y.double().cpu()
    assert got.shape == want.shape
    bad = (got - want).abs() > bound
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / bound).max()), torch.nonzero(bad)[:4].tolist())


PAIRS = [("int4", 0, "int4", 0, "f32"), ("int4", 0, "int4", 128, "f16"), ("int4", 128, "int4", 0, "f16"), ("int4", 128, "int4", 256, "f32"),
         ("int4", 64, "int4", 128, "f16"), ("int4", 0, "int4", 32, "f32"), ("int4", 16, "int4", 64, "f16"), ("int8", 0, "int4", 0, "f32"),
         ("int8", 0, "int4", 128, "f16"), ("int8", 128, "int4", 128, "f32"), ("int8", 0, "int4", 64, "f32"), ("int8", 32, "int4", 0, "f16"),
         ("int8", 16, "int4", 16, "f32"), ("nvfp4", 16, "nvfp4", 16, "e4m3"), ("mxfp4", 32, "mxfp4", 32, "e8m0"),
         ("mxfp8", 32, "mxfp4", 32, "e8m0")]


def fits(n, *groups):
    return all(g == 0 or n % g == 0 for g in groups)


@pytest.mark.parametrize("pair", PAIRS, ids=lambda p: "-".join(map(str, p)))
@pytest.mark.parametrize("tokens,n,rows", [(1, 256, 16), (3, 512, 33), (17, 768, 100), (33, 256, 20), (50, 1280, 64), (65, 256, 130), (130, 512, 127),
                                           (200, 1024, 260)])
def test_product(pair, tokens, n, rows):
    a, ag, w, wg, scale = pair
    g = gen(tokens * n + rows)
    ra, rw = M.random_rows((tokens, n), a, ag, scale, g), M.random_rows((rows, n), w, wg, scale, g)
    av, wv = M.values(*ra, a), M.values(*rw, w)
    for out in ("f32", "bf16"):
        y = R.rhtq_matmul(to_rows(ra, a, ag), to_rows(rw, w, wg), out_dtype=OUT[out])
        expect(y, av, wv, out)


@pytest.mark.parametrize("pair", [p for p in PAIRS if p[1] <= 32 and p[3] <= 32], ids=lambda p: "-".join(map(str, p)))
@pytest.mark.parametrize("n", [32, 64, 96, 160, 224, 1088])
@pytest.mark.parametrize("tokens", [5, 40, 70])
def test_product_ends_inside_a_step(pair, n, tokens):
    a, ag, w, wg, scale = pair
    g = gen(n + tokens)
    ra, rw = M.random_rows((tokens, n), a, ag, scale, g), M.random_rows((37, n), w, wg, scale, g)
    y = R.rhtq_matmul(to_rows(ra, a, ag), to_rows(rw, w, wg), out_dtype=torch.float32)
    expect(y, M.values(*ra, a), M.values(*rw, w), "f32")


@pytest.mark.parametrize("fmt", ["int4", "nvfp4", "mxfp4"])
def test_product_large_tiles(fmt):
    """Enough tiles of 256 x 256 for the kernel that takes them; the first and last rows and columns are compared."""
    tokens, rows, n = 4100, 4104, 384
    group = 128 if fmt == "int4" else 0
    g = gen(1)
    ra, rw = M.random_rows((tokens, n), fmt, group, "f16", g), M.random_rows((rows, n), fmt, group, "f16", g)
    y = R.rhtq_matmul(to_rows(ra, fmt, group), to_rows(rw, fmt, group), out_dtype=torch.float16 if fmt != "nvfp4" else torch.bfloat16)
    av, wv = M.values(*ra, fmt), M.values(*rw, fmt)
    pick = torch.cat([torch.arange(0, 260), torch.arange(2000, 2100), torch.arange(tokens - 260, tokens)])
    cols = torch.cat([torch.arange(0, 260), torch.arange(rows - 260, rows)])
    expect(y.cpu()[pick][:, cols], av[pick], wv[cols], "f16" if fmt != "nvfp4" else "bf16")


def test_whole_sums_do_not_overflow():
    """INT8 x INT4, every product the largest: 127 * 8 * n, at the longest row that is summed in whole numbers and beyond."""
    for n in (65536, 65664, 1 << 20):
        ra = (torch.full((2, n), -128, dtype=torch.int8), torch.ones(2, 1), None)
        rw = (torch.full((16, n // 2), 0x88, dtype=torch.uint8), torch.ones(16, 1), None)
        y = R.rhtq_matmul(to_rows(ra, "int8"), to_rows(rw, "int4"), out_dtype=torch.float32)
        assert (y == 1024.0 * n).all()


def starts_of(lengths):
    return torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32)


def grouped_model(av, wv, starts, index, old):
    y = old.double().clone()
    for e in range(wv.shape[0]):
        for i in range(int(starts[e]), int(starts[e + 1])):
            j = i if index is None else int(index[i])
            y[i] = wv[e] @ av[j] if 0 <= j < av.shape[0] else 0.0
    return y


@pytest.mark.parametrize("pair", PAIRS, ids=lambda p: "-".join(map(str, p)))
@pytest.mark.parametrize("lengths,rows", [([3, 0, 1, 7], 40), ([0, 30, 0, 2], 17), ([70, 1, 0, 40], 24), ([0, 0, 0, 300], 130), ([128, 256, 1, 129], 20)])
def test_grouped(pair, lengths, rows):
    a, ag, w, wg, scale = pair
    n, experts = 256, len(lengths)
    total = sum(lengths)
    tokens = total + 3                                   # three rows of y belong to nobody
    g = gen(total)
    a_rows = max(2, total // 2)
    ra, rw = M.random_rows((a_rows, n), a, ag, scale, g), M.random_rows((experts, rows, n), w, wg, scale, g)
    index = torch.randint(0, a_rows, (tokens,), generator=g, dtype=torch.int32)
    index[0], index[total // 2] = -1, a_rows             # no rows
    starts = starts_of(lengths)
    out = torch.full((tokens, rows), 7.0, device="cuda")
    y = R.rhtq_grouped_matmul(to_rows(ra, a, ag), to_rows(rw, w, wg), starts.cuda(), index.cuda(), out=out)
    assert y is out
    av, wv = M.values(*ra, a), M.values(*rw, w)
    want = grouped_model(av, wv, starts, index, torch.full((tokens, rows), 7.0))
    mags = grouped_model(av.abs(), wv.abs(), starts, index, torch.zeros(tokens, rows))
    got = y.double().cpu()
    assert ((got - want).abs() <= mags * (n + 8) * 2.0 ** -23 + 2.0 ** -126).all()
    assert (got[total:] == 7.0).all() and (got[0] == 0).all() and (got[total // 2] == 0).all()


def test_grouped_many_experts_without_index():
    """300 experts: the search for a tile's expert goes over several chunks of 64."""
    g = gen(5)
    lengths = [int(v) for v in torch.randint(0, 4, (300,), generator=g)]
    total, n, rows = sum(lengths), 128, 16
    ra, rw = M.random_rows((total, n), "mxfp4", 0, "", g), M.random_rows((300, rows, n), "mxfp4", 0, "", g)
    starts = starts_of(lengths)
    y = R.rhtq_grouped_matmul(to_rows(ra, "mxfp4"), to_rows(rw, "mxfp4"), starts.cuda(), out_dtype=torch.float32)
    av, wv = M.values(*ra, "mxfp4"), M.values(*rw, "mxfp4")
    want = grouped_model(av, wv, starts, None, torch.zeros(total, rows))
    mags = grouped_model(av.abs(), wv.abs(), starts, None, torch.zeros(total, rows))
    assert ((y.double().cpu() - want).abs() <= mags * (n + 8) * 2.0 ** -23 + 2.0 ** -126).all()


def test_grouped_starts_out_of_range():
    """Starts outside [0, tokens], or falling: nothing outside y is touched, the experts that lie inside are right."""
    n, rows = 128, 16
    g = gen(6)
    ra, rw = M.random_rows((8, n), "int4", 0, "f32", g), M.random_rows((3, rows, n), "int4", 0, "f32", g)
    starts = torch.tensor([-5, 4, 6, 1 << 30], dtype=torch.int32)
    y = R.rhtq_grouped_matmul(to_rows(ra, "int4"), to_rows(rw, "int4"), starts.cuda(), out_dtype=torch.float32)
    av, wv = M.values(*ra, "int4"), M.values(*rw, "int4")
    want = grouped_model(av, wv, [0, 4, 6, 8], None, torch.zeros(8, rows))
    mags = grouped_model(av.abs(), wv.abs(), [0, 4, 6, 8], None, torch.zeros(8, rows))
    assert ((y.double().cpu() - want).abs() <= mags * (n + 8) * 2.0 ** -23).all()
    out = torch.full((8, rows), 3.0, device="cuda")
    R.rhtq_grouped_matmul(to_rows(ra, "int4"), to_rows(rw, "int4"), torch.tensor([8, 2, 2, 2], dtype=torch.int32).cuda(), out=out)
    assert (out == 3.0).all()


# ------------------------------------------------------------------------------------------------------------------- the norm

NORMS = [("int8", 0, "f32"), ("int8", 128, "f16"), ("int8", 32, "f32"), ("mxfp8", 32, "e8m0"), ("int4", 0, "f16"), ("int4", 64, "f32"),
         ("int4", 16, "f16"), ("mxfp4", 32, "e8m0"), ("nvfp4", 16, "e4m3")]


def norm_case(tokens, n, dtype, g):
    x = torch.randn(tokens, n, generator=g) * torch.exp(0.5 * torch.randn(n, generator=g))
    return x.to(OUT[dtype])


def check_rows(rows, y, fmt, group, scale, off):
    """Codes and scales against y in 64 bits, whose fp32 form may be off by `off` (absolute): each scale is that of a y that near, each value
    the nearest of its format or off by no more than `off` from where its neighbour takes over."""
    tensor = rows.tensor_scale.cpu() if rows.tensor_scale is not None else None
    codes, scales = rows.codes.cpu(), rows.scales.cpu()
    want = M.group_scales(y, fmt, group, tensor)
    each = y.shape[-1] // scales.shape[-1]
    got = M.scale_values(scales, fmt, tensor)
    off_group = off.reshape(*off.shape[:-1], -1, each).amax(-1)
    if fmt in ("int4", "int8"):
        steps = 2.0 ** -11 if scale == "f16" else 2.0 ** -22
        least = 2.0 ** -25 if scale == "f16" else 0.0
        assert ((got - want).abs() <= want * steps + off_group + least).all()
    elif fmt == "nvfp4":
        byte = got / tensor.double()
        assert ((byte - want).abs() <= (want * 2.0 ** -4).clamp(min=2.0 ** -10) * (1 + 2.0 ** -20) + off_group / (6 * tensor.double())).all()
    else:
        emax = 2 if fmt == "mxfp4" else 8
        lo, hi = torch.floor(torch.log2(want - off_group)) - emax, torch.floor(torch.log2(want + off_group)) - emax
        e = torch.log2(got)
        assert ((e >= lo) & (e <= hi)).all()
    v, s = M.unpack(codes, fmt), got.repeat_interleave(each, -1)
    most = {"int4": 7.0, "int8": 127.0, "mxfp8": 448.0}.get(fmt, 6.0)
    low = -most - 1 if fmt in ("int4", "int8") else -most
    z = torch.where(s > 0, y / torch.where(s > 0, s, 1.0), 0.0).clamp(low, most)
    # distance to the nearest code, and what the fp32 value (and its division) may be off
    if fmt in ("int4", "int8"):
        half = torch.full_like(z, 0.5)
    elif fmt == "mxfp8":
        half = 2.0 ** (torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 4)
    else:
        half = torch.where(z.abs() < 2, 0.25, torch.where(z.abs() < 4, 0.5, 1.0)).double()
    slack = torch.where(s > 0, off / torch.where(s > 0, s, 1.0), 0.0) + z.abs() * 2.0 ** -21
    assert ((v - z).abs() <= half + slack).all(), float(((v - z).abs() - half - slack).max())


@pytest.mark.parametrize("fmt,group,scale", NORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,n,block,parts", [(1, 128, 0, "rw"), (5, 512, 512, "r"), (3, 1024, 1024, "w"), (2, 4096, 4096, "rw"), (3, 4096, 128, ""),
                                                  (2, 1408, 128, "rw"), (2, 5504, 0, "r"), (2, 8192, 8192, "rw"), (2, 16384, 16384, "r"),
                                                  (1, 24576, 2048, "w"), (1, 32768, 32768, "rw"), (3, 2048, 256, "r")])
def test_norm(fmt, group, scale, dtype, tokens, n, block, parts):
    g = gen(n + block)
    x = norm_case(tokens, n, dtype, g)
    residual = norm_case(tokens, n, dtype, g) if "r" in parts else None
    weight = (1 + 0.2 * torch.randn(n, generator=g)).to(x.dtype) if "w" in parts else None
    signs = (torch.randint(0, 2, (n,), generator=g) * 2 - 1).to(torch.int8) if block else None
    ts = torch.tensor([0.01]) if fmt == "nvfp4" else None
    up = lambda t: None if t is None else t.cuda()  # noqa: E731
    rows, h = R.rhtq_norm_forward(up(x), up(weight), up(residual), 1e-5, up(signs), block, fmt, group, scale, up(ts))
    y, h64 = M.normed(x, weight, residual, 1e-5, signs, block)
    if residual is None:
        assert h is None
    else:
        assert torch.equal(h.cpu(), h64)
    # y in fp32: the mean of squares is off by its roundings (at most n / 32 + 20 sums one after the other in any place), halved by the root; six more
    # roundings; a rotation adds a rounding a stage to values as large as the block's root mean square times the square root of its size
    rel = (n / 32 + 20) * 2.0 ** -25 + 6 * 2.0 ** -24
    off = y.abs() * rel
    if block:
        size = (y.reshape(tokens, -1, block).square().mean(-1, keepdim=True).sqrt() * math.sqrt(block)).expand(-1, -1, block).reshape(y.shape)
        off = size * math.log2(block) * 2.0 ** -24 + y.abs() * rel
    check_rows(rows, y, fmt, group, scale, off)


def test_norm_in_place_and_rows_of_zeros():
    g = gen(3)
    x = norm_case(4, 256, "bf16", g).cuda()
    x[1] = 0
    res = norm_case(4, 256, "bf16", g).cuda()
    res[1] = 0
    want, h = R.rhtq_norm_forward(x, None, res.clone())
    rows, h2 = R.rhtq_norm_forward(x, None, res, residual_out=res)
    assert h2 is res and torch.equal(h, res) and torch.equal(rows.codes, want.codes) and torch.equal(rows.scales, want.scales)
    assert (rows.codes[1] == 0).all() and (rows.scales[1] == 0).all()
    for fmt in ("mxfp8", "mxfp4", "int4"):
        rows, _ = R.rhtq_norm_forward(x, None, res, fmt=fmt)
        assert (rows.codes[1] == 0).all() and (rows.scales[1] == 0).all()
    ts = torch.tensor([0.01], device="cuda")
    rows, _ = R.rhtq_norm_forward(x, None, res, fmt="nvfp4", tensor_scale=ts)
    assert (rows.codes[1] == 0).all() and (rows.scales[1] == 0).all()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("fmt,w", [("int8", "int4"), ("int4", "int4"), ("mxfp8", "mxfp4"), ("mxfp4", "mxfp4"), ("nvfp4", "nvfp4")])
def test_what_is_not_finite_shows(bad, fmt, w):
    """A row with such a value gets NaN scales, and its products are NaN; the others stay as they are."""
    g = gen(4)
    x = norm_case(3, 256, "f32", g)
    x[1, 17] = bad
    ts = torch.tensor([0.01], device="cuda") if fmt == "nvfp4" else None
    rows, _ = R.rhtq_norm_forward(x.cuda(), fmt=fmt, tensor_scale=ts)
    weights = to_rows(M.random_rows((20, 256), w, 0, "f32", g), w)
    for tokens in (3, 70):
        pick = torch.tensor([i % 3 for i in range(tokens)], device="cuda")
        y = R.rhtq_matmul(R.RhtqRows(rows.codes[pick], rows.scales[pick], ts, fmt), weights, out_dtype=torch.float32)
        assert torch.isnan(y[pick == 1]).all() and torch.isfinite(y[pick != 1]).all()


# ----------------------------------------------------------------------------------------------------------------- together

def test_block_of_a_layer():
    """Norm, rotation and INT4 rows; the experts' up projections on the rows that call them; their outputs through a second product."""
    g = gen(9)
    tokens, n, hidden, experts, top = 37, 512, 256, 6, 2
    x = norm_case(tokens, n, "bf16", g).cuda()
    res = norm_case(tokens, n, "bf16", g).cuda()
    signs = (torch.randint(0, 2, (n,), generator=g) * 2 - 1).to(torch.int8).cuda()
    w = (torch.randn(experts * hidden, n, generator=g) * 0.05).cuda()
    packed, scales, _ = R.rhtq_forward(w, signs, fmt="int4", group=128, scale_dtype="f16")
    weights = R.RhtqRows(packed.view(experts, hidden, -1), scales.view(experts, hidden, -1), None, "int4", 128)
    rows, h = R.rhtq_norm_forward(x, None, res, signs=signs, block=n, fmt="int4", scale_dtype="f16")
    pick = torch.stack([torch.randperm(experts, generator=g)[:top] for _ in range(tokens)])
    order = torch.argsort(pick.reshape(-1), stable=True)
    starts = starts_of(torch.bincount(pick.reshape(-1), minlength=experts).tolist())
    index = (order // top).to(torch.int32)
    y = R.rhtq_grouped_matmul(rows, weights, starts.cuda(), index.cuda(), out_dtype=torch.float32)
    xq = R.rhtq_inverse(rows.codes, rows.scales, n, signs, fmt="int4", group=0, scale_dtype="f16").double()
    wq = R.rhtq_inverse(packed, scales, n, signs, fmt="int4", group=128, scale_dtype="f16").double().view(experts, hidden, n)
    for e in range(experts):
        i, j = int(starts[e]), int(starts[e + 1])
        want = xq[index[i:j].long().cuda()] @ wq[e].t()
        # both inverses are fp32 transforms of 9 stages: 2^-24 a stage of a row's size, which the sum of n products adds up as magnitudes
        mags = xq[index[i:j].long().cuda()].norm(dim=1)[:, None] * wq[e].norm(dim=1)[None]
        assert ((y[i:j].double() - want).abs() <= mags * 40 * 2.0 ** -24).all()
    again, _, _ = R.rhtq_forward(y, None, fmt="mxfp4")
    assert again.shape == (tokens * top, hidden // 2)


def test_graph_replays_and_other_stream():
    """The three calls captured as one graph, replayed on new inputs between eager work, and the calls on a stream of their own."""
    g = gen(10)
    n, rows = 1024, 300
    w = to_rows(M.random_rows((rows, n), "mxfp4", 0, "", g), "mxfp4")
    we = to_rows(M.random_rows((4, 64, n), "mxfp4", 0, "", g), "mxfp4")
    starts = torch.tensor([0, 5, 5, 60, 90], dtype=torch.int32, device="cuda")
    x = norm_case(90, n, "bf16", g).cuda()
    res = norm_case(90, n, "bf16", g).cuda()

    def layer():
        q, h = R.rhtq_norm_forward(x, None, res, block=n, fmt="mxfp8")
        return h, R.rhtq_matmul(q, w), R.rhtq_grouped_matmul(q, we, starts)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer()
    for k in range(4):
        x.copy_(norm_case(90, n, "bf16", gen(20 + k)).cuda())
        graph.replay()
        torch.cuda.synchronize()
        eager = layer()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b)
    own = torch.cuda.Stream()
    q, h = R.rhtq_norm_forward(x, None, res, block=n, fmt="mxfp8", stream=own)
    y = R.rhtq_matmul(q, w, stream=own)
    z = R.rhtq_grouped_matmul(q, we, starts, stream=own)
    own.synchronize()
    for a, b in zip((h, y, z), layer()):
        assert torch.equal(a, b)


def test_views_and_empty_calls():
    g = gen(11)
    ra, rw = M.random_rows((6, 256), "int4", 64, "f16", g), M.random_rows((20, 256), "int4", 64, "f16", g)
    a, w = to_rows(ra, "int4", 64), to_rows(rw, "int4", 64)
    want = R.rhtq_matmul(a, w)
    odd = torch.zeros(6 * 128 + 3, dtype=torch.uint8, device="cuda")
    odd[3:] = a.codes.reshape(-1)
    moved = R.RhtqRows(odd[3:].view(6, 128), torch.stack((a.scales, a.scales), 2)[:, :, 0], None, "int4", 64)
    assert torch.equal(R.rhtq_matmul(moved, w), want)
    none = R.RhtqRows(a.codes[:0], a.scales[:0], None, "int4", 64)
    assert R.rhtq_matmul(none, w).shape == (0, 20)
    assert R.rhtq_matmul(a, R.RhtqRows(w.codes[:0], w.scales[:0], None, "int4", 64)).shape == (6, 0)
    assert R.rhtq_norm_forward(torch.zeros(0, 64, device="cuda"))[0].codes.shape == (0, 64)
    x = torch.randn(3, 128, device="cuda").to(torch.bfloat16)
    rows, _ = R.rhtq_norm_forward(x.t().contiguous().t())
    assert torch.equal(rows.codes, R.rhtq_norm_forward(x)[0].codes)


def on_gpu(rows, fmt):
    return M.values(*rows, fmt).cuda()


def expect_on_gpu(y, av, wv, out):
    """expect() with the 64-bit product on the GPU, in blocks of rows."""
    step = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}[out]
    for i in range(0, av.shape[0], 1024):
        a = av[i:i + 1024]
        want, mags = a @ wv.t(), a.abs() @ wv.abs().t()
        bound = step * want.abs() + (1 + step) * mags * (av.shape[-1] + 8) * 2.0 ** -24 + 2.0 ** -25
        assert ((y[i:i + 1024].double() - want).abs() <= bound).all()


@pytest.mark.parametrize("pair", [PAIRS[0], PAIRS[1], PAIRS[3], PAIRS[7], PAIRS[8], PAIRS[9], PAIRS[13], PAIRS[14], PAIRS[15]], ids=lambda p: "-".join(map(str, p)))
@pytest.mark.parametrize("n,tokens,rows", [(256, 4090, 4088), (768, 4096, 4096), (1280, 3850, 4001)])
def test_product_whole_rounds_of_large_tiles(pair, n, tokens, rows):
    """As many tiles of 256 x 256 as the chip has room for; one stage of k, an odd number of them, rows that no vector store fits."""
    a, ag, w, wg, scale = pair
    g = gen(n)
    ra, rw = M.random_rows((tokens, n), a, ag, scale, g), M.random_rows((rows, n), w, wg, scale, g)
    out = "bf16" if rows % 8 == 0 else "f32"
    y = R.rhtq_matmul(to_rows(ra, a, ag), to_rows(rw, w, wg), out_dtype=OUT[out])
    expect_on_gpu(y, on_gpu(ra, a), on_gpu(rw, w), out)


@pytest.mark.parametrize("pair", [PAIRS[0], PAIRS[7], PAIRS[13], PAIRS[14], PAIRS[15]], ids=lambda p: "-".join(map(str, p)))
@pytest.mark.parametrize("n", [32, 224, 352, 608])
def test_large_tiles_end_inside_a_stage(pair, n):
    a, ag, w, wg, scale = pair
    g = gen(n)
    ra, rw = M.random_rows((4096, n), a, ag, scale, g), M.random_rows((4096, n), w, wg, scale, g)
    y = R.rhtq_matmul(to_rows(ra, a, ag), to_rows(rw, w, wg), out_dtype=torch.float16)
    # sums beyond fp16's largest number are infinite there
    av, wv = on_gpu(ra, a), on_gpu(rw, w)
    want = av @ wv.t()
    mags = av.abs() @ wv.abs().t()
    inside = want.abs() < 65000
    bound = 2.0 ** -11 * want.abs() + mags * (n + 8) * 2.0 ** -23 + 2.0 ** -25
    assert ((y.double() - want).abs() <= bound)[inside].all() and (y[want.abs() > 66000].isinf()).all()


@pytest.mark.parametrize("pair", PAIRS, ids=lambda p: "-".join(map(str, p)))
@pytest.mark.parametrize("n", [8448, 8320, 8224])
def test_product_in_parts_of_k(pair, n):
    """Few tiles and a long k: several workgroups share it, and their sums are joined.  33 stages, the last one whole, half full or an eighth."""
    a, ag, w, wg, scale = pair
    if not fits(n, ag, wg):
        pytest.skip("a group does not divide n")
    tokens, rows = 70, 100
    g = gen(77)
    ra, rw = M.random_rows((tokens, n), a, ag, scale, g), M.random_rows((rows, n), w, wg, scale, g)
    assert R.lib.rhtq_matmul_workspace(tokens, n, rows, 0) == 2 * 4 * tokens * rows       # two parts of at least 16 stages
    for out in ("f32", "bf16"):
        y = R.rhtq_matmul(to_rows(ra, a, ag), to_rows(rw, w, wg), out_dtype=OUT[out])
        expect_on_gpu(y, on_gpu(ra, a), on_gpu(rw, w), out)


@pytest.mark.parametrize("pair", [PAIRS[1], PAIRS[3], PAIRS[13], PAIRS[14], PAIRS[15]], ids=lambda p: "-".join(map(str, p)))
def test_grouped_large_tiles(pair):
    a, ag, w, wg, scale = pair
    n, rows, lengths = 256, 4088, [1000, 0, 513, 1, 900, 700]
    tokens, a_rows = sum(lengths), 300
    g = gen(78)
    ra, rw = M.random_rows((a_rows, n), a, ag, scale, g), M.random_rows((6, rows, n), w, wg, scale, g)
    index = torch.randint(0, a_rows, (tokens + 5,), generator=g, dtype=torch.int32)
    index[7] = -3
    starts = starts_of(lengths)
    out = torch.full((tokens + 5, rows), 7.0, device="cuda", dtype=torch.bfloat16)
    R.rhtq_grouped_matmul(to_rows(ra, a, ag), to_rows(rw, w, wg), starts.cuda(), index.cuda(), out=out)
    av, wv = on_gpu(ra, a), on_gpu(rw, w)
    assert (out[tokens:] == 7.0).all() and (out[7] == 0).all()
    picked = av[index.clamp(min=0).long().cuda()]
    picked[7] = 0
    for e in range(6):
        i, j = int(starts[e]), int(starts[e + 1])
        if j > i:
            expect_on_gpu(out[i:j], picked[i:j], wv[e], "bf16")


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8", "nvfp4"])
@pytest.mark.parametrize("tokens", [4, 70, 300])
def test_block_scales_at_odd_addresses(fmt, tokens):
    g = gen(tokens)
    w = "nvfp4" if fmt == "nvfp4" else "mxfp4"
    n, rows = 512, 130
    ra, rw = M.random_rows((tokens, n), fmt, 0, "", g), M.random_rows((rows, n), w, 0, "", g)
    a, b = to_rows(ra, fmt), to_rows(rw, w)
    want = R.rhtq_matmul(a, b, out_dtype=torch.float32)
    for off in (1, 2, 3):
        def moved(r):
            s = torch.zeros(r.scales.numel() + 8, dtype=torch.uint8, device="cuda")[off:off + r.scales.numel()].view(r.scales.shape)
            s.copy_(r.scales)
            return r._replace(scales=s)
        assert torch.equal(R.rhtq_matmul(moved(a), b, out_dtype=torch.float32), want)
        assert torch.equal(R.rhtq_matmul(a, moved(b), out_dtype=torch.float32), want)


def test_calls_on_two_streams_at_once():
    """Each call has a workspace of its own: twelve pairs of calls at once give what they give one after the other."""
    g = gen(80)
    a = to_rows(M.random_rows((70, 8448), "mxfp8", 0, "", g), "mxfp8")
    w = to_rows(M.random_rows((200, 8448), "mxfp4", 0, "", g), "mxfp4")
    b = to_rows(M.random_rows((90, 8448), "int4", 0, "f16", g), "int4")
    v = to_rows(M.random_rows((200, 8448), "int4", 0, "f16", g), "int4")
    want = R.rhtq_matmul(a, w), R.rhtq_matmul(b, v)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    got = [(R.rhtq_matmul(a, w, stream=one), R.rhtq_matmul(b, v, stream=two)) for _ in range(12)]
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])


def test_norm_scales_of_rows_beyond_fp32():
    """A mean of squares that fp32 does not hold gives NaN scales, as a value that is not finite does; the rows beside it stay."""
    x = torch.ones(3, 128, device="cuda")
    x[1] = 1e25
    for fmt in ("int8", "int4"):
        rows, _ = R.rhtq_norm_forward(x, fmt=fmt)
        assert torch.isnan(rows.scales[1]).all() and torch.isfinite(rows.scales[[0, 2]]).all()
    rows, _ = R.rhtq_norm_forward(x, fmt="mxfp4")
    assert (rows.scales[1] == 255).all() and (rows.scales[[0, 2]] < 255).all()


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("fmt", ["int8", "int4", "mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("block", [0, 32])
def test_a_weight_that_is_not_finite_shows(bad, fmt, block):
    """Its groups get NaN scales, the others none."""
    x = torch.rand(3, 256, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) + 0.5
    weight = torch.ones(256, device="cuda")
    weight[100] = bad
    ts = torch.tensor([0.01], device="cuda") if fmt == "nvfp4" else None
    rows, _ = R.rhtq_norm_forward(x, weight, fmt=fmt, group=32 if fmt in ("int8", "int4") else 0, block=block, tensor_scale=ts)
    nan = torch.isnan(rows.scales) if fmt in ("int8", "int4") else rows.scales == (127 if fmt == "nvfp4" else 255)
    size = 16 if fmt == "nvfp4" else 32
    want = torch.zeros_like(nan)
    first, last = (96, 128) if block else (100 // size * size, 100 // size * size + size)     # a rotation spreads it over its block
    want[:, first // size:last // size] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("fmt", ["int8", "int4", "mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("weight", [False, True])
def test_norm_of_zeros_without_eps(fmt, weight):
    x = torch.zeros(2, 128, device="cuda")
    x[1] = 3.0
    ts = torch.tensor([0.01], device="cuda") if fmt == "nvfp4" else None
    rows, _ = R.rhtq_norm_forward(x, torch.ones(128, device="cuda") if weight else None, eps=0.0, fmt=fmt, tensor_scale=ts, block=64)
    assert (rows.codes[0] == 0).all() and (rows.scales[0] == 0).all() and (rows.scales[1] != 0).any()


@pytest.mark.parametrize("fmt", ["int8", "int4", "nvfp4"])
def test_norm_scales_below_the_normal_range(fmt):
    """Weights of 2^-133: 1 / scale is beyond fp32, the codes are right nevertheless.  Both y and the scale are whole multiples of 2^-149; a code is
    off by half a step, of NVFP4 by up to one (between 4 and 6), and the scale's rounding times the code, up to 127, adds to that; so does the
    rounding of weight / root mean square times x."""
    x = norm_case(5, 256, "f32", gen(11)).cuda()
    weight = torch.full((256,), 2.0 ** -133, device="cuda")
    ts = torch.tensor([2.0 ** -138], device="cuda") if fmt == "nvfp4" else None
    rows, _ = R.rhtq_norm_forward(x, weight, fmt=fmt, group=16 if fmt != "nvfp4" else 0, tensor_scale=ts)
    xd = x.double()
    y = (xd * 2.0 ** -133 / (xd.square().mean(1, keepdim=True) + 1e-5).sqrt()).cpu()
    got = M.values(rows.codes.cpu(), rows.scales.cpu(), None if ts is None else ts.cpu(), fmt)
    scale = M.scale_values(rows.scales.cpu(), fmt, None if ts is None else ts.cpu()).repeat_interleave(16, -1)
    most = {"int8": 0.5, "int4": 0.5, "nvfp4": 1.0}[fmt]
    # NVFP4: a group's scale is rounded to E4M3, 2^-4 of it: the largest code, 6, may fall short by 6 / 16 of a step more
    more = 6 * 2.0 ** -4 if fmt == "nvfp4" else 0.0
    assert ((got - y).abs() <= (most + more) * scale * (1 + 2.0 ** -10) + (130 + xd.abs().cpu()) * 2.0 ** -149).all()
    assert (got.abs().amax(1) > 0).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("tokens", [3, 70])
def test_block_scales_of_the_whole_range(fmt, tokens):
    """E8M0 scales from 2^-120 to 2^120 that meet their opposites, give or take 2^8."""
    g = gen(12)
    n, rows = 256, 20
    ca, _, _ = M.random_rows((tokens, n), fmt, 0, "", g)
    cw, _, _ = M.random_rows((rows, n), "mxfp4", 0, "", g)
    e = torch.randint(-120, 121, (n // 32,), generator=g)
    sa = (127 + e).to(torch.uint8).expand(tokens, -1).contiguous()
    sw = (127 - e + torch.randint(-7, 7, (rows, n // 32), generator=g)).clamp(0, 254).to(torch.uint8)
    ra, rw = (ca, sa, None), (cw, sw, None)
    y = R.rhtq_matmul(to_rows(ra, fmt), to_rows(rw, "mxfp4"), out_dtype=torch.float32)
    expect(y, M.values(*ra, fmt), M.values(*rw, "mxfp4"), "f32")


def random_on_gpu(shape, fmt, group, g):
    """Rows of random codes made on the GPU, scales fp16 or E8M0, as RhtqRows."""
    *lead, n = shape
    wide = fmt in ("int8", "mxfp8")
    codes = torch.randint(0, 256, (*lead, n if wide else n // 2), device="cuda", dtype=torch.uint8, generator=g)
    if fmt == "mxfp4":
        scales = torch.randint(120, 132, (*lead, n // 32), device="cuda", dtype=torch.uint8, generator=g)
    else:
        scales = torch.rand(*lead, n // (group or n), device="cuda", generator=g).mul_(0.1).add_(0.01).half()
    return R.RhtqRows(codes.view(torch.int8) if fmt == "int8" else codes, scales, None, fmt, group)


def values_of(rows, *at):
    return M.values(*(t[at].cpu() for t in (rows.codes, rows.scales)), None, rows.fmt).cuda()


@pytest.mark.parametrize("each", [1, 65])
@pytest.mark.parametrize("a,w,group", [("mxfp4", "mxfp4", 0), ("int8", "int4", 128)])
def test_weights_beyond_4_gib(each, a, w, group):
    """Three experts of 2 GiB of codes each, few tokens and tiles: the first and the last rows of every expert."""
    n, rows, experts = 4096, 1 << 20, 3
    g = torch.Generator("cuda").manual_seed(3)
    rw, ra = random_on_gpu((experts, rows, n), w, group, g), random_on_gpu((experts * each, n), a, 0, g)
    starts = torch.arange(0, experts * each + 1, each, dtype=torch.int32, device="cuda")
    y = R.rhtq_grouped_matmul(ra, rw, starts, out_dtype=torch.bfloat16)
    for e in range(experts):
        for part in (slice(0, 300), slice(rows - 300, rows)):
            expect_on_gpu(y[e * each:(e + 1) * each, part], values_of(ra, slice(e * each, (e + 1) * each)), values_of(rw, e, part), "bf16")


@pytest.mark.parametrize("tokens", [3, 70])
def test_rows_taken_from_beyond_4_gib(tokens):
    n, a_rows = 4096, (1 << 21) + 100
    g = torch.Generator("cuda").manual_seed(4)
    ra, rw = random_on_gpu((a_rows, n), "int4", 0, g), random_on_gpu((1, 40, n), "int4", 0, g)
    index = torch.arange(a_rows - tokens, a_rows, dtype=torch.int32, device="cuda")
    y = R.rhtq_grouped_matmul(ra, rw, torch.tensor([0, tokens], dtype=torch.int32, device="cuda"), index, out_dtype=torch.float32)
    expect_on_gpu(y, values_of(ra, slice(a_rows - tokens, a_rows)), values_of(rw, 0), "f32")


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_results_beyond_4_gib(out):
    n, tokens, rows = 32, 2200, (1 << 20) + 8
    g = torch.Generator("cuda").manual_seed(5)
    ra, rw = random_on_gpu((tokens, n), "mxfp4", 0, g), random_on_gpu((rows, n), "mxfp4", 0, g)
    y = R.rhtq_matmul(ra, rw, out_dtype=OUT[out])
    for part in (slice(0, 300), slice(rows - 300, rows)):
        expect_on_gpu(y[tokens - 300:, part], values_of(ra, slice(tokens - 300, tokens)), values_of(rw, part), out)
