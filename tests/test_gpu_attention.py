"""GPU: paged attention held to a bound that a lost chunk of positions exceeds (tests/test_attention_bound.py), at the lengths that are
split over workgroups and joined; and its rounding against the output type's own."""
import math
import sys

import numpy as np
import pytest

import oracle as O
from tests import attention_model as A

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
SUBNORMAL = {"bf16": 0.0, "f16": 2.0 ** -25}     # half a step of the type's subnormals


def say(*msg):
    print("[case]", *msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    import randomized_hadamard_rotation_amd as R
    return R


def device(R, cache):
    kc, ks, vc, vs, table = (torch.from_numpy(t).cuda() for t in cache)
    return R.RhtqCache(kc, ks, vc, vs), table


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def signs_of(n, seed):
    return np.where(np.random.RandomState(seed).rand(n) < 0.5, -1, 1).astype(np.int8)


def check(o, ref, bound, qt):
    bad = A.off(o.double().cpu().numpy(), ref, bound, torch.finfo(DT[qt]).eps / 2, SUBNORMAL[qt])
    assert not bad.any(), f"heads off: {np.argwhere(bad).tolist()[:10]}"


@pytest.mark.parametrize("lens,heads,kv,dim,page,sd,qt,window,sinks", A.LONG)
def test_long_sequences(R, lens, heads, kv, dim, page, sd, qt, window, sinks):
    say("attention, long", lens, heads, kv, dim, page, sd, qt, window, sinks)
    cache = A.make(lens, kv, dim, page, sd, seed=heads + dim)
    c, table = device(R, cache)
    q = torch.from_numpy(np.random.RandomState(7).randn(len(lens), heads, dim)).to(DT[qt])
    ks, vs = signs_of(dim, 3), signs_of(dim, 4)
    o = R.rhtq_paged_attention(q.cuda(), c, table, ints(*lens), ks, vs, window=window, sinks=sinks)
    ref, bound = A.reference(q.double().numpy(), cache, lens, ks, vs, 1 / math.sqrt(dim), window, sinks)
    check(o, ref, bound, qt)


@pytest.mark.parametrize("n,dim,page", [(700, 128, 16), (4097, 64, 32), (12000, 128, 64), (6000, 256, 16)])
def test_one_position_outweighs_the_rest(R, n, dim, page):
    """Each query's weight lies on one position: the first, the last, and those on both sides of a tile's, a chunk's, a workgroup's round
    and a part's end.  All queries look at the same pages."""
    say("attention, one position", n, dim, page)
    at = sorted({p for p in (0, 1, 15, 16, 63, 64, 511, 512, 1023, 1024, 2560, 4095, 4096, 5119, 5120, n // 2, n - 65, n - 17, n - 2, n - 1)
                 if 0 <= p < n})
    kc, ks, vc, vs, table = A.make([n], 1, dim, page, "f16", seed=n)
    rs = np.random.RandomState(n)
    u = rs.choice([-7, 7], (len(at), dim))
    for i, p in enumerate(at):
        kc[table[0, p // page], 0, p % page] = O.pack_nibbles(u[i][None].astype(np.int64))[0]
        ks[table[0, p // page], 0, p % page] = 0.5
    q = torch.from_numpy(O.inverse_rotate(u / 7.0, None)).to(torch.bfloat16)[:, None]
    table = np.repeat(table, len(at), 0)
    cache = (kc, ks, vc, vs, table)
    c, tb = device(R, cache)
    lens = [n] * len(at)
    o = R.rhtq_paged_attention(q.cuda(), c, tb, ints(*lens), scale=1.0)
    ref, bound = A.reference(q.double().numpy(), cache, lens, None, None, 1.0)
    for i, p in enumerate(at):                                     # the case is what it says
        v, sv = A.rows_of(vc, vs, table[0], 0, [p], page)
        row = O.inverse_rotate(v * sv[:, None], None)[0]
        assert np.linalg.norm(ref[i, 0] - row) < 1e-3 * np.linalg.norm(row)
    check(o, ref, bound, "bf16")


@pytest.mark.parametrize("heads", [16, 28])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("size", [1, 4])
@pytest.mark.parametrize("spread", [False, True])
def test_outputs_are_the_rounded_ones(R, heads, dim, size, spread):
    """Nothing is lost before the output's own rounding: all but 2% of the fp16 outputs are the 64-bit result, rounded once.  fp32 arithmetic
    leaves about 2^-20 of a typical output before that rounding, whose steps are 2^-10.5 of it (twice as fine for small ones): a neighbour
    is taken for 2^-9 of them or so.  Operands of 16 bits took it for 12 to 22%."""
    say("attention, rounding", heads, dim, size, spread)
    lens = [300, 64, 1000, 130]
    cache = A.make(lens, 4, dim, 16, "f16", seed=dim)
    if spread:                                  # a few positions with far larger keys and values
        rs = np.random.RandomState(5)
        cache = (cache[0], (np.exp(rs.randn(*cache[1].shape)) * 0.1).astype(np.float16), cache[2],
                 (np.exp(rs.randn(*cache[3].shape)) * 0.1).astype(np.float16), cache[4])
    c, table = device(R, cache)
    q = torch.from_numpy(np.random.RandomState(3).randn(4, heads, dim) * size).half()
    o = R.rhtq_paged_attention(q.cuda(), c, table, ints(*lens)).cpu().numpy()
    ref, bound = A.reference(q.double().numpy(), cache, lens, None, None, 1 / math.sqrt(dim))
    check(torch.from_numpy(o), ref, bound, "f16")
    other = (o != torch.from_numpy(ref).half().numpy()).mean()
    assert other <= 0.02, f"{other:.3g} of the outputs are another number than the rounded result"


@pytest.mark.parametrize("heads", [8, 14])                    # 4 and 7 query heads of a key-value head
@pytest.mark.parametrize("sd", ["f16", "f32"])
def test_what_is_not_finite_shows(R, sd, heads):
    """A NaN or infinity in one query, or in a scale that a query sees, gives NaN for the heads that it takes part in, and those alone; also
    where the sequence is split and only one part holds it."""
    say("attention, not finite", sd, heads)
    lens, each = [40, 3000, 1], heads // 2
    cache = A.make(lens, 2, 128, 16, sd, seed=3)
    c, table = device(R, cache)
    n = ints(*lens)
    q = torch.randn(3, heads, 128, device="cuda").half()
    ref = R.rhtq_paged_attention(q, c, table, n)
    assert torch.isfinite(ref).all()
    for bad in (float("nan"), float("inf"), -float("inf")):
        for s, h, e in ((0, 0, 0), (1, heads - 1, 77), (2, each, 127)):
            broken = q.clone()
            broken[s, h, e] = bad
            o = R.rhtq_paged_attention(broken, c, table, n)
            assert torch.isnan(o[s, h]).all()
            o[s, h] = ref[s, h]
            assert torch.equal(o, ref)
        for s, p, kv in ((0, 39, 0), (1, 5, 1), (1, 2999, 0), (1, 1500, 1)):
            for which in (1, 3):
                t = [x.clone() for x in c]
                t[which][table[s, p // 16], kv, p % 16] = bad
                o = R.rhtq_paged_attention(q, R.RhtqCache(*t), table, n)
                if which == 3 or bad != bad:        # a key's scale of +-inf: scores of +-inf, NaN only where the largest is +inf
                    assert torch.isnan(o[s, kv * each:(kv + 1) * each]).all(), (bad, s, p, kv, which)
                o[s, kv * each:(kv + 1) * each] = ref[s, kv * each:(kv + 1) * each]
                assert torch.equal(o, ref)


@pytest.mark.parametrize("heads", [3, 6])
@pytest.mark.parametrize("q_size,k_scale,scale,v_scale", [(1e37, 1e-30, 1e-7, 1.0), (1e-29, 1e25, 1e3, 1.0), (1.0, 1.0, 0.05, 1e35),
                                                          (1.0, 1.0, 0.05, 1e-33), (1e36, 1e-36, 1.0, 1e-30)])
def test_ends_of_the_types(R, heads, q_size, k_scale, scale, v_scale):
    """Queries and scales near the ends of bf16 and fp32, scores of ordinary size: the result is as exact as for ordinary ones."""
    say("attention, ends of the types", heads, q_size, k_scale, scale, v_scale)
    n = 300
    kc, ks, vc, vs, table = A.make([n], 1, 128, 16, "f32", seed=2)
    vc[:, :, :, :] = 0x77                                       # every code 7: the rotated sum has all its weight in one element
    vc[table[0, 3], 0, 5] = 0x99                                # but one row of -7
    ks, vs = (ks * k_scale).astype(np.float32), (vs * v_scale).astype(np.float32)
    cache = (kc, ks, vc, vs, table)
    c, tb = device(R, cache)
    q = torch.from_numpy(np.random.RandomState(1).randn(1, heads, 128) * q_size).to(torch.bfloat16)
    o = R.rhtq_paged_attention(q.cuda(), c, tb, ints(n), scale=scale)
    ref, bound = A.reference(q.double().numpy(), cache, [n], None, None, scale)
    # elements that cancel to 0: fp32 sums of 128 values of the largest one's size
    check(o, ref, bound + 2.0 ** -20 * np.abs(ref).max(-1), "bf16")


@pytest.mark.parametrize("heads", [6, 14])
def test_captured_calls_replay_as_eager(R, heads):
    """Split and joined, captured into two graphs, replayed in turn with eager calls and other lengths between."""
    say("attention, captured", heads)
    lens = [6000, 70, 0]
    cache = A.make(lens, 2, 128, 16, "f16", seed=4)
    c, table = device(R, cache)
    sets = [(torch.randn(3, heads, 128, device="cuda").half(), ints(*lens)) for _ in range(2)]
    graphs, outs = [], []
    for q, n in sets:
        R.rhtq_paged_attention(q, c, table, n)
    torch.cuda.synchronize()
    for q, n in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(R.rhtq_paged_attention(q, c, table, n))
        graphs.append(g)
    for turn in range(4):
        for q, n in sets:
            q.mul_(0.5 + turn)
            n.copy_(ints(6000 - 777 * turn, 70 - turn, turn))
        for g in graphs:
            g.replay()
        want = [R.rhtq_paged_attention(q, c, table, n) for q, n in sets]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), turn
