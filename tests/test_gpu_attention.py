"""GPU: paged attention's rounding against the output type's own."""
import math
import sys

import numpy as np
import pytest

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


def check(o, ref, bound, qt):
    bad = A.off(o.double().cpu().numpy(), ref, bound, torch.finfo(DT[qt]).eps / 2, SUBNORMAL[qt])
    assert not bad.any(), f"heads off: {np.argwhere(bad).tolist()[:10]}"


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
