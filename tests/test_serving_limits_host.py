"""CPU: calls at the edges of what the serving header allows, answered or refused on the host before any HIP call."""
import ctypes
import os
import subprocess
import sys

import torch

import randomized_hadamard_rotation_amd as R
from randomized_hadamard_rotation_amd import serving

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, NIL = 0x100000, None       # never dereferenced: every call below is refused or has nothing to do
EINVAL, EUNS, OK = R.RHTQ_EINVAL, R.RHTQ_EUNSUPPORTED, R.RHTQ_OK


def cache(**kw):
    a = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, layers=1, pages=10, kv_heads=2, page=16, head_dim=128,
             scale_dtype=R.RHTQ_SCALE_F16)
    a.update(kw)
    return ctypes.byref(serving._CacheStruct(**a))


def append(c=None, k=FAKE, tokens=4, table=FAKE, width=3, lengths=FAKE, starts=NIL, seqs=4):
    return R.lib.rhtq_cache_append(c or cache(), k, k, R.RHTQ_IN_BF16, tokens, 256, 128, 256, 128, table, width, lengths, starts, seqs, NIL,
                                   NIL, NIL)


def read(c=None, k=FAKE, tokens=4, table=FAKE, width=3, lengths=FAKE, starts=NIL, seqs=4):
    return R.lib.rhtq_cache_read(c or cache(), k, k, R.RHTQ_IN_BF16, tokens, table, width, lengths, starts, seqs, NIL, NIL, NIL)


def test_rows_of_no_sequence_without_sequences():
    """seqs = 0: lengths and the table have no entry, and starts has one.  Rows are passed over; nothing is enqueued to store them."""
    assert append(seqs=0, starts=FAKE, lengths=NIL, table=NIL) == OK
    assert append(seqs=0, starts=FAKE) == OK
    assert append(seqs=0, starts=NIL) == EINVAL          # without starts there is one row a sequence
    assert append(seqs=0, starts=FAKE, k=NIL) == EINVAL
    assert append(seqs=1, starts=FAKE, lengths=NIL) == EINVAL and read(seqs=1, starts=FAKE, table=NIL) == EINVAL


def test_most_rows_of_a_call():
    """2^31 - 2^23 rows: the numbers of the rows that a call's last, partly empty column of blocks stands for stay below 2^31."""
    most = 2 ** 31 - 2 ** 23
    assert append(tokens=most + 1, starts=FAKE) == EINVAL and read(tokens=most + 1, starts=FAKE) == EINVAL
    assert append(tokens=most, starts=FAKE, seqs=0) == OK
    for per in (16, 64, 128):                            # rows of a block
        blocks = -(-most // per)
        last = -(-blocks // 32768) * 32768 * per         # blocks in whole columns of 32768
        assert last <= 2 ** 31 - 1


def test_most_rows_of_weights():
    most = 2 ** 31 - 1024
    call = lambda rows: R.lib.rhtq_matvec(FAKE, 0, 1, 32, 32, NIL, 1, FAKE, FAKE, NIL, rows, 0, 0, 0, FAKE, 0, NIL, 0, NIL)  # noqa: E731
    assert call(most + 1) == EINVAL and R.lib.rhtq_matvec_workspace(1, 32, most + 1) == 0
    assert R.lib.rhtq_matvec_workspace(1, 32, most) > 0 and R.lib.rhtq_matvec_workspace(300, 32, most) > 0
    assert -(-most // 256) * 512 < 2 ** 32               # work items along a grid's x


def test_most_queries_of_a_call():
    """2^26 - 64 query heads over all sequences: 64 threads each in the kernel that joins parts."""
    call = lambda seqs, heads: R.lib.rhtq_paged_attention(NIL, 0, seqs, heads, 8, 8, cache(), FAKE, 3, FAKE, NIL, NIL, 0.1, 0, 0, FAKE, FAKE,  # noqa: E731
                                                          1 << 40, NIL)
    assert call(32768, 2048) == EUNS and call(65535, 1026) == EUNS
    assert call(65535, 1022) == EINVAL                   # in range: refused for q's null pointer only


def test_scales_that_are_loaded_in_pairs():
    """NVFP4's bytes and attention's scales are refused at odd places; others are taken one by one.  The launch hook answers RHTQ_EHIP for a
    call that passes its checks, and enqueues nothing."""
    code = """
import sys
sys.path.insert(0, {tests!r})
import test_serving_limits_host as T
R, F, N = T.R, T.FAKE, None
mv = lambda scales, fmt, group, sd: R.lib.rhtq_matvec(F, 0, 1, 32, 32, N, 1, F, scales, F, 4, fmt, group, sd, F, 0, F, 1 << 40, N)
assert mv(F + 1, R.RHTQ_FMT_NVFP4, 16, R.RHTQ_SCALE_E4M3) == T.EINVAL
assert mv(F + 2, R.RHTQ_FMT_NVFP4, 16, R.RHTQ_SCALE_E4M3) == R.RHTQ_EHIP
assert mv(F + 1, R.RHTQ_FMT_MXFP4, 32, R.RHTQ_SCALE_E8M0) == R.RHTQ_EHIP
at = lambda **kw: R.lib.rhtq_paged_attention(F, 0, 4, 8, 1024, 128, T.cache(**kw), F, 9, F, N, N, 0.1, 0, 0, F, F, 1 << 40, N)
f32 = R.RHTQ_SCALE_F32
for kw in (dict(k_scales=F + 2), dict(v_scales=F + 2), dict(k_scales=F + 4, scale_dtype=f32), dict(v_scales=F + 4, scale_dtype=f32)):
    assert at(**kw) == T.EINVAL, kw
    assert T.append(T.cache(**kw)) == R.RHTQ_EHIP, kw
for kw in (dict(), dict(k_scales=F + 4), dict(v_scales=F + 8, scale_dtype=f32)):
    assert at(**kw) == R.RHTQ_EHIP, kw
""".format(tests=os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, RHTQ_TEST_FAIL_LAUNCH="1", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]


def test_row_strides():
    """Rows that start on 16 bytes are taken where they lie, also where an axis of one entry has an odd stride; others are copied."""
    from randomized_hadamard_rotation_amd import serving
    base = torch.arange(6 * 1540, dtype=torch.float32).to(torch.bfloat16).view(6, 1540)
    heads = base[:, :1536].unflatten(1, (12, 128))
    assert heads[:1].stride(0) == 1540
    taken = [(heads[:1], (0, 128)), (heads[::2, 3:4], (3080, 0)), (heads[2:3, 5:6], (0, 0)),
             (heads[:0], (0, 128)), (torch.zeros(4, 5, 2, 128, dtype=torch.bfloat16)[:, :, 1].transpose(0, 1), (256, 1280)),
             (torch.zeros(1, 1, 128, dtype=torch.bfloat16).expand(3, 4, 128), (0, 0))]
    for x, strides in taken:
        got, *s = serving._row_strides(x)
        assert got is x and tuple(s) == strides, (x.shape, x.stride(), s)
    copied = [base[:, 4:1540].unflatten(1, (12, 128)), base[:1, 4:1540].unflatten(1, (12, 128)), torch.ones(2, 128, 4).transpose(1, 2),
              heads[:2]]                                                # and two rows 1540 apart
    for x in copied:
        got, *s = serving._row_strides(x)
        assert got is not x and torch.equal(got, x)
        assert got.is_contiguous() and got.data_ptr() % 16 == 0 and tuple(s) == (x.shape[1] * x.shape[2], x.shape[2])


def test_reference_counts_are_needed_without_sequences_too():
    """Reserve and fork count the free pages whether or not there are sequences."""
    L = R.lib
    assert L.rhtq_pages_reserve(NIL, 3, NIL, 0, NIL, 10, 16, NIL, FAKE, FAKE, 1 << 30, NIL) == EINVAL
    assert L.rhtq_pages_fork(cache(), NIL, 3, NIL, 0, NIL, NIL, NIL, 0, FAKE, FAKE, 1 << 30, NIL) == EINVAL


def test_most_heads_of_a_page():
    """65535 key-value heads, for page calls as for the others."""
    L, many = R.lib, cache(kv_heads=65536)
    assert L.rhtq_pages_copy(many, FAKE, FAKE, 2, NIL) == EUNS
    assert L.rhtq_pages_fork(many, FAKE, 3, FAKE, 4, FAKE, FAKE, FAKE, 2, FAKE, FAKE, 1 << 30, NIL) == EUNS
    assert L.rhtq_pages_compact(many, FAKE, 3, 4, FAKE, FAKE, FAKE, 1 << 30, NIL) == EUNS
    assert L.rhtq_pages_copy(cache(kv_heads=65535), NIL, NIL, 0, NIL) == OK
    assert append(many) == EUNS and read(many) == EUNS
