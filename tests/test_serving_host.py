"""CPU: the serving calls are exported, refuse bad arguments on the host before any HIP call, and their index arithmetic holds
for any table (no kernel is launched here)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import randomized_hadamard_rotation_amd as R
from randomized_hadamard_rotation_amd import serving

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, MIS, NIL = 0x100000, 0x100004, None       # never dereferenced: every call below is refused or has nothing to do
EINVAL, EUNS, OK = R.RHTQ_EINVAL, R.RHTQ_EUNSUPPORTED, R.RHTQ_OK


def test_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "serving", "rhtq_serving.h")).read()
    names = sorted(re.findall(r"^(?:int|int64_t)\s+(rhtq_\w+)\s*\(", src, re.M))
    assert names == sorted(serving.EXPORTED_SERVING)
    lib = ctypes.CDLL(R.LIB_PATH)
    for name in names:
        assert hasattr(lib, name), name
    assert R.rhtq_serving_version() == 1


def test_header_is_c99(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    c = tmp_path / "h.c"
    c.write_text('#include "serving/rhtq_serving.h"\nint main(void) { rhtq_cache_t c; (void)c; return rhtq_serving_version() != 1; }\n')
    pkg = os.path.dirname(R.LIB_PATH)
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(c), "-o",
                    str(tmp_path / "h"), "-L", pkg, "-lrhtq", f"-Wl,-rpath,{pkg}"], check=True, timeout=60)


def test_index_arithmetic(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "paging")
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I",
                    os.path.join(ROOT, "randomized_hadamard_rotation_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c", "rhtq_paging_check.cpp"), "-o", exe], check=True, timeout=120)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


def matvec(**kw):
    a = dict(x=FAKE, dt=0, tokens=4, n=4096, block=4096, signs=NIL, rotated=0, packed=FAKE, scales=FAKE, ts=NIL, rows=8, fmt=0,
             group=128, sd=1, y=FAKE, out=0, work=FAKE, bytes=1 << 40)
    a.update(kw)
    return R.lib.rhtq_matvec(a["x"], a["dt"], a["tokens"], a["n"], a["block"], a["signs"], a["rotated"], a["packed"], a["scales"],
                             a["ts"], a["rows"], a["fmt"], a["group"], a["sd"], a["y"], a["out"], a["work"], a["bytes"], NIL)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), EINVAL), (dict(out=5), EINVAL), (dict(tokens=-1), EINVAL), (dict(rows=-1), EINVAL), (dict(fmt=4), EINVAL),
    (dict(n=16, block=16), EUNS), (dict(n=48, block=48), EUNS), (dict(n=96, block=96), EUNS), (dict(block=100), EUNS),
    (dict(group=96), EUNS), (dict(group=8), EUNS), (dict(sd=2), EUNS), (dict(fmt=1, group=32, sd=2), EUNS),
    (dict(fmt=2, group=32, sd=0), EUNS), (dict(fmt=1, group=16, sd=2), EINVAL), (dict(x=NIL), EINVAL), (dict(packed=NIL), EINVAL),
    (dict(scales=NIL), EINVAL), (dict(y=NIL), EINVAL), (dict(work=NIL), EINVAL), (dict(bytes=4 * 4 * 4096 - 1), EINVAL),
    (dict(x=MIS), EINVAL), (dict(packed=MIS), EINVAL), (dict(y=MIS), EINVAL), (dict(work=MIS), EINVAL), (dict(signs=MIS), EINVAL),
    (dict(scales=FAKE + 1), EINVAL), (dict(tokens=0, x=NIL, y=NIL, work=NIL, bytes=0), OK), (dict(rows=0, packed=NIL, y=NIL), OK),
    (dict(tokens=1 << 40), EINVAL), (dict(rows=1 << 40), EINVAL),
])
def test_matvec_refusals(kw, status):
    assert matvec(**kw) == status


def cache(**kw):
    a = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, layers=1, pages=10, kv_heads=2, page=16, head_dim=128,
             scale_dtype=1)
    a.update(kw)
    return ctypes.byref(serving._CacheStruct(**a))


BAD_CACHES = [(dict(layers=0), EINVAL), (dict(pages=-1), EINVAL), (dict(kv_heads=0), EINVAL), (dict(page=24), EUNS), (dict(page=8), EUNS),
              (dict(page=512), EUNS), (dict(head_dim=96), EUNS), (dict(scale_dtype=2), EUNS), (dict(k_codes=NIL), EINVAL),
              (dict(v_codes=MIS), EINVAL), (dict(v_scales=FAKE + 1), EINVAL), (dict(layers=2), EINVAL)]


def append(c=None, k=FAKE, v=FAKE, dt=0, tokens=4, ks=256, hs=128, vs=256, vh=128, table=FAKE, width=3, lengths=FAKE, starts=NIL,
           seqs=4, signs=NIL):
    return R.lib.rhtq_cache_append(c or cache(), k, v, dt, tokens, ks, hs, vs, vh, table, width, lengths, starts, seqs, signs, signs, NIL)


def read(c=None, k=FAKE, v=FAKE, dt=0, tokens=4, table=FAKE, width=3, lengths=FAKE, starts=NIL, seqs=4, signs=NIL):
    return R.lib.rhtq_cache_read(c or cache(), k, v, dt, tokens, table, width, lengths, starts, seqs, signs, signs, NIL)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(kw, status):
    assert append(cache(**kw)) == status
    assert read(cache(**kw)) == status
    assert attention(c=cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), EINVAL), (dict(tokens=5), EINVAL), (dict(dt=7), EINVAL), (dict(table=NIL), EINVAL), (dict(lengths=NIL), EINVAL),
    (dict(lengths=FAKE + 2), EINVAL), (dict(starts=FAKE + 2), EINVAL), (dict(signs=FAKE + 1), EINVAL), (dict(width=-1), EINVAL),
    (dict(width=1 << 30), EINVAL), (dict(width=(1 << 27) - 1), EINVAL), (dict(seqs=-1, starts=FAKE), EINVAL), (dict(tokens=0, seqs=0, table=NIL, lengths=NIL), OK),
    (dict(tokens=1 << 40, starts=FAKE), EINVAL), (dict(tokens=(1 << 31) - 1, starts=FAKE), EINVAL),
])
def test_row_refusals(kw, status):
    assert append(**kw) == status
    assert read(**kw) == status


def test_append_alignment():
    assert append(k=MIS) == EINVAL and append(v=NIL) == EINVAL and append(ks=130) == EINVAL and append(vh=-128) == EINVAL
    assert append(dt=1, hs=126) == EINVAL
    assert read(k=MIS) == EINVAL and read(k=NIL, v=NIL) == OK


def attention(c=None, q=FAKE, dt=0, seqs=4, heads=8, qs=1024, qh=128, table=FAKE, width=3, lengths=FAKE, scale=0.1, window=0, sinks=0,
              out=FAKE, work=FAKE, size=1 << 40, signs=NIL):
    return R.lib.rhtq_paged_attention(q, dt, seqs, heads, qs, qh, c or cache(), table, width, lengths, signs, signs, scale, window, sinks,
                                      out, work, size, NIL)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=R.RHTQ_IN_F32), EUNS), (dict(dt=9), EINVAL), (dict(heads=0), EINVAL), (dict(heads=3), EUNS), (dict(qs=100), EINVAL),
    (dict(qh=-8), EINVAL), (dict(window=-1), EINVAL), (dict(sinks=-1), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(seqs=70000), EUNS), (dict(q=NIL), EINVAL),
    (dict(out=MIS), EINVAL), (dict(lengths=NIL), EINVAL), (dict(table=NIL), EINVAL), (dict(seqs=-1), EINVAL), (dict(seqs=0, q=NIL), OK),
    (dict(width=1 << 20, work=NIL), EINVAL), (dict(width=1 << 20, size=4), EINVAL), (dict(signs=FAKE + 1), EINVAL),
])
def test_attention_refusals(kw, status):
    assert attention(**kw) == status


def test_page_refusals():
    L = R.lib
    res = lambda **k: L.rhtq_pages_reserve(*(dict(t=FAKE, w=3, l=FAKE, s=4, r=FAKE, p=10, g=16, a=FAKE, st=FAKE, wk=FAKE, b=1 << 30, x=NIL) | k).values())  # noqa: E731,E501
    for kw in (dict(t=NIL), dict(l=NIL), dict(r=NIL), dict(a=NIL), dict(st=NIL), dict(wk=NIL), dict(b=8), dict(w=-1), dict(s=-1), dict(p=-1),
               dict(g=24), dict(g=8), dict(w=1 << 30), dict(t=FAKE + 2), dict(st=FAKE + 1)):
        assert res(**kw) == EINVAL, kw
    fr = lambda **k: L.rhtq_pages_free(*(dict(t=FAKE, w=3, l=FAKE, s=4, r=FAKE, p=10, i=FAKE, c=2, x=NIL) | k).values())  # noqa: E731
    for kw in (dict(t=NIL), dict(l=NIL), dict(r=NIL), dict(i=NIL), dict(c=-1), dict(i=FAKE + 1), dict(w=-1)):
        assert fr(**kw) == EINVAL, kw
    assert fr(c=0, i=NIL) == OK and fr(s=0, t=NIL) == OK
    tr = lambda **k: L.rhtq_pages_trim(*(dict(t=FAKE, w=3, l=FAKE, s=4, r=FAKE, p=10, g=16, n=8, k=1, x=NIL) | k).values())  # noqa: E731
    for kw in (dict(t=NIL), dict(l=NIL), dict(r=NIL), dict(n=0), dict(k=-1), dict(g=20)):
        assert tr(**kw) == EINVAL, kw
    fo = lambda **k: L.rhtq_pages_fork(*(dict(c=cache(), t=FAKE, w=3, l=FAKE, s=4, r=FAKE, i=FAKE, j=FAKE, n=2, st=FAKE, wk=FAKE, b=1 << 30, x=NIL) | k).values())  # noqa: E731,E501
    for kw in (dict(t=NIL), dict(i=NIL), dict(j=NIL), dict(n=-1), dict(st=NIL), dict(wk=NIL), dict(b=16), dict(c=cache(k_scales=FAKE + 2))):
        assert fo(**kw) == EINVAL, kw
    assert fo(c=cache(page=24)) == EUNS
    cp = lambda **k: L.rhtq_pages_copy(*(dict(c=cache(), i=FAKE, j=FAKE, n=2, x=NIL) | k).values())  # noqa: E731
    assert cp(n=-1) == EINVAL and cp(i=NIL) == EINVAL and cp(j=FAKE + 2) == EINVAL and cp(n=0, i=NIL) == OK
    co = lambda **k: L.rhtq_pages_compact(*(dict(c=cache(), t=FAKE, w=3, s=4, r=FAKE, l=FAKE, wk=FAKE, b=1 << 30, x=NIL) | k).values())  # noqa: E731
    for kw in (dict(t=NIL), dict(r=NIL), dict(l=NIL), dict(wk=NIL), dict(b=16), dict(w=-1)):
        assert co(**kw) == EINVAL, kw


def tensors():
    c = R.rhtq_cache_new(6, 2, 16, 128, device="cpu")
    return c, torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(6, dtype=torch.int32)


def test_python_checks_before_the_device():
    c, table, lens, refs = tensors()
    kv = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    ints = torch.zeros(3, dtype=torch.int32)
    bad = [
        lambda: R.rhtq_cache_append(c, kv, kv[:2], table, lens), lambda: R.rhtq_cache_append(c, kv, kv.half(), table, lens),
        lambda: R.rhtq_cache_append(c, kv[:2], kv[:2], table, lens), lambda: R.rhtq_cache_append(c, kv[..., :64], kv[..., :64], table, lens),
        lambda: R.rhtq_cache_append(c, kv, kv, table.long(), lens), lambda: R.rhtq_cache_append(c, kv, kv, table, lens[:2]),
        lambda: R.rhtq_cache_append(c, kv, kv, table, lens, starts=ints), lambda: R.rhtq_cache_append(c, kv.double(), kv.double(), table, lens),
        lambda: R.rhtq_cache_append(c._replace(v_scales=c.v_scales.float()), kv, kv, table, lens),
        lambda: R.rhtq_cache_append(c._replace(v_codes=c.v_codes[:3]), kv, kv, table, lens),
        lambda: R.rhtq_cache_append(R.rhtq_cache_new(6, 2, 16, 128, layers=2, device="cpu"), kv, kv, table, lens),
        lambda: R.rhtq_cache_read(c, table, lens, None, 4), lambda: R.rhtq_cache_read(c, table, lens, None, 3, dtype=torch.int8),
        lambda: R.rhtq_paged_attention(q.float(), c, table, lens), lambda: R.rhtq_paged_attention(q[:2], c, table, lens),
        lambda: R.rhtq_paged_attention(q[:, :3], c, table, lens), lambda: R.rhtq_paged_attention(q, c, table, lens, window=-1),
        lambda: R.rhtq_paged_attention(q, c, table, lens, out=q.float()), lambda: R.rhtq_paged_attention(q[..., :64], c, table, lens),
        lambda: R.rhtq_pages_fork(c, table, lens, refs[:5], ints, ints), lambda: R.rhtq_pages_fork(c, table, lens, refs, ints, ints[:2]),
        lambda: R.rhtq_pages_reserve(table, lens, refs, ints[:2], 16), lambda: R.rhtq_pages_free(table, lens, refs, ints.long()),
        lambda: R.rhtq_pages_copy(c, ints, ints.long()), lambda: R.rhtq_pages_compact(c, table.t(), refs),
        lambda: R.rhtq_cache_new(6, 2, 24, 128, device="cpu"), lambda: R.rhtq_cache_new(6, 2, 16, 96, device="cpu"),
        lambda: R.rhtq_cache_new(6, 2, 16, 128, scale_dtype="e4m3", device="cpu"),
    ]
    w, s = torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 1, dtype=torch.float32)
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    bad += [
        lambda: R.rhtq_matvec(w, s, x[0]), lambda: R.rhtq_matvec(w, s, x.double()), lambda: R.rhtq_matvec(w, s, x[:, :64]),
        lambda: R.rhtq_matvec(w, s.half(), x), lambda: R.rhtq_matvec(w, s, x, fmt="nvfp4"), lambda: R.rhtq_matvec(w, s, x, fmt="int8"),
        lambda: R.rhtq_matvec(w, s, x, out=torch.zeros(2, 9)), lambda: R.rhtq_matvec(w, s, x, out_dtype=torch.int32),
        lambda: R.rhtq_matvec(w, torch.zeros(8, 8, dtype=torch.uint8), x, fmt="nvfp4", tensor_scale=torch.zeros(2)),
        lambda: R.rhtq_matvec(w, s, x, group=96),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
    # well-formed CPU tensors get through the checks and stop at the device check
    good = [
        lambda: R.rhtq_matvec(w, s, x), lambda: R.rhtq_cache_append(c, kv, kv, table, lens), lambda: R.rhtq_cache_read(c, table, lens, None, 3),
        lambda: R.rhtq_paged_attention(q, c, table, lens), lambda: R.rhtq_pages_reserve(table, lens, refs, ints, 16),
        lambda: R.rhtq_pages_free(table, lens, refs, ints), lambda: R.rhtq_pages_trim(table, lens, refs, 16, 4),
        lambda: R.rhtq_pages_fork(c, table, lens, refs, ints, ints), lambda: R.rhtq_pages_copy(c, ints, ints),
        lambda: R.rhtq_pages_compact(c, table, refs),
    ]
    for call in good:
        with pytest.raises(ValueError, match="GPU only"):
            call()
