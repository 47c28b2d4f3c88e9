"""CPU: the calls of include/serving/rhtq_products.h are exported and refuse bad arguments on the host before any HIP call (no kernel is
launched here)."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest
import torch

import randomized_hadamard_rotation_amd as R
from randomized_hadamard_rotation_amd import products

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, MIS, NIL = 0x100000, 0x100004, None       # never dereferenced: every call below is refused or has nothing to do
EINVAL, EUNS, OK = R.RHTQ_EINVAL, R.RHTQ_EUNSUPPORTED, R.RHTQ_OK
INT4, NV, MX, INT8, MX8 = 0, 1, 2, 3, 4


def test_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "serving", "rhtq_products.h")).read()
    names = sorted(re.findall(r"^(?:int|int64_t)\s+(rhtq_\w+)\s*\(", src, re.M))
    assert names == sorted(products.EXPORTED_PRODUCTS)
    lib = ctypes.CDLL(R.LIB_PATH)
    for name in names:
        assert hasattr(lib, name), name
    assert R.rhtq_products_version() == 1


def test_header_is_c99(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    c = tmp_path / "h.c"
    c.write_text('#include "serving/rhtq_products.h"\nint main(void) { rhtq_rows_t r; (void)r; return rhtq_products_version() != RHTQ_PRODUCTS_VERSION; }\n')
    pkg = os.path.dirname(R.LIB_PATH)
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(c), "-o",
                    str(tmp_path / "h"), "-L", pkg, "-lrhtq", f"-Wl,-rpath,{pkg}"], check=True, timeout=60)


def rows(fmt=INT4, group=128, sd=1, codes=FAKE, scales=FAKE, ts=NIL):
    return ctypes.byref(products._RowsStruct(codes, scales, ts, fmt, group, sd))


SIDES = {"nv": dict(fmt=NV, group=16, sd=2, ts=FAKE), "mx": dict(fmt=MX, group=32, sd=3), "mx8": dict(fmt=MX8, group=32, sd=3), "i4": {},
         "i8": dict(fmt=INT8, group=0, sd=0)}


def matmul(a="i4", w="i4", ka=(), kw=(), **k):
    v = dict(tokens=4, n=4096, rows=8, y=FAKE, out=0, work=FAKE, bytes=1 << 40)
    v.update(k)
    return R.lib.rhtq_matmul(rows(**{**SIDES[a], **dict(ka)}), v["tokens"], v["n"], rows(**{**SIDES[w], **dict(kw)}), v["rows"], v["y"], v["out"],
                             v["work"], v["bytes"], NIL)


def grouped(a="i4", w="i4", ka=(), kw=(), **k):
    v = dict(a_rows=4, tokens=4, n=4096, experts=2, rows=8, starts=FAKE, index=FAKE, y=FAKE, out=0)
    v.update(k)
    return R.lib.rhtq_grouped_matmul(rows(**{**SIDES[a], **dict(ka)}), v["a_rows"], v["tokens"], v["n"], rows(**{**SIDES[w], **dict(kw)}), v["experts"],
                                     v["rows"], v["starts"], v["index"], v["y"], v["out"], NIL)


BOTH = [
    (dict(out=3), EINVAL), (dict(tokens=-1), EINVAL), (dict(rows=-1), EINVAL), (dict(n=16), EUNS), (dict(n=0), EUNS), (dict(n=48), EUNS),
    (dict(n=(1 << 20) + 32), EUNS), (dict(n=4128), EUNS), (dict(tokens=(1 << 20) + 1), EINVAL), (dict(rows=(1 << 24) + 1), EINVAL),
    (dict(tokens=1 << 20, a_rows=1 << 20, rows=1 << 17), EINVAL), (dict(ka=dict(fmt=5)), EINVAL), (dict(ka=dict(fmt=-1)), EINVAL),
    (dict(ka=dict(group=96)), EUNS), (dict(ka=dict(group=8)), EUNS), (dict(kw=dict(sd=2)), EUNS), (dict(a="nv", w="nv", ka=dict(group=32)), EUNS),
    (dict(a="mx", w="mx", kw=dict(sd=0)), EUNS), (dict(a="mx8", w="mx", ka=dict(group=16)), EUNS), (dict(w="i8"), EUNS), (dict(w="mx"), EUNS),
    (dict(a="nv", w="mx"), EUNS), (dict(a="mx", w="nv"), EUNS), (dict(a="mx", w="mx8"), EUNS), (dict(a="i8", w="mx"), EUNS),
    (dict(ka=dict(codes=NIL)), EINVAL), (dict(ka=dict(scales=NIL)), EINVAL), (dict(kw=dict(codes=MIS)), EINVAL), (dict(kw=dict(scales=FAKE + 1)), EINVAL),
    (dict(a="nv", w="nv", kw=dict(ts=NIL)), EINVAL), (dict(a="nv", w="nv", ka=dict(ts=FAKE + 2)), EINVAL), (dict(y=NIL), EINVAL), (dict(y=MIS), EINVAL),
    (dict(tokens=0, y=NIL, ka=dict(codes=NIL)), OK), (dict(rows=0, y=NIL), OK),
]


@pytest.mark.parametrize("kw,status", BOTH)
def test_matmul_refusals(kw, status):
    assert matmul(**{k: v for k, v in kw.items() if k != "a_rows"}) == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(experts=0), EINVAL), (dict(experts=32768), EINVAL), (dict(a_rows=-1), EINVAL), (dict(a_rows=1 << 31), EINVAL), (dict(a_rows=3, index=NIL), EINVAL),
    (dict(a_rows=0), EINVAL), (dict(starts=NIL), EINVAL), (dict(starts=FAKE + 2), EINVAL), (dict(index=FAKE + 2), EINVAL)])
def test_grouped_refusals(kw, status):
    assert grouped(**kw) == status


def test_null_rows_and_workspace():
    assert R.lib.rhtq_matmul(NIL, 4, 128, rows(), 8, FAKE, 0, FAKE, 1 << 40, NIL) == EINVAL
    assert R.lib.rhtq_matmul(rows(), 4, 128, NIL, 8, FAKE, 0, FAKE, 1 << 40, NIL) == EINVAL
    assert R.lib.rhtq_matmul_workspace(0, 128, 8, 0) == 0 and R.lib.rhtq_matmul_workspace(1 << 40, 128, 8, 0) == 0
    for fmt in range(5):
        for tokens in (1, 70, 333, 2048):
            need = R.lib.rhtq_matmul_workspace(tokens, 12288, 256, fmt)
            assert need >= 0 and need % 16 == 0
            if need:
                side = ("i4", "nv", "mx", "i8", "mx8")[fmt]
                w = {"i8": "i4", "mx8": "mx"}.get(side, side)
                assert matmul(side, w, tokens=tokens, n=12288, rows=256, bytes=need - 1) == EINVAL
                assert matmul(side, w, tokens=tokens, n=12288, rows=256, work=NIL) == EINVAL
                assert matmul(side, w, tokens=tokens, n=12288, rows=256, work=MIS) == EINVAL


def norm(**kw):
    v = dict(x=FAKE, res=FAKE, out=FAKE, dt=0, tokens=4, n=4096, weight=FAKE, eps=1e-5, signs=NIL, block=0, fmt=INT8, group=0, sd=0, codes=FAKE, scales=FAKE,
             ts=NIL)
    v.update(kw)
    return R.lib.rhtq_norm_forward(v["x"], v["res"], v["out"], v["dt"], v["tokens"], v["n"], v["weight"], v["eps"], v["signs"], v["block"], v["fmt"],
                                   v["group"], v["sd"], v["codes"], v["scales"], v["ts"], NIL)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), EINVAL), (dict(tokens=-1), EINVAL), (dict(tokens=1 << 22), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=math.nan), EINVAL),
    (dict(eps=math.inf), EINVAL), (dict(n=16), EUNS), (dict(n=100), EUNS), (dict(n=32800), EUNS), (dict(fmt=5), EINVAL), (dict(group=96), EUNS),
    (dict(sd=2), EUNS), (dict(fmt=NV, group=16, sd=2), EINVAL), (dict(fmt=MX8, group=32, sd=0), EUNS), (dict(fmt=MX, group=16, sd=3), EUNS),
    (dict(block=8), EUNS), (dict(block=96), EUNS), (dict(block=8192), EUNS), (dict(n=5504, block=256), EUNS), (dict(block=64, group=128), EUNS),
    (dict(block=128, signs=MIS), EINVAL), (dict(x=NIL), EINVAL), (dict(x=MIS), EINVAL), (dict(out=NIL), EINVAL), (dict(out=MIS), EINVAL),
    (dict(res=MIS), EINVAL), (dict(weight=MIS), EINVAL), (dict(codes=NIL), EINVAL), (dict(codes=MIS), EINVAL), (dict(scales=NIL), EINVAL),
    (dict(scales=FAKE + 2), EINVAL), (dict(tokens=0, x=NIL), OK),
])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status


# ------------------------------------------------------------------------------------------------------- the Python side, on CPU tensors

def side(rows_=4, n=128, fmt="int4", group=0, lead=(), **kw):
    wide = fmt in ("int8", "mxfp8")
    g = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}.get(fmt) or group or n
    codes = torch.zeros(*lead, rows_, n if wide else n // 2, dtype=torch.int8 if fmt == "int8" else torch.uint8)
    scales = torch.zeros(*lead, rows_, n // g, dtype=torch.float16 if fmt in ("int4", "int8") else torch.uint8)
    return R.RhtqRows(codes, scales, torch.ones(*(lead or (1,))) if fmt == "nvfp4" else None, fmt, group)._replace(**kw)


def refused(call, word):
    with pytest.raises(ValueError, match=word):
        call()


def test_python_refusals():
    ok = side()
    refused(lambda: R.rhtq_matmul(ok, ok), "GPU")                                      # CPU tensors, after every other check
    refused(lambda: R.rhtq_matmul(side(fmt="int5"), ok), "unknown fmt")
    refused(lambda: R.rhtq_matmul(side(lead=(2,)), ok), "2-D")
    refused(lambda: R.rhtq_matmul(ok, side(lead=(2,))), "2-D")
    refused(lambda: R.rhtq_matmul(ok._replace(codes=ok.codes.to(torch.int8)), ok), "expected uint8")
    refused(lambda: R.rhtq_matmul(ok._replace(group=48), ok), "does not divide")
    refused(lambda: R.rhtq_matmul(ok._replace(group=-1), ok), "does not divide")
    refused(lambda: R.rhtq_matmul(ok._replace(scales=ok.scales.double()), ok), "float16 or float32")
    refused(lambda: R.rhtq_matmul(ok._replace(scales=ok.scales[:2]), ok), "scales")
    refused(lambda: R.rhtq_matmul(side(fmt="mxfp4")._replace(scales=torch.zeros(4, 4)), side(fmt="mxfp4")), "expected uint8")
    refused(lambda: R.rhtq_matmul(side(fmt="nvfp4")._replace(tensor_scale=None), side(fmt="nvfp4")), "tensor_scale")
    refused(lambda: R.rhtq_matmul(side(fmt="nvfp4")._replace(tensor_scale=torch.ones(2)), side(fmt="nvfp4")), "tensor_scale")
    refused(lambda: R.rhtq_matmul(ok, side(n=256)), "rows of 128")
    refused(lambda: R.rhtq_matmul(ok, side(fmt="mxfp4")), "multiplied with")
    refused(lambda: R.rhtq_matmul(ok, side(fmt="int8")), "multiplied with")
    refused(lambda: R.rhtq_matmul(ok, ok, out_dtype=torch.float64), "out_dtype")
    refused(lambda: R.rhtq_matmul(ok, ok, out=torch.zeros(4, 5)), "out")
    refused(lambda: R.rhtq_matmul(ok, ok, out=torch.zeros(4, 8)[:, ::2]), "contiguous")
    we, starts = side(lead=(2,)), torch.zeros(3, dtype=torch.int32)
    refused(lambda: R.rhtq_grouped_matmul(ok, we, starts), "GPU")
    refused(lambda: R.rhtq_grouped_matmul(ok, ok, starts), "3-D")
    refused(lambda: R.rhtq_grouped_matmul(ok, we, starts[:2]), "starts")
    refused(lambda: R.rhtq_grouped_matmul(ok, we, starts.long()), "starts")
    refused(lambda: R.rhtq_grouped_matmul(ok, we, starts, torch.zeros(2, 2, dtype=torch.int32)), "1-D")
    refused(lambda: R.rhtq_grouped_matmul(ok, we, starts, torch.zeros(6)), "index")
    refused(lambda: R.rhtq_grouped_matmul(ok, we, starts, torch.zeros(6, dtype=torch.int32), out=torch.zeros(4, 4)), "out")


def test_python_norm_refusals():
    x = torch.zeros(4, 128)
    refused(lambda: R.rhtq_norm_forward(x), "GPU")
    refused(lambda: R.rhtq_norm_forward(x, fmt="fp8"), "unknown fmt")
    refused(lambda: R.rhtq_norm_forward(x[0]), "2-D")
    refused(lambda: R.rhtq_norm_forward(x.double()), "bfloat16, float16 or float32")
    refused(lambda: R.rhtq_norm_forward(x, scale_dtype="f64"), "scale_dtype")
    refused(lambda: R.rhtq_norm_forward(x, group=48), "does not divide")
    refused(lambda: R.rhtq_norm_forward(x, fmt="nvfp4"), "tensor_scale")
    refused(lambda: R.rhtq_norm_forward(x, residual=x.half()), "residual")
    refused(lambda: R.rhtq_norm_forward(x, residual=x[:2]), "residual")
    refused(lambda: R.rhtq_norm_forward(x, residual_out=x), "without a residual")
    refused(lambda: R.rhtq_norm_forward(x, residual=x, residual_out=x.half()), "residual_out")
    refused(lambda: R.rhtq_norm_forward(x, weight=torch.zeros(64)), "weight")
    refused(lambda: R.rhtq_norm_forward(x, weight=torch.zeros(128).half()), "weight")


def test_grouped_results_beyond_a_grid():
    """(tokens + 64 experts) rows: up to 2^35."""
    assert grouped(tokens=1 << 19, a_rows=1 << 19, rows=1 << 16, n=128) == EINVAL
    assert grouped(tokens=64, a_rows=64, experts=16384, rows=1 << 15, n=128) == EINVAL
    assert grouped(tokens=0, experts=32767, rows=16384, n=128) == OK
