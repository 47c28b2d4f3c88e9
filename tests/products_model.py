"""Plain 64-bit forms of quantised rows, of their products and of the norm in front of them (CPU tensors, torch only)."""
import math

import torch

E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
BLOCK = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}
TYPES = {"f32": torch.float32, "f16": torch.float16}


def e4m3(b):
    b = b.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10).double())
    v = torch.where((b & 127) == 127, torch.full_like(v, math.nan), v)
    return torch.where(b >= 128, -v, v)


def unpack(codes, fmt):
    """Codes as the numbers that they stand for, without scales."""
    if fmt == "int8":
        return codes.double()
    if fmt == "mxfp8":
        return e4m3(codes)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int64)
    if fmt == "int4":
        return torch.where(c > 7, c - 16, c).double()
    return E2M1[c & 7] * torch.where(c > 7, -1.0, 1.0).double()


def scale_values(scales, fmt, tensor=None):
    if fmt in ("int4", "int8"):
        return scales.double()
    if fmt == "nvfp4":
        return e4m3(scales) * tensor.double().reshape((-1,) + (1,) * (scales.dim() - 1))
    v = 2.0 ** (scales.double() - 127)
    return torch.where(scales == 255, torch.full_like(v, math.nan), v)


def values(codes, scales, tensor, fmt):
    v = unpack(codes, fmt)
    s = scale_values(scales, fmt, tensor)
    return v * s.repeat_interleave(v.shape[-1] // s.shape[-1], -1)


def random_rows(shape, fmt, group, scale, g, any_code=True):
    """Rows [.., n] of any codes and scales that the format has (finite ones), as CPU tensors: codes, scales, tensor scale."""
    *lead, n = shape
    groups = n // (BLOCK.get(fmt) or group or n)
    if fmt == "int8":
        codes = torch.randint(-128, 128, (*lead, n), generator=g).to(torch.int8)
    elif fmt == "mxfp8":
        codes = torch.randint(0, 256, (*lead, n), generator=g)
        codes = torch.where((codes & 127) == 127, codes - 1, codes).to(torch.uint8)
    else:
        codes = torch.randint(0, 256, (*lead, n // 2), generator=g).to(torch.uint8)
    tensor = None
    if fmt in ("int4", "int8"):
        scales = (torch.rand((*lead, groups), generator=g) * 0.1 + 0.01).to(TYPES[scale])
    elif fmt == "nvfp4":
        scales = torch.randint(0, 127, (*lead, groups), generator=g).to(torch.uint8)
        tensor = torch.rand((lead[0] if len(lead) == 2 else 1,), generator=g) * 0.01 + 0.001
    else:
        scales = torch.randint(120, 132, (*lead, groups), generator=g).to(torch.uint8)
    return codes, scales, tensor


def hadamard(y, block):
    n, step = y.shape[-1], 1
    while step < block:
        y = y.reshape(-1, n // (2 * step), 2, step)
        y = torch.stack((y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]), 2).reshape(-1, n)
        step *= 2
    return y / math.sqrt(block)


def normed(x, weight, residual, eps, signs, block):
    """(y, h) in 64 bits; h rounded to x's type."""
    h = x
    if residual is not None:
        h = (x.double() + residual.double()).float().to(x.dtype)
    y = h.double()
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    if block:
        y = hadamard(y if signs is None else y * signs.double(), block)
    return y, h


def group_scales(y, fmt, group, tensor=None):
    """The scale that each group of y [.., n] asks for, before it is rounded to its type."""
    n = y.shape[-1]
    top = y.reshape(*y.shape[:-1], -1, BLOCK.get(fmt) or group or n).abs().amax(-1)
    if fmt in ("int4", "int8"):
        return top / (7 if fmt == "int4" else 127)
    if fmt == "nvfp4":
        return top / (6 * tensor.double())
    return top
