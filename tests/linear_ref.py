"""The products with activation, residual and experts in 64 bits, for the tests: operands decoded from their bytes."""
import math

import torch

F64 = torch.float64


def decode(q):
    """The values of a QTensor in fp64, per-tensor scale included."""
    block = 16 if q.fmt == 2 else 32

    def e4m3(b):
        b = b.to(torch.int32)
        e, m = (b >> 3) & 15, (b & 7).to(F64)
        size = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2((e - 7).to(F64)))
        return torch.where(b >= 128, -size, size)

    if q.fmt == 1:
        v = e4m3(q.codes)
    else:
        c = torch.stack([q.codes & 15, q.codes >> 4], -1).reshape(-1).to(torch.int32)
        e, m = (c & 7) >> 1, (c & 1).to(F64)
        v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).to(F64)))
        v = torch.where(c >= 8, -v, v)
    r = torch.arange(q.rows, device=q.codes.device)[:, None]
    c = torch.arange(q.cols // block, device=q.codes.device)[None]
    across = -(-(q.cols // block) // 4)
    byte = q.scales[((r // 128) * across + c // 4) * 512 + (r % 32) * 16 + (r // 32) % 4 * 4 + c % 4]
    s = e4m3(byte) if q.fmt == 2 else torch.exp2(byte.to(F64) - 127)
    v = v.reshape(q.rows, q.cols) * s.repeat_interleave(block, 1)
    return v * q.scales[-16:-12].view(torch.float32).to(F64) if q.fmt == 2 else v


def act(name, v):
    if name == "gelu":
        return v * torch.special.ndtr(v)
    if name == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3))
    if name == "silu":
        return v * torch.sigmoid(v)
    return v.clamp(min=0) if name == "relu" else v


def slope(name, v):
    if name == "gelu":
        return torch.special.ndtr(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (v + 0.044715 * v ** 3))
        return 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * c * (1 + 3 * 0.044715 * v * v)
    if name == "silu":
        s = torch.sigmoid(v)
        return s * (1 + v * (1 - s))
    return (v > 0).to(F64) if name == "relu" else torch.ones_like(v)


def sums(a, b, spans, cols, stacked_cols=False):
    """(product, product of magnitudes) of rows' operand a with each span's weights out of b; zeros elsewhere."""
    v, size = (torch.zeros(a.shape[0], cols, dtype=F64, device=a.device) for _ in range(2))
    depth = a.shape[1]
    for e, (lo, hi) in enumerate(spans):
        w = b[:, e * depth:(e + 1) * depth] if stacked_cols else b[e * cols:(e + 1) * cols]
        v[lo:hi] = a[lo:hi] @ w.t()
        size[lo:hi] = a[lo:hi].abs() @ w.abs().t()
    return v, size


# What an output may be off. Sums: 1e-5 of the sum of magnitudes, the GEMMs' bound. An activation's and its derivative's
# slope is at most 1.13; their fp32 evaluation is within 2^-20 of |v| (erfc by the 1.5e-7 formula, exp2 and reciprocal of
# 2^-22). bf16: half a step, 2^-8 of the value; fp32: 2^-23 covers an addition and its rounding.
SUM, ACT = 1e-5, 2.0 ** -20


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, want, tol, what=""):
    assert got.shape == want.shape, (what, got.shape, want.shape)
    err = (got.to(F64) - want).abs()
    bad = ~(err <= tol)  # NaN is bad
    assert not bad.any(), "%s: %d of %d off, worst %.3g of what it may be, first at %s" % (
        what, int(bad.sum()), bad.numel(), float((err / tol.clamp(min=1e-300)).nan_to_num(1e30).max()),
        tuple(bad.nonzero()[0].tolist()))
