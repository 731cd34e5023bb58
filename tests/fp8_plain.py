"""The FP8 operators stated plainly (CPU tensors): rows bit for bit, products in 64 bits with the errors that sums in fp32
and a rounding may make."""

import math

import torch

TOP = 448.0


def blocks(n):
    return -(-n // 128)


def quantise(x):
    """bf16 rows -> (codes as bytes, scales [rows, blocks])."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -cols % 128)).reshape(rows, -1, 128)
    amax = v.abs().amax(2)
    bad = ~v.isfinite().all(2)
    scale = torch.where(amax > 0, amax / TOP, 1.0)
    scale = torch.where(scale > 0, scale, 1.0)
    scale = torch.where(bad, math.nan, scale)
    q = (v / scale[..., None]).clamp(-TOP, TOP)
    q = torch.where(bad[..., None], 0.0, q)
    return q.reshape(rows, -1)[:, :cols].to(torch.float8_e4m3fn).view(torch.uint8), scale


def values(codes, scales):
    v = codes.view(torch.float8_e4m3fn).double()
    return v * scales[:, :blocks(codes.shape[1])].double().repeat_interleave(128, 1)[:, :codes.shape[1]]


def weight_values(codes, scales):
    """[E, n_out, k] codes, [E, blocks, blocks] scales."""
    v = codes.view(torch.float8_e4m3fn).double()
    s = scales.double().repeat_interleave(128, 1)[:, :codes.shape[1]].repeat_interleave(128, 2)[:, :, :codes.shape[2]]
    return v * s


def product(x, w, offsets):
    """fp64 rows times their experts' matrices, and the sums of the terms' magnitudes; rows of no expert are NaN."""
    out = torch.full((x.shape[0], w.shape[1]), math.nan, dtype=torch.float64)
    size = torch.zeros_like(out)
    for e, (a, b) in enumerate(zip(offsets, offsets[1:])):
        out[a:b] = x[a:b] @ w[e].T
        size[a:b] = x[a:b].abs() @ w[e].T.abs()
    return out, size


def tolerance(out, size, k, dtype):
    """The products of codes are exact; a block's 128 are summed on the tensor core (fp32, an ulp an addition at most), the
    blocks in fp32 with their factors' products, the row weight; then half a step of the result's type."""
    sums = (128 + blocks(k) + 8) * 2.0**-23 * size
    return sums + torch.finfo(dtype).eps / 2 * (out.abs() + sums)


def packed(codes):
    """The packed layout, byte by byte as the header says."""
    E, n, k = codes.shape
    U, C = -(-n // 256), blocks(k)
    out = torch.zeros(E * U * C * 32768, dtype=torch.uint8)
    row, col = torch.meshgrid(torch.arange(n), torch.arange(k), indexing="ij")
    u, r, c, b = row // 256, row % 256, col // 128, col % 128
    at = (u * C + c) * 32768 + 128 * r + 16 * ((b // 16) ^ (r % 8)) + b % 16
    for e in range(E):
        out[e * U * C * 32768 + at.flatten()] = codes[e].flatten()
    return out
