"""Plain 64-bit statements of the microscaled formats and of the products on them (CPU tensors, no library code)."""

import torch

FORMATS = ["bf16", "mxfp8", "mxfp4", "nvfp4"]
GROUP = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
TOP = {"mxfp8": 448.0, "mxfp4": 6.0}
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
E4M3 = torch.tensor([(c % 8) * 2.0**-9 if c < 8 else (1 + c % 8 / 8) * 2.0 ** (c // 8 - 7) for c in range(127)],
                    dtype=torch.float64)


def levels(fmt):
    return E4M3 if fmt == "mxfp8" else E2M1


def nearest(t, lv):
    """Index of the nearest level, ties to the even index (t >= 0; beyond the last level: the last)."""
    mids = (lv[1:] + lv[:-1]) / 2
    low, high = torch.bucketize(t, mids), torch.bucketize(t, mids, right=True)
    return torch.where(low % 2 == 0, low, high)


def f32(t):
    """A 64-bit value rounded once to 32 bits."""
    return t.float().double()


def group_divisor(amax, fmt, g=1.0):
    """(scale byte, divisor) of groups from their largest magnitudes (float64, finite)."""
    if fmt == "nvfp4":
        g = float(torch.tensor(g, dtype=torch.float32))
        byte = nearest(f32(amax / float(f32(torch.tensor(6.0 * g, dtype=torch.float64)))), E4M3)
        return byte, f32(E4M3[byte] * g)
    k = torch.full_like(amax, -126.0)
    at = torch.where(amax > 0, amax, 1.0)
    e = torch.floor(torch.log2(at / TOP[fmt])) - 1
    for _ in range(3):                      # the smallest k with amax <= top * 2^k
        e = torch.where(at > TOP[fmt] * torch.exp2(e), e + 1, e)
    k = torch.where(amax > 0, e.clamp(min=-126), k)
    return (k + 127).long(), torch.exp2(k)


def encode(v, fmt, g=1.0):
    """(code bytes, scale bytes) of float64 rows v: what the library has to write, bit for bit, for bf16 input."""
    if fmt == "bf16":
        return v.to(torch.bfloat16).view(torch.uint8), None
    grp = v.reshape(v.shape[0], -1, GROUP[fmt])
    amax = grp.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    byte, div = group_divisor(torch.where(bad, 0.0, amax), fmt, g)
    div = div[..., None]
    t = torch.where((div > 0) & ~bad[..., None], f32(grp.abs() / torch.where(div > 0, div, 1.0)), 0.0)
    code = nearest(t, levels(fmt))
    sign = (torch.signbit(grp) & ~bad[..., None] & (div > 0)).long()
    byte = torch.where(bad, 255 if fmt != "nvfp4" else 127, byte).to(torch.uint8)
    if fmt == "mxfp8":
        return (code + 128 * sign).reshape(v.shape).to(torch.uint8), byte
    half = (code + 8 * sign).reshape(v.shape)
    return (half[:, 0::2] + 16 * half[:, 1::2]).to(torch.uint8), byte


def scale_values(byte, fmt, g=1.0):
    byte = byte.long()
    if fmt == "nvfp4":
        g = float(torch.tensor(g, dtype=torch.float32))
        return torch.where(byte == 127, torch.nan, E4M3[byte.clamp(max=126)]) * g
    return torch.where(byte == 255, torch.nan, torch.exp2(byte.double() - 127))


def code_values(codes, fmt):
    if fmt == "bf16":
        return codes.contiguous().view(torch.bfloat16).double()
    c = codes.long()
    if fmt == "mxfp8":
        return E4M3[(c % 128).clamp(max=126)] * torch.where(c >= 128, -1.0, 1.0)
    half = torch.stack([c % 16, c // 16], -1).flatten(1)
    return E2M1[half % 8] * torch.where(half >= 8, -1.0, 1.0)


def decode(codes, scales, fmt, cols, g=1.0):
    v = code_values(codes, fmt)
    if fmt == "bf16":
        return v
    s = scale_values(scales[:, :cols // GROUP[fmt]], fmt, g)
    return v * s.repeat_interleave(GROUP[fmt], 1)


def pack(parts, fmt, num_experts):
    """The packed layout from [(codes, scales)] of one matrix or of gate and up, addressed byte by byte."""
    words = {"bf16": 0, "mxfp8": 1, "mxfp4": 2, "nvfp4": 4}[fmt]
    tall = 256 // len(parts)
    n_out, width = parts[0][0].shape[0] // num_experts, parts[0][0].shape[1]
    groups = 0 if fmt == "bf16" else width * (1 if fmt == "mxfp8" else 2) // GROUP[fmt]
    units, chunks = -(-n_out // tall), -(-width // 128)
    out = torch.zeros(num_experts, units, chunks, 32768 + 1024 * words, dtype=torch.uint8)
    for m, (codes, scales) in enumerate(parts):
        for r in range(n_out):
            u, br = r // tall, r % tall + m * tall
            for c in range(chunks):
                for j in range(8):
                    piece = codes[r::n_out][:, 128 * c + 16 * j:128 * c + 16 * j + 16]
                    at = 128 * br + 16 * (j ^ (br % 8))
                    out[:, u, c, at:at + piece.shape[1]] = piece
                for w in range(words):
                    g0 = (c * words + w) * 4
                    s = scales[r::n_out][:, g0:min(g0 + 4, groups)]
                    at = 32768 + 1024 * w + 512 * (br // 128) + 16 * (br % 32) + 4 * ((br // 32) % 4)
                    out[:, u, c, at:at + s.shape[1]] = s
    return out.flatten()
