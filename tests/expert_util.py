"""Shared pieces of the tests of RMS norm and the grouped products: segments, operands and the values they stand for."""
import torch

import scaled_quantize_gemm_amax_gb300 as fq
from row_util import F8, FMAX, gen

R, F, O = fq.Recipe, fq.Format, fq.OutDtype
MX = R.MX_1x32_TILED


def e8m0_values(s, rows, cols, tiled):
    """The powers of two that E8M0 bytes stand for, one a 1x32 block, in 64 bits [rows, ceil(cols / 32)]."""
    b = s.view(torch.uint8)
    if tiled:
        b = b.view(rows // 128, cols // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rows, cols // 32)
    return torch.exp2(b.double() - 127)


def values(q, recipe, fmt, s):
    """The values a row-wise copy stands for, in 64 bits."""
    v = q.contiguous().view(F8[int(fmt)]).double()
    rows, cols = v.shape
    if recipe == R.TENSOR:
        return v * s.double().reshape(-1)[0]
    if recipe == R.BLOCK_1x128:
        return v * s.double().repeat_interleave(128, 1)[:, :cols]
    tiled = recipe in (R.MX_1x32_TILED, R.MX_1x32_FLOOR_TILED)
    return v * e8m0_values(s, rows, cols, tiled).repeat_interleave(32, 1)[:, :cols]


def operand(v, recipe, fmt):
    """A matrix quantised by the library's cast: (codes, scales, the values they stand for in 64 bits)."""
    if recipe == R.TENSOR:
        scale = (FMAX[int(fmt)] / v.float().abs().max().clamp(min=1e-20)).reshape(1) if v.numel() else torch.ones(1, device="cuda")
        q, s, _, _ = fq.cast_transpose(v, recipe, fmt, scale, col=False)
        s.copy_(1 / scale)
    else:
        q, s, _, _ = fq.cast_transpose(v, recipe, fmt, col=False)
    return q, s, values(q, recipe, fmt, s)


def offsets_of(blocks, first=0):
    """Segments of the given numbers of 128-row blocks, the first at block `first`."""
    at = [first]
    for b in blocks:
        at.append(at[-1] + b)
    return [128 * a for a in at], torch.tensor([128 * a for a in at], dtype=torch.int32, device="cuda")


def spread(rows, cols, seed, span=6):
    """Normal values, every 128 x 128 block times its own power of two: a block taken from another place is far off."""
    v = torch.randn((rows, cols), generator=gen(seed), device="cuda")
    i = torch.arange((rows + 127) // 128, device="cuda")[:, None]
    j = torch.arange((cols + 127) // 128, device="cuda")[None]
    e = (i * 5 + j * 3 + seed) % (2 * span + 1) - span
    return v * torch.exp2(e.float()).repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def product_tol(a, b, depth, dtype):
    """Of sum_k a b over `depth` products: every 32-deep MMA adds its products and the accumulator with at most one binary32
    truncation (2^-23) an addition, at the magnitude of the sum of absolute products; the scale is one more rounding."""
    return (depth / 32 + 33) * 2.0 ** -23 * (a.abs() @ b.abs().t())
