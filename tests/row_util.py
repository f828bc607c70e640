"""Shared pieces of the row operators' tests: inputs of any width, stride and alignment, and
the comparison with a 64-bit result under a tolerance given element by element."""
import torch

U = 2.0 ** -24            # unit roundoff of binary32
BF16 = 2.0 ** -8          # unit roundoff of bfloat16
TINY = 2.0 ** -120        # below this, results may be flushed or lose digits

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
FMAX = {0: 448.0, 1: 57344.0}
F8 = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def matrix(rows, cols, dtype, seed, pad=0, offset=0, sigma=1.0):
    """[rows, cols] normal values with row stride cols + pad, starting `offset` elements into its buffer; what lies
    between the rows is NaN."""
    buf = torch.full((offset + rows * (cols + pad),), float("nan"), dtype=dtype, device="cuda")
    v = buf[offset:].view(rows, cols + pad)[:, :cols]
    v.copy_((torch.randn((rows, cols), generator=gen(seed), device="cuda") * sigma).to(dtype))
    return v


def out_tol(ref, tol, dtype):
    """`tol` of the binary32 result plus one rounding to the output's type."""
    return tol + TINY + ((ref.abs() + tol) * BF16 if dtype == torch.bfloat16 else U * ref.abs())


def assert_within(got, ref, tol, what):
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    nan = ref.isnan()
    assert torch.equal(got.isnan(), nan), f"{what}: NaN at {int((got.isnan() != nan).sum())} other places"
    off = torch.where(nan, 0.0, (got - ref).abs() - tol)
    if off.numel() and not bool((off <= 0).all()):
        i = int(off.argmax())
        raise AssertionError(f"{what}: {int((off > 0).sum())} of {off.numel()} outside; worst at {i}: got "
                             f"{got.flatten()[i]:.9g} ref {ref.flatten()[i]:.9g} tol {tol.expand_as(ref).flatten()[i]:.3g}")


def code_values(q, s, fmt):
    """The values an 8-bit copy stands for, in 64 bits (the product is exact)."""
    v = q.contiguous().view(F8[int(fmt)]).double()
    return v * s.double().repeat_interleave(128, 1)[:, : q.shape[1]]


def codes_of(rows, cols, fmt, seed, pad=0):
    """Random finite codes (row stride cols + pad) and multipliers."""
    g = gen(seed)
    v = torch.randn((rows, cols), generator=g, device="cuda") * FMAX[int(fmt)] / 8
    q = torch.zeros((rows, cols + pad), dtype=torch.uint8, device="cuda")[:, :cols]
    q.copy_(v.clamp(-FMAX[int(fmt)], FMAX[int(fmt)]).to(F8[int(fmt)]).view(torch.uint8))
    s = (0.5 + torch.rand((rows, (cols + 127) // 128), generator=g, device="cuda")) * 8 / FMAX[int(fmt)]
    return q, s
