"""How far a correctly rounded result may be from its float64 definition.

A 16-bit output is off by its own rounding (half a unit in the last place:
2^-8 of the value for bf16, 2^-11 for fp16, 2^-25 below fp16's normal range)
and by the fp32 arithmetic before it; a sum of n fp32 terms in any order is
off by at most (n - 1) 2^-24 of the sum of their magnitudes, and an order of
depth d (threads, then lanes, warps, CTAs) by d 2^-24 of it.
"""
import numpy as np

U16 = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
U32 = 2.0 ** -24


def check16(got, ref, mag, dtype, depth=128, what=""):
    """got (float64 of 16-bit values) against ref; mag: sum of the terms' magnitudes."""
    got, ref, mag = (np.asarray(v, np.float64) for v in (got, ref, mag))
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    before = depth * U32 * mag
    bound = U16[dtype] * (np.abs(ref) + before) + before + (2.0 ** -25 if dtype == "f16" else 0.0)
    off = np.abs(got - ref) - bound
    assert not np.isnan(off).any(), f"{what}: NaN"
    assert (off <= 0).all(), f"{what}: {int((off > 0).sum())} of {off.size} off, worst by {off.max():.3e}"


def check32(got, ref, mag, depth=128, what=""):
    got, ref, mag = (np.asarray(v, np.float64) for v in (got, ref, mag))
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    off = np.abs(got - ref) - (depth * U32 * mag + U32 * np.abs(ref) + 1e-45)
    assert not np.isnan(off).any(), f"{what}: NaN"
    assert (off <= 0).all(), f"{what}: {int((off > 0).sum())} of {off.size} off, worst by {off.max():.3e}"
