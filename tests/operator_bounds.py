"""Rounding bounds for the tests of the operators around the head, from the
arithmetic alone: fp32 sums (unit roundoff 2^-24) of a known depth and one
rounding to the output type."""
import numpy as np
import torch

U32 = 2.0 ** -24
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U32}
# half the spacing of the type's subnormal numbers
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def np64(t):
    return t.detach().double().cpu().numpy()


def rounded(ref, dtype):
    """Error of the one rounding to the output type."""
    return UNIT[dtype] * np.abs(ref) + TINY[dtype]


def within(name, got, ref, bound):
    got = np64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, err / np.maximum(bound, 1e-300), 0)), err.shape)
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} outside; at {i}: got {got[i]!r}, "
                             f"want {ref[i]!r}, bound {np.broadcast_to(bound, err.shape)[i]:.3e}")


def sum_depth(D):
    """Additions a term of a row's sum goes through: at least 32 lanes share a row, and
    their partial sums are joined over at most 16 levels."""
    return -(-D // 32) + 16
