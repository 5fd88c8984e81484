"""Helpers of the block operators' GPU tests: matrices with guard bands around
them, and error bounds derived from the formulas."""
import numpy as np
import torch

U32 = 2.0 ** -24          # half a unit in the last place of fp32 (rounding to nearest)
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # bf16: 2^-9 to nearest, doubled for values that
#                                                              the fp32 error moves across a rounding boundary


def np64(t):
    return t.detach().double().cpu().numpy()


class Guarded:
    """A rows x cols view in a larger buffer filled with a sentinel; check()
    says that nothing outside the view changed."""

    def __init__(self, rows, cols, dtype, pad=0, offset=0, like=None):
        self.ld = cols + pad
        n = offset + rows * self.ld + 64
        self.buf = torch.full((n,), -77.0, dtype=dtype, device="cuda")
        self.t = torch.as_strided(self.buf, (rows, cols), (self.ld, 1), offset)
        mask = torch.ones(n, dtype=torch.bool, device="cuda")
        torch.as_strided(mask, (rows, cols), (self.ld, 1), offset).fill_(False)
        self.outside = mask
        if like is not None:
            self.t.copy_(like)

    def check(self):
        assert bool((self.buf[self.outside] == -77.0).all()), "written outside the matrix"


def inside(got, want, tol, what):
    got, want = np64(got) if isinstance(got, torch.Tensor) else got, np.asarray(want)
    assert got.shape == want.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    fine = ~np.isnan(want)
    bad = np.abs(got - want)[fine] > np.broadcast_to(tol, want.shape)[fine]
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} beyond the bound, worst "
                           f"{float(np.max((np.abs(got - want) / np.broadcast_to(tol, want.shape))[fine])):.3g} times it")


def product_bound(a, b, k):
    """|error| of an fp32 sum of k products, whatever its order and with each
    addition off by a whole unit in the last place: k * 2^-23 * sum |a b|."""
    return (k + 4) * 2.0 ** -23 * (np.abs(a) @ np.abs(b))


def act_bound(z, ez, kind):
    """Error of activation(z) for a z known to ez: the slope is at most 1.13
    in magnitude; the fp32 evaluation of the formula errs by a few units of the
    exponential's argument (at most 2 |u| with u up to 20 before the result
    saturates) and of erf, 2^-18 of |z| covers both."""
    return ez if kind in ("none", "relu") else 1.13 * ez + 2.0 ** -18 * np.abs(z)


def slope_bound(kind):
    """Error of the slope's fp32 evaluation: it is at most 1.13 in size; 2^-17
    covers exp at arguments up to 40 and the products behind it."""
    return 2.0 ** -24 if kind in ("none", "relu") else 2.0 ** -17
