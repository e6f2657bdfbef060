"""Values in 64 bits with a bound on how far a computation in 32 bits may be from them.

A ``Bound`` holds a value ``v`` and an error ``e``.  Its operations are those of an evaluation in fp32: every result
is off by what its operands' errors do to it, plus the rounding of the operation itself, ``U`` = 2^-24 of the value for
sums, products and square roots, 2 ``U`` for the hardware's exponential and reciprocal (1 unit in the last place).  A
sum of n terms in any order is off by at most n ``U`` times the sum of their magnitudes."""

import numpy as np

U = 2.0 ** -24


class Bound:
    __array_ufunc__ = None

    def __init__(self, v, e=0.0):
        self.v = np.asarray(v, dtype=np.float64)
        self.e = np.broadcast_to(np.asarray(e, dtype=np.float64), self.v.shape)

    def _made(v, e, u=U):
        return Bound(v, e + u * (np.abs(v) + e))

    def __add__(self, o):
        o = o if isinstance(o, Bound) else Bound(o)
        return Bound._made(self.v + o.v, self.e + o.e)

    __radd__ = __add__

    def __neg__(self):
        return Bound(-self.v, self.e)

    def __sub__(self, o):
        return self + (-(o if isinstance(o, Bound) else Bound(o)))

    def __rsub__(self, o):
        return (-self) + o

    def __mul__(self, o):
        o = o if isinstance(o, Bound) else Bound(o)
        return Bound._made(self.v * o.v, np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e)

    __rmul__ = __mul__

    def __getitem__(self, i):
        return Bound(self.v[i], self.e[i])

    def reshape(self, *shape):
        return Bound(self.v.reshape(*shape), self.e.reshape(*shape))

    def where(self, on, other=0.0):
        return Bound(np.where(on, self.v, other), np.where(on, self.e, 0.0))

    def sum(self, axis):
        n = np.prod([self.v.shape[a] for a in np.atleast_1d(axis)])
        return Bound(self.v.sum(axis), self.e.sum(axis) + n * U * np.abs(self.v).sum(axis))

    def exp(self):
        """Through the exponential of base 2: the factor's and the product's rounding belong to the argument."""
        v = np.exp(self.v)
        return Bound._made(v, v * np.expm1(self.e + 2 * U * np.abs(self.v)), 2 * U)

    def recip(self):
        with np.errstate(divide="ignore"):
            v = 1 / self.v
        return Bound._made(v, self.e / np.maximum(np.abs(self.v) * (np.abs(self.v) - self.e), 1e-300), 2 * U)

    def rsqrt(self):
        v = self.v ** -0.5
        return Bound._made(v, 0.5 * v / self.v * self.e * 1.01, 4 * U)

    def sigmoid(self):
        """1 / (1 + exp(-x)), as the reciprocal gives it on the side where nothing cancels."""
        v = 1 / (1 + np.exp(-np.abs(self.v)))
        v = np.where(self.v >= 0, v, np.exp(-np.abs(self.v)) * v)
        slope = v * (1 - v)
        return Bound._made(v, slope * (self.e + 2 * U * np.abs(self.v)) * 1.01, 8 * U)

    def softplus(self):
        """Within 8 U of the value, besides what the argument's error does."""
        v = np.maximum(self.v, 0) + np.log1p(np.exp(-np.abs(self.v)))
        return Bound._made(v, self.e + 2 * U * np.abs(self.v) * np.exp(-np.abs(self.v)), 8 * U)


def stack(bounds):
    return Bound(np.stack([b.v for b in bounds]), np.stack([b.e for b in bounds]))


HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}      # half a step of the type, relative


def check(name, got, want, dtype="f32", factor=2.0):
    """``got`` (a tensor) within ``factor`` times the bound (for pieces that are composed in another order than one
    after the other, and fused roundings) and half a step of its type of ``want``."""
    g = got.detach().double().cpu().numpy()
    assert g.shape == want.v.shape, (name, g.shape, want.v.shape)
    tol = factor * want.e + HALF[dtype] * (np.abs(want.v) + factor * want.e) + 1e-38
    off = np.abs(g - want.v)
    bad = ~(off <= tol)
    assert not bad.any(), (name, int(bad.sum()), "worst", float((off / tol)[bad].max()),
                           "at", [int(i[0]) for i in np.nonzero(bad)], g[bad][:3], want.v[bad][:3])
