"""Plain 64-bit forms of the 16-bit products, with the error each computed value may have.

Every bound counts roundings: a product's fp32 sum of K terms is off by at most K 2^-23 sum|a b| (K
additions, each off by at most one step of the running sum, whatever their order), a value rounded
to a type of relative step eps by eps / 2 of itself, and an operand rounded before a product by the
same part of every term.  A bound is a tensor of the output's shape."""
import math

import torch

U32 = 2.0 ** -23


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# absolute part: results below the normal range are rounded to a fixed step
def tiny(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def d(t):
    return t.detach().to("cpu", torch.float64)


def mm(a, b):
    """a b^T in 64 bits and the bound of its fp32 sum."""
    return a @ b.T, a.shape[1] * U32 * (a.abs() @ b.abs().T)


def check(got, ref, bound, what):
    """|got - ref| within the sum's bound and one rounding to got's type."""
    g = d(got)
    lim = bound + (ref.abs() + bound) * half_step(got.dtype) + tiny(got.dtype)
    assert g.shape == ref.shape, f"{what}: shape {tuple(g.shape)}, expected {tuple(ref.shape)}"
    bad = ~((g - ref).abs() <= lim)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; at {i} got {float(g[i])}, expected "
                             f"{float(ref[i])} +- {float(lim[i])}")


def sig(z):
    return 1.0 / (1.0 + torch.exp(-z))


def act(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * sig(z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    return z


def slope(name, z):
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        return sig(z) * (1 + z * (1 - sig(z)))
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


# |act'| <= 1.13 and |act''| <= 1.6 for all of them (relu's slope is given the sign it was computed
# with); a function value costs a few fp32 steps (8 are allowed)
SLOPE, CURVE, FEW = 1.13, 1.6, 8 * U32


class Routing:
    """k distinct experts for each token, grouped; experts of `empty` get none."""

    def __init__(self, T, k, E, seed, empty=(), skew=0.0, own=None):
        g = torch.Generator().manual_seed(seed)
        z = torch.randn((T, E), generator=g) - skew * torch.arange(E).float()
        for e in empty:
            z[:, e] = -1e9
        ids = torch.topk(z, k, dim=1).indices.reshape(-1)
        self.T, self.k, self.E = T, k, E
        self.counts = torch.bincount(ids, minlength=E)
        self.slots = torch.sort(ids, stable=True).indices.to(torch.int32)
        self.offsets = torch.zeros(E + 1, dtype=torch.int32)
        self.offsets[1:] = self.counts.cumsum(0)
        self.g2l = None
        self.E_local = E
        if own is not None:        # local ids in the order given
            self.g2l = torch.full((E,), -1, dtype=torch.int32)
            self.g2l[torch.tensor(own)] = torch.arange(len(own), dtype=torch.int32)
            self.E_local = len(own)

    def spans(self):
        """(local expert, first position, end) of owned experts, rows or none."""
        for e in range(self.E):
            l = e if self.g2l is None else int(self.g2l[e])
            if l >= 0:
                yield l, int(self.offsets[e]), int(self.offsets[e + 1])

    def owned(self):
        m = torch.zeros(self.T * self.k, dtype=torch.bool)
        for _, a, b in self.spans():
            m[a:b] = True
        return m

    def index(self, order):
        """Row of each position in a tensor of that order (0 grouped, 1 slot, 2 token)."""
        if order == 0:
            return torch.arange(self.T * self.k)
        return self.slots.long() if order == 1 else self.slots.long() // self.k

    def rows(self, order):
        return self.T if order == 2 else self.T * self.k
