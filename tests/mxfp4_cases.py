"""Inputs of the MXFP4 tests whose products are exact in fp32.

Codes are arbitrary E2M1 values (multiples of 1/2, at most 6) and scales
2^(p - 1), 2^p or 2^(p + 1) for a p of each operand, so every product is a
multiple of 2^(pa + pw - 4) and at most 36 * 2^(pa + pw + 2) in magnitude: a
sum of K <= 7000 of them, and each partial sum in any order, is an integer
below 2^24 times 2^(pa + pw - 4), exact in fp32.  With a bias that is such a
multiple too, y is the correctly rounded sum: kernels have to give it bit for
bit.
"""
import numpy as np
import torch

from oracle import formats as F
from oracle import mxfp4 as O


def operand(rng, rows, K, p):
    """(codes [rows, K], scale bytes [rows, K/32])."""
    codes = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    scales = (127 + p + rng.integers(-1, 2, (rows, K // 32))).astype(np.uint8)
    return codes, scales


def weight(rng, lead, N, K, p, device="cuda"):
    """A device weight dict of prod(lead) matrices and its fp64 values [*lead, N, K]."""
    E = int(np.prod(lead)) if lead else 1
    codes, scales = operand(rng, E * N, K, p)
    tiled = np.stack([O.tile(scales[e * N:(e + 1) * N], K) for e in range(E)])
    w = {"codes": torch.from_numpy(O.pack(codes).reshape(*lead, N, K // 2)).to(device),
         "scales": torch.from_numpy(tiled.reshape(*lead, -1)).to(device), "N": N, "K": K, "E": E}
    return w, O.values(codes, scales).reshape(*lead, N, K)


def bias(rng, shape, p):
    """Multiples of 2^(p - 2) that bf16 and fp16 hold exactly."""
    return rng.integers(-100, 101, shape) * 2.0 ** (p - 2)


def rounded(y, dtype):
    """fp64 values that fp32 holds exactly -> dtype (torch, round to nearest even)."""
    y32 = torch.from_numpy(np.asarray(y, np.float64)).to(torch.float32)
    assert np.array_equal(y32.double().numpy(), y), "the case's sums are not exact in fp32"
    return y32.to(dtype)


def rows(rng, M, K, dtype):
    """Rows of x in dtype, with large channels, a zero block and tiny and large rows."""
    x = rng.standard_normal((M, K)).astype(np.float32)
    x *= np.where(rng.random(K) < 0.02, 30.0, 1.0).astype(np.float32)
    x *= np.exp2(rng.integers(-6, 4, (M, 1))).astype(np.float32)
    x[rng.integers(0, M), :32] = 0.0
    return torch.from_numpy(x).to(dtype)


E2M1 = F.E2M1_VALUE
