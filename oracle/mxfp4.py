"""MXFP4 on the CPU (test infrastructure only): quantizer, layouts, products.

Definitions (OCP Microscaling Formats v1.0): blocks of 32 along K; E8M0 scale
byte b = 2^(b - 127), 0xFF NaN; elements E2M1.  For a block with t = max|v|
the scale is 2^max(floor(log2 t) - 2, -127) (section 6.3), the codes the
nearest E2M1 values of v / scale, ties to the even code, saturating at 6.  A
block with a NaN or an infinity gets byte 0xFF and zero codes.
"""
import numpy as np

from oracle import formats as F

BLOCK = 32
MAX_GROUPS = 512


def quantize(x):
    """x float [rows, K] (values exact in fp32) -> (codes [rows, K] one per
    element, scale bytes [rows, K/32])."""
    x = np.asarray(x, dtype=np.float64)
    rows, K = x.shape
    v = x.reshape(rows, K // BLOCK, BLOCK)
    bad = ~np.all(np.isfinite(v), axis=2)
    v = np.where(bad[:, :, None], 0.0, v)
    top = np.max(np.abs(v), axis=2)
    _, e = np.frexp(top)                              # top = m 2^e, m in [1/2, 1)
    e = np.where(top > 0, np.maximum(e - 3, -127), -127)
    u = np.ldexp(v, -e[:, :, None])
    codes = F.e2m1_encode(np.clip(u, -8.0, 8.0).astype(np.float32)) if _exact32(u) else _encode64(u)
    codes = np.where(bad[:, :, None], 0, codes)
    return codes.reshape(rows, K).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def _exact32(u):
    c = np.clip(u, -8.0, 8.0)
    return bool(np.all(c.astype(np.float32).astype(np.float64) == c))


def _encode64(u):
    """The encoder on fp64 values (fp64 intermediate results, not fp32 inputs)."""
    a = np.abs(u)
    step = np.where(a >= 4, 2.0, np.where(a >= 2, 1.0, 0.5))
    mag = np.minimum(np.rint(a / step) * step, 6.0)
    code = np.searchsorted(F.E2M1_MAG, mag)
    return (code | (np.signbit(u).astype(np.int64) << 3)).astype(np.uint8)


def values(codes, scales):
    """fp64 values of codes [rows, K] and scale bytes [rows, K/32]."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return F.e2m1_decode(codes).reshape(*scales.shape, BLOCK).__mul__(s[..., None]).reshape(codes.shape)


def pack(codes):
    """[rows, K] codes -> [rows, K/2] bytes, element 2j in the low nibble."""
    codes = np.asarray(codes, dtype=np.uint8)
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def scale_place(row, group, K):
    """Byte of (row, group) in the tiled layout, by its definition."""
    return ((row // 128) * -(-K // 128) + group // 4) * 512 + (row % 32) * 16 + (row % 128) // 32 * 4 + group % 4


def tile(scales, K):
    """Row-major [rows, K/32] -> the tiled bytes, padding 0."""
    rows, G = scales.shape
    out = np.zeros(-(-rows // 128) * -(-K // 128) * 512, np.uint8)
    r, g = np.meshgrid(np.arange(rows), np.arange(G), indexing="ij")
    out[scale_place(r, g, K)] = scales
    return out


def tile_grouped(scales, K, offsets):
    """Row-major scales -> the grouped layout (group e from block
    offsets[e] // 128 + e on), padding and rows of no group 0."""
    rows, groups = scales.shape[0], len(offsets) - 1
    out = np.zeros((rows // 128 + groups) * -(-K // 128) * 512, np.uint8)
    for e in range(groups):
        lo, hi = offsets[e], offsets[e + 1]
        t = tile(scales[lo:hi], K)
        at = (lo // 128 + e) * -(-K // 128) * 512
        out[at:at + t.size] = t
    return out


def product(a, w, bias=None):
    """fp64 a [M, K] times w [N, K]^T, plus bias."""
    y = a @ w.T
    return y if bias is None else y + bias


def swiglu(g, u):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u
