"""MXFP4 operators on the GPU against the CPU oracle.

Quantized values are compared byte for byte.  Products run on inputs whose
sums are exact in fp32 (mxfp4_cases.py), so y has to equal the rounded exact
sum bit for bit, whatever the order; products of ordinary values are held to
the bound of fp32 summation.
"""
import collections
import sys
import threading

import numpy as np
import pytest
import torch

import bit_w4a4_diffusion_b200 as B
from oracle import formats as F
from oracle import mxfp4 as O
from tests import mxfp4_cases as C
from tests.helpers import nibbles

pytestmark = pytest.mark.gpu

KERNELS = ["pair256", "pair384", "narrow", None]
DTYPES = [torch.bfloat16, torch.float16]


def pick(monkeypatch, kernel):
    if kernel is None:
        monkeypatch.delenv("SVDQ_MXFP4_GEMM_KERNEL", raising=False)
    else:
        monkeypatch.setenv("SVDQ_MXFP4_GEMM_KERNEL", kernel)


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def same_bits(got, want):
    """Equal values, NaN where NaN is wanted (zeros of either sign are equal)."""
    got, want = got.cpu(), want.cpu()
    assert got.dtype == want.dtype and got.shape == want.shape
    bad = ~((got == want) | (torch.isnan(got) & torch.isnan(want)))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values differ, first at {bad.nonzero()[0].tolist()}"


# ---------------------------------------------------------------- quantize --

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 32), (1, 4096), (5, 96), (32, 128), (33, 160), (97, 288), (128, 256),
                                 (129, 1056), (300, 2080), (1000, 640)])
def test_quantize(M, K, dtype):
    x = C.rows(np.random.default_rng(M * 7 + K), M, K, dtype)
    codes, scales = B.mxfp4_quantize(x.cuda())
    want_c, want_s = O.quantize(x.double().numpy())
    assert np.array_equal(nibbles(codes.cpu().numpy()), want_c)
    assert np.array_equal(B.mxfp4_scales_to_rowmajor(scales.cpu().numpy(), M, K), want_s)
    if K % 128:     # the padding groups of real rows are zero
        tiles = scales.cpu().numpy().reshape(-(-M // 128), -(-K // 128), 32, 4, 4)
        assert not tiles[0, -1, 0, 0, K % 128 // 32:].any()
    for out in (torch.bfloat16, torch.float32):
        v = B.mxfp4_dequantize(codes, scales, dtype=out)
        same_bits(v.double(), torch.from_numpy(O.values(want_c, want_s)))


def test_quantize_every_bf16_value():
    """Every bf16 pattern alone in a block, in a block with a neighbour four
    times its power of two, NaN, infinities and subnormals included."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    X = np.zeros((1 << 16, 64), np.uint16)
    X[:, 3] = bits
    X[:, 32] = bits
    X[:, 47] = np.where((bits & 0x7F80) < 0x7E00, (bits & 0x7F80) + 0x0100, bits)
    codes, scales = B.mxfp4_quantize(B.bits_to_bf16(X, "cuda"))
    want = B.mxfp4_pack_weights(X)
    assert np.array_equal(codes.cpu().numpy(), want["codes"])
    assert np.array_equal(B.mxfp4_scales_to_rowmajor(scales.cpu().numpy(), 1 << 16, 64),
                          B.mxfp4_scales_to_rowmajor(want["scales"], 1 << 16, 64))


def test_quantize_fp32_extremes():
    f = np.finfo(np.float32)
    x = np.zeros((8, 32), np.float32)
    x[0, 0] = f.max
    x[1, 1] = f.tiny
    x[2, 2] = f.smallest_subnormal
    x[3, :3] = [f.tiny, -f.tiny / 2, f.tiny / 4]
    x[4, 4] = np.nan
    x[5, 5] = -np.inf
    x[6, :2] = [-0.0, 0.0]
    x[7, :2] = [np.nextafter(np.float32(8), np.float32(0)), 1.0]
    codes, scales = B.mxfp4_quantize(cuda(x))
    want_c, want_s = O.quantize(x)
    assert np.array_equal(nibbles(codes.cpu().numpy()), want_c)
    assert np.array_equal(B.mxfp4_scales_to_rowmajor(scales.cpu().numpy(), 8, 32), want_s)
    v = B.mxfp4_dequantize(codes, scales, dtype=torch.float32).cpu()
    assert torch.isnan(v[4:6]).all() and not torch.isnan(v[:4]).any()


def test_quantize_strided_rows_and_gather():
    rng = np.random.default_rng(3)
    base = C.rows(rng, 200, 800, torch.bfloat16).cuda()
    x = base[:, 64:64 + 352]                     # rows 800 elements apart
    idx = rng.integers(0, 200, 333).astype(np.int32)
    for ri in (None, cuda(idx)):
        codes, scales = B.mxfp4_quantize(x, row_index=ri)
        src = x.cpu().double().numpy() if ri is None else x.cpu().double().numpy()[idx]
        want_c, want_s = O.quantize(src)
        assert np.array_equal(nibbles(codes.cpu().numpy()), want_c)
        assert np.array_equal(B.mxfp4_scales_to_rowmajor(scales.cpu().numpy(), *src.shape[:1], 352), want_s)


GROUPS = {   # offsets, rows (the capacity)
    "one": ([0, 5], 5),
    "empty ones": ([0, 0, 3, 3, 3, 131, 131, 132], 132),
    "at the borders": ([0, 128, 256, 257, 384, 512], 512),
    "behind the borders": ([0, 129, 130, 259, 515, 516], 516),
    "first and last rows of no group": ([7, 40, 40, 300], 345),
    "all empty": ([9, 9, 9], 20),
    "long": ([0, 1, 700, 701, 1300], 1300),
    "around the tiles": ([0, 383, 767, 1152, 1408, 1408, 1665, 2434], 2440),
}


@pytest.mark.parametrize("name", GROUPS)
def test_quantize_grouped_layout(name):
    off, rows = GROUPS[name]
    K = 416
    rng = np.random.default_rng(rows)
    x = C.rows(rng, rows, K, torch.bfloat16)
    codes = torch.full((rows, K // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((B.mxfp4_scale_bytes(rows, K, len(off) - 1),), 0xFF, dtype=torch.uint8, device="cuda")
    B.mxfp4_quantize(x.cuda(), offsets=cuda(off, torch.int32), out=(codes, scales))
    want_c, want_s = O.quantize(x.double().numpy())
    lo, hi = off[0], off[-1]
    got = codes.cpu().numpy()
    assert np.array_equal(nibbles(got)[lo:hi], want_c[lo:hi])
    assert (got[:lo] == 0xA5).all() and (got[hi:] == 0xA5).all()
    want = O.tile_grouped(want_s, K, off)
    mask = O.tile_grouped(np.ones_like(want_s), K, off).astype(bool)
    assert np.array_equal(scales.cpu().numpy()[mask], want[mask])
    v = B.mxfp4_dequantize(codes, scales, offsets=cuda(off, torch.int32), dtype=torch.float32)
    same_bits(v[lo:hi].double(), torch.from_numpy(O.values(want_c, want_s)[lo:hi]))
    assert not v[:lo].any() and not v[hi:].any()


def test_bad_row_index_is_reported():
    x = C.rows(np.random.default_rng(0), 16, 64, torch.bfloat16).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = cuda([0, 16, 3, -1, 15], torch.int32)
    codes, scales = B.mxfp4_quantize(x, row_index=idx, dev_status=status)
    assert int(status) == 5
    v = B.mxfp4_dequantize(codes, scales)
    assert torch.isnan(v[[1, 3]]).all() and not torch.isnan(v[[0, 2, 4]]).any()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("off", [[0, 5, 3, 8], [0, 4, 9], [-1, 4, 8], [0, -3, 8]])
def test_bad_offsets_are_reported(monkeypatch, kernel, off):
    pick(monkeypatch, kernel)
    rng = np.random.default_rng(0)
    rows, N, K = 8, 32, 64
    w, _ = C.weight(rng, (len(off) - 1,), N, K, 0)
    x = C.rows(rng, rows, K, torch.bfloat16).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    B.mxfp4_grouped_linear(x, cuda(off, torch.int32), w, y=y, dev_status=status)
    assert int(status) == 5
    assert (y == 7.0).all()


@pytest.mark.parametrize("off", [[0, 200, 100, 300], [0, 100, 301, 300], [-1, 0, 10, 300]] +
                         [[0] * 400 + [300, 20, 300]])
def test_bad_offsets_are_reported_by_the_quantizer_alone(off):
    """Also where no row's group has them, and behind the first 32."""
    x = torch.ones(300, 64, dtype=torch.bfloat16, device="cuda")
    offs = cuda(off, torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales = B.mxfp4_quantize(x, offsets=offs, dev_status=status)
    assert int(status) == 5
    status.zero_()
    B.mxfp4_dequantize(codes, scales, offsets=offs, dev_status=status)
    assert int(status) == 5


# ----------------------------------------------------------------- product --

def dense_case(M, N, K, dtype, with_bias, seed, device="cuda"):
    rng = np.random.default_rng(seed)
    a, sa = C.operand(rng, M, K, -3)
    w, wv = C.weight(rng, (), N, K, -2, device)
    b = C.bias(rng, N, -7) if with_bias else None
    y = O.product(O.values(a, sa), wv, b)
    return cuda(O.pack(a)), cuda(O.tile(sa, K)), w, None if b is None else cuda(b, dtype), C.rounded(y, dtype)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("M,N,K", [
    (1, 8, 32), (1, 1024, 2048), (2, 136, 96), (15, 24, 64), (16, 128, 256), (17, 520, 160), (31, 200, 320),
    (32, 128, 288), (33, 392, 512), (64, 1000, 1056), (65, 256, 768), (97, 128, 544), (127, 520, 224),
    (128, 256, 4096), (129, 264, 640), (200, 128, 6400), (255, 304, 96), (256, 256, 256), (257, 520, 352),
    (272, 136, 96), (384, 256, 2048), (385, 512, 288), (512, 264, 64), (600, 1304, 512), (769, 384, 1312),
    (1030, 2056, 1024), (1153, 128, 256), (2900, 1032, 320),
])
def test_gemm_exact(monkeypatch, kernel, M, N, K):
    pick(monkeypatch, kernel)
    for dtype in DTYPES:
        a, sa, w, b, want = dense_case(M, N, K, dtype, dtype == torch.float16 or M % 2 == 0, M + N + K)
        same_bits(B.mxfp4_gemm(a, sa, w, bias=b, dtype=dtype), want)


@pytest.mark.parametrize("kernel", ["pair256", "pair384", "narrow"])
@pytest.mark.parametrize("M,N", [(1, 72), (40, 136), (129, 72), (300, 264)])
def test_gemm_writes_only_y(monkeypatch, kernel, M, N):
    """y as a window of a larger matrix: the rows and columns around it stay."""
    pick(monkeypatch, kernel)
    a, sa, w, b, want = dense_case(M, N, 320, torch.bfloat16, True, 5)
    big = torch.full((M + 2, N + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    y = big[1:M + 1, 8:8 + N]
    assert B.mxfp4_gemm(a, sa, w, bias=b, y=y) is y
    same_bits(y, want)
    big[1:M + 1, 8:8 + N] = 3.0
    assert (big == 3.0).all()


@pytest.mark.parametrize("kernel", ["pair256", "pair384", "narrow"])
def test_gemm_every_code_pair(monkeypatch, kernel):
    """One-element rows: every pair of E2M1 codes at every place of a block,
    scales over a wide range, gives the exact product."""
    pick(monkeypatch, kernel)
    K = 256
    a = np.zeros((256, K), np.uint8)
    w = np.zeros((256, K), np.uint8)
    a[np.arange(256), np.arange(256)] = np.arange(256) % 16
    w[np.arange(256), np.arange(256)] = np.arange(256) // 16
    # y[m, n] is nonzero on the diagonal only; shift the weight rows to see every pair
    rng = np.random.default_rng(0)
    sa = (127 + rng.integers(-40, 41, (256, 8))).astype(np.uint8)
    sw = (127 + rng.integers(-40, 41, (256, 8))).astype(np.uint8)
    wd = {"codes": cuda(O.pack(w)), "scales": cuda(O.tile(sw, K)), "N": 256, "K": K, "E": 1}
    y = B.mxfp4_gemm(cuda(O.pack(a)), cuda(O.tile(sa, K)), wd)
    want = O.values(a, sa) @ O.values(w, sw).T
    same_bits(y.double(), torch.from_numpy(want))      # at most 6 significant bits: exact in bf16


@pytest.mark.parametrize("kernel", ["pair256", "pair384", "narrow"])
def test_nan_and_infinity_reach_only_their_rows_and_columns(monkeypatch, kernel):
    pick(monkeypatch, kernel)
    rng = np.random.default_rng(9)
    M, N, K = 70, 136, 352
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[3, 5], x[40, 351], x[69, 64] = np.nan, np.inf, -np.inf
    w = rng.standard_normal((N, K)).astype(np.float32)
    w[7, 300] = np.nan
    wd = B.to_device(B.mxfp4_pack_weights(F.bf16_bits(w)))
    y = B.mxfp4_linear(cuda(x, torch.bfloat16), wd).cpu()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[[3, 40, 69]] = True
    bad[:, 7] = True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.isfinite(y[~bad]).all()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(1, 2056, 4096), (50, 136, 1056), (300, 520, 736)])
def test_linear_of_ordinary_values(monkeypatch, kernel, dtype, M, N, K):
    """Ordinary x: |y - exact| is at most the output's half unit (finfo.eps / 2
    of the value; the smallest subnormal's half below) and fp32 summation's
    K 2^-23 sum |a w|, each addition truncating at worst."""
    pick(monkeypatch, kernel)
    rng = np.random.default_rng(M + N)
    x = C.rows(rng, M, K, dtype)
    W = rng.standard_normal((N, K)).astype(np.float32) * 0.02
    pk = B.mxfp4_pack_weights(F.bf16_bits(W))
    bias = cuda(rng.standard_normal(N).astype(np.float32), dtype)
    y = B.mxfp4_linear(x.cuda(), B.to_device(pk), bias=bias).cpu().double().numpy()
    a = O.values(*O.quantize(x.double().numpy()))
    w = O.values(nibbles(pk["codes"]), B.mxfp4_scales_to_rowmajor(pk["scales"], N, K))
    want = O.product(a, w, bias.cpu().double().numpy())
    info = torch.finfo(dtype)
    tol = (np.abs(want) * info.eps / 2 + info.smallest_normal * info.eps / 2 +
           (K + 1) * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T + np.abs(bias.cpu().double().numpy())) * (1 + info.eps))
    assert (np.abs(y - want) <= tol).all(), np.max(np.abs(y - want) / tol)


def test_linear_strided_x_and_workspace():
    rng = np.random.default_rng(11)
    base = C.rows(rng, 100, 512, torch.float16).cuda()
    x = base[::2, 128:128 + 288]
    w, _ = C.weight(rng, (), 264, 288, -2)
    want = B.mxfp4_gemm(*B.mxfp4_quantize(x.contiguous()), w, dtype=torch.float16)
    ws = torch.empty(B.mxfp4_workspace_bytes(50, 288), dtype=torch.uint8, device="cuda")
    same_bits(B.mxfp4_linear(x, w, workspace=ws), want)


def steps_linear(x, w, bias=None, **kw):
    """mxfp4_linear in its two steps."""
    return B.mxfp4_gemm(*B.mxfp4_quantize(x), w, bias=bias, dtype=x.dtype, **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,K", [(8, 32), (136, 96), (1000, 544), (2056, 4096)])
def test_linear_around_the_fused_limit(N, K, dtype):
    """Up to eight rows the product quantizes x itself: the same bits as the two
    steps, below the limit and above, special values included."""
    rng = np.random.default_rng(N + K)
    w = B.to_device(B.mxfp4_pack_weights(F.bf16_bits(rng.standard_normal((N, K)).astype(np.float32))))
    b = cuda(rng.standard_normal(N).astype(np.float32), dtype)
    base = C.rows(rng, 40, K + 24, dtype).cuda()
    base[3, 8] = float("inf")
    base[5, 20:K] = 0
    base[6] *= 2.0 ** -18 if dtype == torch.float16 else 2.0 ** -120
    for M in (1, 2, 3, 4, 5, 6, 7, 8, 9, 40):
        x = base[:M, 8:8 + K]
        same_bits(B.mxfp4_linear(x, w, bias=b), steps_linear(x, w, b))


@pytest.mark.parametrize("M", [1, 4])
def test_fused_layers_with_many_slices_and_tiles_per_cta(M):
    """More weight tiles than CTAs and many K slices each: the ring goes round
    often, at another stage for every tile."""
    rng = np.random.default_rng(M)
    g = torch.Generator(device="cuda").manual_seed(M)
    N, K = 128 * 300 + 8, 2848
    x = C.rows(rng, M, K, torch.bfloat16).cuda()

    def weight(E, n):
        return {"codes": torch.randint(0, 256, (E, n, K // 2), dtype=torch.uint8, device="cuda", generator=g),
                "scales": torch.randint(110, 118, (E, B.mxfp4_scale_bytes(n, K)), dtype=torch.uint8, device="cuda",
                                        generator=g), "N": n, "K": K, "E": E}
    w = weight(1, N)
    want = steps_linear(x, w)
    for _ in range(5):
        same_bits(B.mxfp4_linear(x, w), want)
    up, off = weight(2 * 4, 128 * 100), cuda([0, 1, 1, M, M], torch.int32)
    down = {"codes": torch.randint(0, 256, (4, K, 6400), dtype=torch.uint8, device="cuda", generator=g),
            "scales": torch.randint(110, 118, (4, B.mxfp4_scale_bytes(K, 12800)), dtype=torch.uint8, device="cuda",
                                    generator=g), "N": K, "K": 12800, "E": 4}
    q = B.mxfp4_quantize(x, offsets=off)
    want = B.mxfp4_grouped_gemm(*B.mxfp4_grouped_gemm_swiglu_quant(*q, off, up), off, down)
    for _ in range(5):
        same_bits(B.mxfp4_grouped_mlp_swiglu(x, off, up, down), want)


# ----------------------------------------------------------------- grouped --

def grouped_case(off, rows, N, K, dtype, seed, matrices=1, pa=-3, pw=-2, pb=-7):
    rng = np.random.default_rng(seed)
    E = len(off) - 1
    a, sa = C.operand(rng, rows, K, pa)
    w, wv = C.weight(rng, (E,) if matrices == 1 else (E, matrices), N, K, pw)
    b = C.bias(rng, (E, matrices * N), pb)
    av, wv = O.values(a, sa), wv.reshape(E, matrices * N, K)
    y = np.zeros((rows, matrices * N))
    for e in range(E):
        y[off[e]:off[e + 1]] = O.product(av[off[e]:off[e + 1]], wv[e], b[e])
    return cuda(O.pack(a)), cuda(O.tile_grouped(sa, K, off)), cuda(off, torch.int32), w, cuda(b, dtype), y


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("N,K", [(8, 32), (264, 416), (136, 1120)])
def test_grouped_gemm_exact(monkeypatch, kernel, name, N, K):
    pick(monkeypatch, kernel)
    off, rows = GROUPS[name]
    for dtype in DTYPES:
        a, sa, offs, w, b, want = grouped_case(off, rows, N, K, dtype, rows + N)
        y = torch.full((rows, N), -9.0, dtype=dtype, device="cuda")
        B.mxfp4_grouped_gemm(a, sa, offs, w, bias=b, dtype=dtype, y=y)
        lo, hi = off[0], off[-1]
        same_bits(y[lo:hi], C.rounded(want, dtype)[lo:hi])
        assert (y[:lo] == -9.0).all() and (y[hi:] == -9.0).all()


@pytest.mark.parametrize("kernel", KERNELS)
def test_grouped_gemm_many_groups(monkeypatch, kernel):
    """512 groups of 0 to 6 rows, and two of a few hundred."""
    pick(monkeypatch, kernel)
    rng = np.random.default_rng(12)
    counts = rng.integers(0, 7, 512)
    counts[100], counts[400] = 300, 260
    off = np.concatenate([[0], np.cumsum(counts)]).tolist()
    a, sa, offs, w, _, _ = grouped_case(off, off[-1], 64, 96, torch.bfloat16, 3)
    want = grouped_case(off, off[-1], 64, 96, torch.bfloat16, 3)
    same_bits(B.mxfp4_grouped_gemm(a, sa, offs, w, bias=want[4]), C.rounded(want[5], torch.bfloat16))


@pytest.mark.parametrize("kernel", KERNELS)
def test_grouped_linear_gathers(monkeypatch, kernel):
    """Rows gathered by index (one token in several groups, some in none)
    equal the dense layer of each group's rows."""
    pick(monkeypatch, kernel)
    rng = np.random.default_rng(4)
    x = C.rows(rng, 90, 384, torch.bfloat16).cuda()
    off = [0, 40, 40, 41, 200, 230]
    idx = cuda(rng.integers(0, 90, 250), torch.int32)
    W = rng.standard_normal((5, 136, 384)).astype(np.float32)
    w = B.to_device(B.mxfp4_pack_weights(F.bf16_bits(W)))
    y = torch.full((250, 136), 2.0, dtype=torch.bfloat16, device="cuda")
    B.mxfp4_grouped_linear(x, cuda(off, torch.int32), w, row_index=idx, y=y)
    for e in range(5):
        if off[e] == off[e + 1]:
            continue
        we = {"codes": w["codes"][e], "scales": w["scales"][e], "N": 136, "K": 384}
        part = x[idx[off[e]:off[e + 1]].long()]
        same_bits(y[off[e]:off[e + 1]], B.mxfp4_linear(part, we))
    assert (y[230:] == 2.0).all()


SMALL = {   # offsets, rows: up to 16 rows the grouped layers quantize x themselves
    "one row": ([0, 1], 1),
    "one group": ([0, 16], 16),
    "all in the last": ([0, 0, 0, 0, 15], 16),
    "a few each": ([0, 3, 3, 5, 6, 15], 15),
    "rows of no group": ([2, 3, 12, 13], 16),
    "above the limit": ([0, 8, 17], 17),
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", SMALL)
@pytest.mark.parametrize("N,K", [(32, 64), (160, 2080)])
def test_grouped_layers_around_the_fused_limit(name, dtype, N, K):
    off, rows = SMALL[name]
    E = len(off) - 1
    rng = np.random.default_rng(rows + N)
    x = C.rows(rng, 30, K, dtype).cuda()
    x[4, 9] = float("nan")
    offs, idx = cuda(off, torch.int32), cuda(rng.integers(0, 30, rows), torch.int32)
    w = B.to_device(B.mxfp4_pack_weights(F.bf16_bits(rng.standard_normal((E, N, K)).astype(np.float32) * .1)))
    up = B.to_device(B.mxfp4_pack_weights(F.bf16_bits(rng.standard_normal((E, 2, N, K)).astype(np.float32) * .1)))
    down = B.to_device(B.mxfp4_pack_weights(F.bf16_bits(rng.standard_normal((E, K, N)).astype(np.float32) * .1)))
    b = cuda(rng.standard_normal((E, N)).astype(np.float32), dtype)
    q = B.mxfp4_quantize(x, offsets=offs, row_index=idx)
    got, want = (torch.full((rows, N), 6.0, dtype=dtype, device="cuda") for _ in range(2))
    B.mxfp4_grouped_linear(x, offs, w, row_index=idx, bias=b, y=got)
    B.mxfp4_grouped_gemm(*q, offs, w, bias=b, dtype=dtype, y=want)
    same_bits(got, want)
    got, want = (torch.full((rows, K), 6.0, dtype=dtype, device="cuda") for _ in range(2))
    B.mxfp4_grouped_mlp_swiglu(x, offs, up, down, row_index=idx, y=got)
    h = B.mxfp4_grouped_gemm_swiglu_quant(*q, offs, up, dtype=dtype)
    B.mxfp4_grouped_gemm(*h, offs, down, dtype=dtype, y=want)
    same_bits(got, want)


def test_bad_row_index_in_the_fused_layer():
    rng = np.random.default_rng(0)
    x = C.rows(rng, 16, 64, torch.bfloat16).cuda()
    w, _ = C.weight(rng, (2,), 32, 64, 0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = B.mxfp4_grouped_linear(x, cuda([0, 2, 5], torch.int32), w, row_index=cuda([0, 16, 3, -1, 15], torch.int32),
                               dev_status=status)
    assert int(status) == 5
    assert torch.isnan(y[[1, 3]]).all() and not torch.isnan(y[[0, 2, 4]]).any()


# --------------------------------------------------------------------- mlp --

def check_hidden(codes, scales, g, u, K):
    """Codes and scales of h = swiglu(g, u), g and u exact, against the
    quantizer applied anywhere within the error of h as computed in fp32:
    exp's argument is rounded (|g| 2^-24 relative in the result) and the
    exponential, the quotient and two products are good to 2^-21 each."""
    h = O.swiglu(g, u)
    delta = np.abs(h) * (np.abs(g) * 2.0 ** -23 + 2.0 ** -19) + 2.0 ** -120
    rows = h.shape[0]
    top = lambda v: np.max(v.reshape(rows, -1, 32), axis=2)   # noqa: E731
    byte = lambda t: np.maximum(np.frexp(t)[1] - 3, -127) + 127   # noqa: E731
    lo, hi = byte(np.maximum(top(np.abs(h) - delta), 0)), byte(top(np.abs(h) + delta))
    assert ((scales >= lo) & (scales <= hi)).all()
    s = np.repeat(np.ldexp(1.0, scales.astype(np.int64) - 127), 32, axis=1)
    got = F.e2m1_decode(codes)
    low = F.E2M1_VALUE[O._encode64((h - delta) / s)]
    high = F.E2M1_VALUE[O._encode64((h + delta) / s)]
    assert ((got >= low) & (got <= high)).all()
    ref_c, ref_s = O.quantize(h)
    return np.mean((ref_c != codes) & ((ref_c | codes) & 7 > 0)), np.mean(ref_s != scales)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("width,K", [(32, 64), (224, 416), (160, 1120)])
def test_swiglu_quant(monkeypatch, kernel, name, width, K):
    pick(monkeypatch, kernel)
    off, rows = GROUPS[name]
    E = len(off) - 1
    # scales small enough that the gate's values stay within a few tens
    a, sa, offs, w, b, y = grouped_case(off, rows, width, K, torch.float16, rows + K, matrices=2, pa=-3, pw=-4, pb=-4)
    codes = torch.full((rows, width // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((B.mxfp4_scale_bytes(rows, width, E),), 0xFF, dtype=torch.uint8, device="cuda")
    B.mxfp4_grouped_gemm_swiglu_quant(a, sa, offs, w, bias=b, dtype=torch.float16, out=(codes, scales))
    lo, hi = off[0], off[-1]
    got = codes.cpu().numpy()
    assert (got[:lo] == 0xA5).all() and (got[hi:] == 0xA5).all()
    # read the scales back through the layout's definition
    sc, raw = np.zeros((rows, width // 32), np.uint8), scales.cpu().numpy()
    chunks = -(-width // 128)
    for e in range(E):
        n = off[e + 1] - off[e]
        r, g = np.meshgrid(np.arange(n), np.arange(4 * chunks), indexing="ij")
        all_groups = raw[(off[e] // 128 + e) * chunks * 512 + O.scale_place(r, g, width)]
        sc[off[e]:off[e + 1]] = all_groups[:, :width // 32]
        assert not all_groups[:, width // 32:].any()
    if hi > lo:
        flips, scale_flips = check_hidden(nibbles(got[lo:hi]), sc[lo:hi], y[lo:hi, :width], y[lo:hi, width:], K)
        # a decision can differ only within delta of a border; few values lie there
        assert flips < 1e-3 and scale_flips < 1e-3


@pytest.mark.parametrize("kernel", ["pair256", "pair384", "narrow"])
def test_swiglu_quant_of_nan_and_large_values(monkeypatch, kernel):
    """A NaN block in x makes its row's hidden blocks NaN (byte 255, codes 0);
    a gate of a few hundred either way gives 0 or the other factor."""
    pick(monkeypatch, kernel)
    rng = np.random.default_rng(2)
    K, width = 64, 64
    x = rng.standard_normal((6, K)).astype(np.float32)
    x[2, 3] = np.nan
    x[4] *= 300
    w = B.to_device(B.mxfp4_pack_weights(F.bf16_bits(rng.standard_normal((1, 2, width, K)).astype(np.float32))))
    off = cuda([0, 6], torch.int32)
    q = B.mxfp4_quantize(cuda(x, torch.bfloat16), offsets=off)
    codes, scales = B.mxfp4_grouped_gemm_swiglu_quant(*q, off, w)
    v = B.mxfp4_dequantize(codes, scales, offsets=off, dtype=torch.float32).cpu()
    assert torch.isnan(v[2]).all()
    keep = [0, 1, 3, 4, 5]
    a = O.values(*O.quantize(F.bf16_round(x)))
    pk = w["codes"].cpu().numpy().reshape(2 * width, K // 2)
    sw = B.mxfp4_scales_to_rowmajor(w["scales"].cpu().numpy(), width, K).reshape(2 * width, K // 32)
    y = a[keep] @ O.values(nibbles(pk), sw).T
    h = O.swiglu(y[:, :width], y[:, width:])
    want = O.values(*O.quantize(h))
    err = np.linalg.norm(v[keep].double().numpy() - want) / np.linalg.norm(want)
    assert err < 1e-3


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("name", GROUPS)
def test_mlp_equals_its_steps(monkeypatch, kernel, name):
    """The whole MLP gives what quantize, up product and down product give."""
    pick(monkeypatch, kernel)
    off, rows = GROUPS[name]
    E, K, width = len(off) - 1, 288, 224
    rng = np.random.default_rng(rows)
    x = C.rows(rng, 64, K, torch.bfloat16).cuda()
    idx = cuda(rng.integers(0, 64, rows), torch.int32)
    offs = cuda(off, torch.int32)
    up = B.to_device(B.mxfp4_pack_weights(F.bf16_bits(rng.standard_normal((E, 2, width, K)).astype(np.float32) * .06)))
    down = B.to_device(B.mxfp4_pack_weights(F.bf16_bits(rng.standard_normal((E, K, width)).astype(np.float32) * .06)))
    ub, db = (cuda(rng.standard_normal(s).astype(np.float32), torch.bfloat16) for s in ((E, 2 * width), (E, K)))
    y = torch.full((rows, K), 5.0, dtype=torch.bfloat16, device="cuda")
    B.mxfp4_grouped_mlp_swiglu(x, offs, up, down, row_index=idx, up_bias=ub, down_bias=db, y=y)
    q = B.mxfp4_quantize(x, offsets=offs, row_index=idx)
    h = B.mxfp4_grouped_gemm_swiglu_quant(*q, offs, up, bias=ub)
    want = torch.full_like(y, 5.0)
    B.mxfp4_grouped_gemm(*h, offs, down, bias=db, y=want)
    same_bits(y, want)


def moe_reference(x, chosen, weights, up, down):
    """fp64: every token through its experts, summed with its weights."""
    T, k = chosen.shape
    out = np.zeros((T, down.shape[1]))
    a = O.values(*O.quantize(x))
    for e in range(up.shape[0]):
        t, j = np.nonzero(chosen == e)
        if len(t) == 0:
            continue
        y = a[t] @ up[e].T
        h = O.swiglu(y[:, :up.shape[1] // 2], y[:, up.shape[1] // 2:])
        out[t] += weights[t, j][:, None] * (O.values(*O.quantize(h)) @ down[e].T)
    return out


@pytest.mark.parametrize("T", [1, 7, 150, 900])
def test_experts_layer(T):
    """The operators as a model uses them: route, sort, MLP over the gathered
    rows, weighted sum back; and a dense layer behind it."""
    rng = np.random.default_rng(T)
    E, k, K, width = 8, 2, 256, 160
    x = C.rows(rng, T, K, torch.bfloat16)
    chosen = np.argsort(rng.random((T, E)) + np.linspace(0, .5, E), axis=1)[:, :k]
    wts = rng.random((T, k)).astype(np.float32)
    upk = B.mxfp4_pack_weights(F.bf16_bits(rng.standard_normal((E, 2, width, K)).astype(np.float32) * 0.06))
    dpk = B.mxfp4_pack_weights(F.bf16_bits(rng.standard_normal((E, K, width)).astype(np.float32) * 0.08))
    flat = torch.from_numpy(chosen.reshape(-1)).cuda()
    order = torch.argsort(flat, stable=True)
    off = torch.cat([flat.new_zeros(1), torch.bincount(flat, minlength=E).cumsum(0)]).to(torch.int32)
    y = B.mxfp4_grouped_mlp_swiglu(x.cuda(), off, B.to_device(upk), B.to_device(dpk),
                                   row_index=(order // k).to(torch.int32))
    out = torch.zeros(T, K, device="cuda")
    out.index_add_(0, order // k, y.float() * torch.from_numpy(wts.reshape(-1)).cuda()[order][:, None])
    up = O.values(nibbles(upk["codes"].reshape(-1, K // 2)),
                  B.mxfp4_scales_to_rowmajor(upk["scales"], width, K).reshape(-1, K // 32)).reshape(E, 2 * width, K)
    down = O.values(nibbles(dpk["codes"].reshape(-1, width // 2)),
                    B.mxfp4_scales_to_rowmajor(dpk["scales"], K, width).reshape(-1, width // 32)).reshape(E, K, width)
    want = moe_reference(x.double().numpy(), chosen, wts.astype(np.float64), up, down)
    # bf16 rounding of each expert's row (2^-8 of it at most), and rare hidden
    # decisions at a border, each worth at most one E2M1 step of one product
    err = np.linalg.norm(out.cpu().double().numpy() - want) / np.linalg.norm(want)
    assert err < 2.0 ** -8
    z = B.mxfp4_linear(out.to(torch.bfloat16), B.to_device(B.mxfp4_pack_weights(
        F.bf16_bits(np.eye(K, dtype=np.float32)))))
    same_bits(z.double(), torch.from_numpy(O.values(*O.quantize(out.to(torch.bfloat16).cpu().double().numpy()))))


# -------------------------------------------------------------- large sizes --

def test_offsets_beyond_32_bits():
    """Matrices of more than 2^32 elements: rows at the end equal those of a
    small call."""
    M, K = 66000, 65536 + 32
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    tail = C.rows(np.random.default_rng(1), 200, K, torch.bfloat16).cuda()
    x[-200:] = tail
    codes, scales = B.mxfp4_quantize(x)
    want_c, want_s = B.mxfp4_quantize(tail)
    assert torch.equal(codes[-200:], want_c)
    v = B.mxfp4_dequantize(codes, scales, out=x)
    assert v is x
    same_bits(x[-200:].cpu(), B.mxfp4_dequantize(want_c, want_s).cpu())
    del x, codes, scales, v
    N, K = 66048, 64
    x = C.rows(np.random.default_rng(2), M, K, torch.bfloat16).cuda()
    w, _ = C.weight(np.random.default_rng(3), (), N, K, 0)
    y = B.mxfp4_linear(x, w)
    same_bits(y[-300:, -520:].cpu(), B.mxfp4_linear(x[-300:], w)[:, -520:].cpu())
    same_bits(y[:300, :520].cpu(), B.mxfp4_linear(x[:300], w)[:, :520].cpu())


# ------------------------------------------------- streams, graphs, threads --

def layer_set(seed=0, T=40, E=6, K=256, width=128):
    rng = np.random.default_rng(seed)
    x = C.rows(rng, T, K, torch.bfloat16).cuda()
    off = cuda(np.concatenate([[0], np.sort(rng.integers(0, T, E - 1)), [T]]), torch.int32)
    up = B.to_device(B.mxfp4_pack_weights(F.bf16_bits(rng.standard_normal((E, 2, width, K)).astype(np.float32) * .1)))
    down = B.to_device(B.mxfp4_pack_weights(F.bf16_bits(rng.standard_normal((E, K, width)).astype(np.float32) * .1)))
    return x, off, up, down


def test_captured_graph_follows_its_inputs():
    """A captured MLP replays with other rows, offsets and weights in place."""
    x, off, up, down = layer_set(1)
    y = torch.empty_like(x)
    ws = torch.empty(B.mxfp4_mlp_workspace_bytes(6, 40, 256, 128), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.mxfp4_grouped_mlp_swiglu(x, off, up, down, y=y, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.mxfp4_grouped_mlp_swiglu(x, off, up, down, y=y, workspace=ws)
    for seed in (2, 3):
        x2, off2, up2, down2 = layer_set(seed)
        x.copy_(x2)
        off.copy_(off2)
        for a, b in ((up, up2), (down, down2)):
            a["codes"].copy_(b["codes"])
            a["scales"].copy_(b["scales"])
        y.fill_(-1)
        g.replay()
        same_bits(y, B.mxfp4_grouped_mlp_swiglu(x2, off2, up2, down2))


def test_weights_written_just_before_the_call():
    """Weights, offsets and rows written on the stream right before the call
    are the ones it uses (its kernels start early and wait)."""
    sets = [layer_set(s) for s in range(6)]
    want = [B.mxfp4_grouped_mlp_swiglu(*s).clone() for s in sets]
    x, off, up, down = layer_set(9)
    for _ in range(5):
        for s, y in zip(sets, want):
            x.copy_(s[0])
            off.copy_(s[1])
            for a, b in ((up, s[2]), (down, s[3])):
                a["scales"].copy_(b["scales"])
                a["codes"].copy_(b["codes"])
            same_bits(B.mxfp4_grouped_mlp_swiglu(x, off, up, down), y)


def test_quantized_weight_used_at_once():
    """A weight quantized on the device and used by the next calls, back to
    back, with nothing between them."""
    rng = np.random.default_rng(8)
    x = C.rows(rng, 3, 512, torch.bfloat16).cuda()
    Ws = [cuda(rng.standard_normal((1024, 512)).astype(np.float32), torch.bfloat16) for _ in range(4)]
    codes = torch.empty(1024, 256, dtype=torch.uint8, device="cuda")
    scales = torch.empty(B.mxfp4_scale_bytes(1024, 512), dtype=torch.uint8, device="cuda")
    w = {"codes": codes, "scales": scales, "N": 1024, "K": 512}
    want = []
    for W in Ws:
        B.mxfp4_quantize(W, out=(codes, scales))
        torch.cuda.synchronize()
        want.append(B.mxfp4_linear(x, w))
        torch.cuda.synchronize()
    got = []
    for W in Ws * 3:
        B.mxfp4_quantize(W, out=(codes, scales))
        got.append(B.mxfp4_linear(x, w))
    for i, y in enumerate(got):
        same_bits(y, want[i % 4])


def test_two_streams_at_once():
    sets = [layer_set(s, T=300) for s in (1, 2)]
    want = [B.mxfp4_grouped_mlp_swiglu(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(B.mxfp4_grouped_mlp_swiglu(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            same_bits(y, want[i])


def test_two_host_threads_at_once():
    """Each with its stream, its layer and sizes that take different kernels."""
    sets = [layer_set(1, T=12), layer_set(2, T=900, E=3)]
    want = [B.mxfp4_grouped_mlp_swiglu(*s) for s in sets]
    torch.cuda.synchronize()
    got = [[], []]

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got[i].append(B.mxfp4_grouped_mlp_swiglu(*sets[i]))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 50
        for y in got[i]:
            same_bits(y, want[i])


def test_stream_argument():
    x, off, up, down = layer_set(5)
    st = torch.cuda.Stream()
    want = B.mxfp4_grouped_mlp_swiglu(x, off, up, down)
    y = torch.empty_like(x)
    ws = torch.empty(B.mxfp4_mlp_workspace_bytes(6, 40, 256, 128), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    B.mxfp4_grouped_mlp_swiglu(x, off, up, down, y=y, workspace=ws, stream=st)
    st.synchronize()
    same_bits(y, want)


def test_stream_argument_owns_what_the_call_allocates():
    """Output and workspace of a call on another stream come from that
    stream's memory: work queued on the current stream does not get them."""
    x, off, up, down = layer_set(5, T=200)
    want = B.mxfp4_grouped_mlp_swiglu(x, off, up, down)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for handle in (st, st.cuda_stream):
        got = []
        for _ in range(20):
            got.append(B.mxfp4_grouped_mlp_swiglu(x, off, up, down, stream=handle))
            junk = torch.full((1 << 20,), 0xAB, dtype=torch.uint8, device="cuda")
            del junk
        torch.cuda.synchronize()
        for y in got:
            same_bits(y, want)


def test_runs_are_bit_identical():
    """No atomics and a fixed order: the same call gives the same bits, also
    where a cluster splits K."""
    rng = np.random.default_rng(6)
    w = B.to_device(B.mxfp4_pack_weights(F.bf16_bits(rng.standard_normal((512, 4096)).astype(np.float32))))
    for M in (1, 30, 200):
        x = C.rows(rng, M, 4096, torch.bfloat16).cuda()
        first = B.mxfp4_linear(x, w)
        for _ in range(5):
            assert torch.equal(B.mxfp4_linear(x, w), first)


def test_pdl_off_gives_the_same(monkeypatch):
    x, off, up, down = layer_set(7)
    want = B.mxfp4_grouped_mlp_swiglu(x, off, up, down)
    monkeypatch.setenv("SVDQ_PDL", "0")
    same_bits(B.mxfp4_grouped_mlp_swiglu(x, off, up, down), want)


def timed_out(call, status):
    """Runs ``call`` with a wait limit of 1 ns and returns the status code."""
    old = B.get_timeout_ns()
    try:
        B.set_timeout_ns(1)
        call()
        torch.cuda.synchronize()
    finally:
        B.set_timeout_ns(old)
    code = int(status)
    status.zero_()
    return code


@pytest.mark.parametrize("kernel,M,N,K", [("pair256", 600, 1024, 65536), ("pair384", 600, 768, 65536),
                                          ("narrow", 700, 8200, 16384), ("narrow", 30, 512, 131072),
                                          (None, 1, 40008, 16384), (None, 2, 1024, 131072)])
def test_a_wait_that_gives_up_is_reported(monkeypatch, kernel, M, N, K):
    """Every kernel, also with K split over a cluster and with the quantizer
    inside, reports a wait that gave up and leaves the library usable.  The
    clock is read every 64 polls, a few microseconds apart, so K is so long
    that the epilogue waits tens of them for its first tile."""
    pick(monkeypatch, kernel)
    g = torch.Generator(device="cuda").manual_seed(M)
    x = C.rows(np.random.default_rng(M), M, K, torch.bfloat16).cuda()
    w = {"codes": torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g),
         "scales": torch.randint(110, 118, (B.mxfp4_scale_bytes(N, K),), dtype=torch.uint8, device="cuda",
                                 generator=g), "N": N, "K": K}
    want = steps_linear(x, w)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert timed_out(lambda: B.mxfp4_linear(x, w, dev_status=status), status) in (1, 2, 3, 4)
    same_bits(B.mxfp4_linear(x, w, dev_status=status), want)
    assert int(status) == 0


def test_many_waits_that_give_up_with_the_quantizer_inside():
    """Wherever in the ring the waits give up, the kernel ends in order, with
    its copies landed, and the next calls are right."""
    M, N, K = 3, 40008, 8192
    g = torch.Generator(device="cuda").manual_seed(M)
    x = C.rows(np.random.default_rng(M), M, K, torch.bfloat16).cuda()
    w = {"codes": torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g),
         "scales": torch.randint(110, 118, (B.mxfp4_scale_bytes(N, K),), dtype=torch.uint8, device="cuda",
                                 generator=g), "N": N, "K": K}
    want = steps_linear(x, w)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for i in range(200):
        old = B.get_timeout_ns()
        try:
            B.set_timeout_ns(1 + 40 * i)
            B.mxfp4_linear(x, w, dev_status=status)
        finally:
            B.set_timeout_ns(old)
        if i % 20 == 19:
            status.zero_()
            same_bits(B.mxfp4_linear(x, w, dev_status=status), want)
            assert int(status) == 0


@pytest.mark.parametrize("kernel,T", [("pair", 3000), ("narrow", 3000), (None, 12)])
def test_a_wait_that_gives_up_in_the_mlp_is_reported(monkeypatch, kernel, T):
    pick(monkeypatch, kernel)
    x, off, up, down = layer_set(3, T=T, E=2, K=32768, width=256)
    want = B.mxfp4_grouped_mlp_swiglu(x, off, up, down)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert timed_out(lambda: B.mxfp4_grouped_mlp_swiglu(x, off, up, down, dev_status=status), status) in (1, 2, 3, 4)
    same_bits(B.mxfp4_grouped_mlp_swiglu(x, off, up, down, dev_status=status), want)
    assert int(status) == 0


def test_no_rows():
    x, off, up, down = layer_set(3)
    none = x[:0]
    zero = torch.zeros_like(off)
    assert B.mxfp4_quantize(none)[0].shape == (0, 128)
    assert B.mxfp4_grouped_mlp_swiglu(none, zero, up, down).shape == (0, 256)
    y = torch.full_like(x, 4.0)
    B.mxfp4_grouped_mlp_swiglu(x, zero, up, down, y=y)
    assert (y == 4.0).all()


def test_python_refusals():
    x, off, up, down = layer_set(4)
    w1 = {"codes": down["codes"][0], "scales": down["scales"][0], "N": 256, "K": 128}
    with pytest.raises(B.SvdqError):
        B.mxfp4_linear(x, w1)                                   # K differs
    with pytest.raises(B.SvdqError):
        B.mxfp4_grouped_linear(x, off[:-1], down)               # one weight too many
    with pytest.raises(TypeError):
        B.mxfp4_grouped_linear(x, off.long(), up)
    with pytest.raises(TypeError):
        B.mxfp4_linear(x.float(), w1)
    with pytest.raises(ValueError):
        B.mxfp4_quantize(x.t())
    with pytest.raises(ValueError):
        B.mxfp4_grouped_mlp_swiglu(x, off, up, down, y=torch.empty(3, 256, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        B.mxfp4_quantize(x, out=(torch.empty(40, 128, dtype=torch.uint8, device="cuda"),
                                 torch.empty(8, dtype=torch.uint8, device="cuda")))
    with pytest.raises(ValueError):
        B.mxfp4_grouped_mlp_swiglu(x, off, up, down, up_bias=torch.empty(4, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        B.mxfp4_linear(x[:, :128].contiguous(), w1, bias=torch.empty(256, dtype=torch.float16, device="cuda"))


def test_sizes_past_an_int_are_refused():
    """They would reach the library cut off (views of one element, no memory)."""
    huge = 2**32 + 32
    x, off, up, _ = layer_set(4)
    with pytest.raises(B.SvdqError):
        B.mxfp4_quantize(x[:1, :1].expand(huge, 1))
    with pytest.raises(B.SvdqError):
        B.mxfp4_quantize(x[:1, :1].expand(1, huge))
    with pytest.raises(B.SvdqError):
        B.mxfp4_quantize(x, row_index=off[:1].expand(huge))
    with pytest.raises(B.SvdqError):
        B.mxfp4_dequantize(up["codes"].reshape(-1)[:1].expand(huge, 1), up["scales"])
    with pytest.raises(B.SvdqError):
        B.mxfp4_linear(x, {**up, "E": 1, "N": huge})


def test_values_past_the_largest_become_infinite():
    """Scale bytes that the quantizer never writes: 6 * 2^127 and so on."""
    a = np.full((1, 32), 7, np.uint8)      # codes of 6
    for byte, want in ((252, 6.0 * 2.0**125), (253, np.inf), (254, np.inf)):
        scales = cuda(O.tile(np.full((1, 1), byte, np.uint8), 32))
        v = B.mxfp4_dequantize(cuda(O.pack(a)), scales, dtype=torch.float32).cpu()
        assert (v == want).all(), byte


def test_binding_arguments():
    """Weights of any mapping; wrong ones are refused before anything runs."""
    x, off, up, down = layer_set(4)
    want = B.mxfp4_grouped_mlp_swiglu(x, off, up, down)
    same_bits(B.mxfp4_grouped_mlp_swiglu(x, off, collections.UserDict(up), collections.UserDict(down)), want)
    codes, scales = B.mxfp4_quantize(x, offsets=off)
    with pytest.raises(KeyError):
        B.mxfp4_grouped_mlp_swiglu(x, off, up, {k: v for k, v in down.items() if k != "scales"})
    with pytest.raises(TypeError):
        B.mxfp4_grouped_mlp_swiglu(x, off, up, {**down, "codes": down["codes"].cpu()})
    with pytest.raises(TypeError):
        B.mxfp4_grouped_mlp_swiglu(x, off, up, None)
    with pytest.raises(TypeError):
        B.mxfp4_grouped_linear(x, None, down)
    with pytest.raises(TypeError):
        B.mxfp4_grouped_gemm(codes, scales, off, down, dtype=torch.float32)
    with pytest.raises(TypeError):
        B.mxfp4_dequantize(codes, scales, offsets=off, dtype=torch.float16)
    with pytest.raises(TypeError):
        B.mxfp4_dequantize(codes, None, offsets=off)
    with pytest.raises(TypeError):
        B.mxfp4_quantize(x, out=codes)
    with pytest.raises(ValueError):
        B.mxfp4_quantize(x, out=(codes,))
    with pytest.raises(TypeError):
        B.mxfp4_grouped_mlp_swiglu(x, off, up, down, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(B.SvdqError) as e:
        B.mxfp4_grouped_mlp_swiglu(x, off, up, down, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 1 and "workspace" in str(e.value)
    with pytest.raises(ValueError):
        B.mxfp4_quantize(x, stream=torch.cuda.Stream(), out=(codes[:, :8], scales))
    same_bits(B.mxfp4_grouped_mlp_swiglu(x, off, up, down), want)


def test_binding_keeps_no_references():
    """References to arguments and results are given back, by calls that
    succeed and by refused ones."""
    x, off, up, down = layer_set(4)
    y = torch.empty_like(x)
    out = B.mxfp4_quantize(x, offsets=off)
    objects = [x, off, y, up, down, up["codes"], up["scales"], down["codes"], down["scales"], out, *out]

    def calls():
        B.mxfp4_grouped_mlp_swiglu(x, off, up, down)
        assert B.mxfp4_grouped_mlp_swiglu(x, off, up, down, y=y) is y
        assert B.mxfp4_quantize(x, offsets=off, out=out)[0] is out[0]
        B.mxfp4_dequantize(*out, offsets=off)
        for bad in (lambda: B.mxfp4_grouped_linear(x, off, up), lambda: B.mxfp4_grouped_linear(x, off[:-1], down),
                    lambda: B.mxfp4_quantize(x, offsets=off, out=(out[0], out[0])),
                    lambda: B.mxfp4_grouped_mlp_swiglu(x, off, up, down, y=x[:3])):
            with pytest.raises((B.SvdqError, ValueError)):
                bad()

    calls()
    torch.cuda.synchronize()
    before, held = [sys.getrefcount(o) for o in objects], torch.cuda.memory_allocated()
    for _ in range(50):
        calls()
    torch.cuda.synchronize()
    assert [sys.getrefcount(o) for o in objects] == before
    assert torch.cuda.memory_allocated() == held
