"""MXFP4 without a GPU: the host pack and scale layouts against the oracle,
the oracle's pins, sizes, and every refusal that comes before a launch."""
import ctypes

import numpy as np
import pytest
import torch

import bit_w4a4_diffusion_b200 as B
from oracle import formats as F
from oracle import mxfp4 as O
from tests.helpers import nibbles

FAKE = 1 << 20   # never dereferenced: every call with it fails a check first


# ------------------------------------------------------------------ oracle --

def test_oracle_grid_points_are_fixed_points():
    """Values on the grid of a block whose largest is 4 or 6 times its scale
    are not changed."""
    for p in (-100, -3, 0, 7, 100):
        block = np.concatenate([F.E2M1_VALUE, F.E2M1_VALUE[::-1]]) * 2.0 ** p
        codes, scales = O.quantize(block[None])
        assert scales[0, 0] == 127 + p
        assert np.array_equal(np.abs(O.values(codes, scales)[0]), np.abs(block))


def test_oracle_brute_force():
    """Each code is the nearest grid value (even code on a tie) of v / scale."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((40, 64)).astype(np.float32)
    x[0, :32] = [i / 4 for i in range(32)]       # ties
    codes, scales = O.quantize(x)
    for r in range(40):
        for b in range(2):
            v = x[r, 32 * b:32 * b + 32].astype(np.float64)
            t = np.max(np.abs(v))
            s = 2.0 ** (np.floor(np.log2(t)) - 2)
            assert scales[r, b] == np.log2(s) + 127
            assert 4.0 <= t / s < 8.0
            for i in range(32):
                a = abs(v[i]) / s
                d = np.abs(F.E2M1_MAG - min(a, 6.0))
                best = np.flatnonzero(d == d.min())
                want = best[0] if len(best) == 1 else best[best % 2 == 0][0]
                assert codes[r, 32 * b + i] == want | (8 if np.signbit(v[i]) else 0)


def test_oracle_special_blocks():
    x = np.zeros((6, 32))
    x[1, 5] = np.nan
    x[2, 7] = -np.inf
    x[3, 0] = 2.0 ** -149                         # smallest fp32
    x[4, 0], x[4, 1] = 2.0 ** -126, -2.0 ** -128
    x[5, 0] = np.finfo(np.float32).max
    codes, scales = O.quantize(x)
    assert scales[:, 0].tolist() == [0, 255, 255, 0, 0, 252]
    assert not codes[:3].any()
    assert codes[3, 0] == 0                       # 2^-149 / 2^-127 rounds to 0
    assert O.values(codes, scales)[4, 0] == 2.0 ** -126 and O.values(codes, scales)[4, 1] == -2.0 ** -128
    assert codes[5, 0] == 7                       # just under 8 scales: saturates at 6


def test_oracle_fp64_encoder_agrees_with_the_fp32_one():
    u = np.concatenate([np.linspace(-8, 8, 4097), [-0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]])
    assert np.array_equal(O._encode64(u), F.e2m1_encode(u.astype(np.float32)))


# -------------------------------------------------------------------- pack --

@pytest.mark.parametrize("E,N,K", [(1, 1, 32), (1, 130, 160), (3, 40, 96), (2, 128, 256), (2, 257, 1056)])
def test_pack_weights_against_oracle(E, N, K):
    rng = np.random.default_rng(E * 1000 + N + K)
    W = rng.standard_normal((E, N, K)).astype(np.float32) * np.exp2(rng.integers(-30, 30, (E, N, 1)))
    W[0, 0, :32] = 0.0
    bits = F.bf16_bits(W)
    pk = B.mxfp4_pack_weights(bits)
    assert (pk["N"], pk["K"], pk["E"]) == (N, K, E)
    x = F.bf16_from_bits(bits).reshape(E, N, K)
    for e in range(E):
        codes, scales = O.quantize(x[e])
        assert np.array_equal(nibbles(pk["codes"][e]), codes)
        assert np.array_equal(pk["scales"][e], O.tile(scales, K))
        assert np.array_equal(B.mxfp4_scales_to_rowmajor(pk["scales"], N, K)[e], scales)
    row = np.stack([O.quantize(x[e])[1] for e in range(E)])
    assert np.array_equal(B.mxfp4_scales_from_rowmajor(row), pk["scales"])


def test_pack_weights_every_bf16_magnitude():
    """Every bf16 pattern, alone in its block and beside a larger value, NaN
    and infinity included."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    W = np.zeros((1 << 16, 64), np.uint16)
    W[:, 3] = bits
    W[:, 32] = bits
    W[:, 40] = np.where((bits & 0x7F80) < 0x7E00, (bits & 0x7F80) + 0x0100, bits)   # four times the power of two
    pk = B.mxfp4_pack_weights(W)
    codes, scales = O.quantize(F.bf16_from_bits(W.reshape(-1)).reshape(W.shape))
    assert np.array_equal(nibbles(pk["codes"]), codes)
    assert np.array_equal(B.mxfp4_scales_to_rowmajor(pk["scales"], 1 << 16, 64), scales)


def test_pack_refusals():
    with pytest.raises(B.SvdqError):
        B.mxfp4_pack_weights(np.zeros((4, 40), np.uint16))
    with pytest.raises(B.SvdqError):
        B.mxfp4_pack_weights(np.zeros((0, 32), np.uint16))
    assert B.lib.mxfp4_pack_weights(1, 8, 32, None, FAKE, FAKE) == 1
    assert B.lib.mxfp4_scales_to_rowmajor(1, 8, 48, FAKE, FAKE) == 2
    assert B.lib.mxfp4_scales_from_rowmajor(0, 8, 32, FAKE, FAKE) == 2
    with pytest.raises(B.SvdqError):
        B.mxfp4_scales_to_rowmajor(np.zeros(100, np.uint8), 8, 32)


# ------------------------------------------------------------------- sizes --

def test_sizes():
    assert B.mxfp4_scale_bytes(1, 32) == 512
    assert B.mxfp4_scale_bytes(129, 160) == 2 * 2 * 512
    assert B.mxfp4_scale_bytes(0, 32) == 0
    assert B.mxfp4_scale_bytes(300, 1024, groups=5) == (2 + 5) * 8 * 512
    assert B.mxfp4_scale_bytes(1, 48) == -1 and B.mxfp4_scale_bytes(-1, 32) == -1
    assert B.mxfp4_scale_bytes(1, 32, groups=513) == -1
    assert B.mxfp4_workspace_bytes(17, 32) == 512 + 512
    assert B.mxfp4_workspace_bytes(4, 32) == 0 and B.mxfp4_workspace_bytes(16, 32, groups=3) == 0
    assert B.mxfp4_mlp_workspace_bytes(4, 100, 64, 96) == (B.mxfp4_workspace_bytes(100, 64, 4) +
                                                           B.mxfp4_workspace_bytes(100, 96, 4))
    assert B.mxfp4_mlp_workspace_bytes(4, 8, 64, 96) == 512 + (4 * 512)
    assert B.mxfp4_mlp_workspace_bytes(0, 100, 64, 96) == -1


def test_sizes_agree_with_the_library():
    for rows in (0, 1, 4, 5, 16, 17, 127, 128, 129, 1000):
        for K in (32, 96, 128, 4128):
            assert B.mxfp4_scale_bytes(rows, K) == B.lib.mxfp4_scale_bytes(rows, K)
            for groups in (0, 1, 7, 512, 513, -1):
                assert B.mxfp4_workspace_bytes(rows, K, groups) == B.lib.mxfp4_workspace_bytes(groups, rows, K)
                if groups:
                    assert B.mxfp4_scale_bytes(rows, K, groups) == B.lib.mxfp4_grouped_scale_bytes(groups, rows, K)
                assert (B.mxfp4_mlp_workspace_bytes(groups, rows, K, 96) ==
                        B.lib.mxfp4_mlp_workspace_bytes(groups, rows, K, 96))
    for rows, K in ((-1, 32), (4, 33), (4, 0), (4, -32)):
        assert B.mxfp4_scale_bytes(rows, K) == B.lib.mxfp4_scale_bytes(rows, K) == -1


def test_grouped_blocks_never_meet():
    """The blocks of a group, from offsets[e] / 128 + e on, end before the
    next group's first, and the last within the buffer."""
    rng = np.random.default_rng(1)
    for _ in range(300):
        groups = int(rng.integers(1, 40))
        off = np.sort(rng.integers(0, 3000, groups + 1))
        rows = int(off[-1] + rng.integers(0, 200))
        for e in range(groups):
            end = off[e] // 128 + e + -(-(off[e + 1] - off[e]) // 128)
            assert end <= (off[e + 1] // 128 + e + 1 if e + 1 < groups else rows // 128 + groups)


# ---------------------------------------------------------------- refusals --

def _q(dtype=0, rows=4, K=64, x=FAKE, ldx=64, idx=None, x_rows=4, groups=0, off=None, codes=FAKE, scales=FAKE):
    return B.lib.mxfp4_quantize(dtype, rows, K, x, ldx, idx, x_rows, groups, off, codes, scales, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(K=40), 2), (dict(K=0), 2), (dict(rows=-1), 2), (dict(rows=(1 << 30) + 1), 2), (dict(groups=-1), 2),
    (dict(groups=513, off=FAKE), 2), (dict(groups=3), 1), (dict(off=FAKE), 1), (dict(groups=3, off=FAKE + 2), 1),
    (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(x=None), 1), (dict(x=FAKE + 8), 1), (dict(ldx=63), 1),
    (dict(ldx=68), 1), (dict(ldx=0), 1), (dict(ldx=-64), 1), (dict(dtype=2, ldx=66), 1), (dict(idx=FAKE + 1), 1),
    (dict(x_rows=3), 1), (dict(idx=FAKE, x_rows=-1), 1), (dict(codes=None), 1), (dict(scales=FAKE + 4), 1),
])
def test_quantize_refusals(kw, status):
    assert _q(**kw) == status, B.lib.svdq_last_error()
    assert B.lib.svdq_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=1), 1), (dict(K=33), 2), (dict(codes=None), 1), (dict(scales=None), 1), (dict(out=FAKE + 2), 1),
    (dict(ldo=32), 1), (dict(groups=2), 1), (dict(rows=-5), 2),
])
def test_dequantize_refusals(kw, status):
    a = dict(dtype=0, rows=4, K=64, codes=FAKE, scales=FAKE, groups=0, off=None, out=FAKE, ldo=64)
    a.update(kw)
    assert B.lib.mxfp4_dequantize(a["dtype"], a["rows"], a["K"], a["codes"], a["scales"], a["groups"], a["off"],
                                  a["out"], a["ldo"], None, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 1), (dict(N=12), 2), (dict(N=0), 2), (dict(K=16), 2), (dict(M=-1), 2), (dict(y=FAKE + 8), 1),
    (dict(ldy=8), 1), (dict(ldy=20), 1), (dict(bias=FAKE + 2), 1), (dict(w=None), 1), (dict(a=FAKE + 1), 1),
    (dict(ws=None), 1), (dict(sc=FAKE + 8), 1), (dict(N=1 << 30, K=1 << 20), 2),
])
def test_gemm_refusals(kw, status):
    a = dict(dtype=0, M=4, N=16, K=64, a=FAKE, sc=FAKE, w=FAKE, ws=FAKE, bias=None, y=FAKE, ldy=16)
    a.update(kw)
    assert B.lib.mxfp4_gemm(a["dtype"], a["M"], a["N"], a["K"], a["a"], a["sc"], a["w"], a["ws"], a["bias"], a["y"],
                            a["ldy"], None, None) == status, B.lib.svdq_last_error()


def _linear(groups=2, rows=70, N=16, K=64, x=FAKE, ldx=64, idx=None, x_rows=70, off=FAKE, ws=FAKE, ws_bytes=1 << 30,
            dtype=0, y=FAKE, ldy=16):
    return B.lib.mxfp4_grouped_linear(dtype, groups, rows, N, K, x, ldx, idx, x_rows, off, FAKE, FAKE, None, y, ldy,
                                      ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(groups=0, off=None), 2), (dict(groups=-2), 2), (dict(groups=600), 2), (dict(off=None), 1),
    (dict(x_rows=69), 1), (dict(ws=None), 1), (dict(ws_bytes=100), 1), (dict(ws=FAKE + 4), 1), (dict(N=4), 2),
    (dict(ldx=32), 1), (dict(y=None), 1), (dict(dtype=2), 1), (dict(groups=500, N=1 << 23), 2),
])
def test_grouped_linear_refusals(kw, status):
    assert _linear(**kw) == status, B.lib.svdq_last_error()


def test_workspace_message():
    assert B.lib.mxfp4_linear(0, 40, 16, 64, FAKE, 64, FAKE, FAKE, None, FAKE, 16, FAKE, 8, None, None) == 1
    assert b"workspace" in B.lib.svdq_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(I=40), 2), (dict(groups=0), 2), (dict(K=48), 2), (dict(up_bias=FAKE + 2), 1), (dict(ws_bytes=64), 1),
    (dict(up=None), 1), (dict(down=None), 1),
])
def test_mlp_refusals(kw, status):
    a = dict(groups=2, rows=4, K=64, I=96, up=FAKE, down=FAKE, up_bias=None, ws_bytes=1 << 30)
    a.update(kw)
    assert B.lib.mxfp4_grouped_mlp_swiglu(0, a["groups"], a["rows"], a["K"], a["I"], FAKE, 64, None, 4, FAKE, a["up"],
                                          FAKE, a["up_bias"], a["down"], FAKE, None, FAKE, 64, FAKE, a["ws_bytes"],
                                          None, None) == status, B.lib.svdq_last_error()


def test_swiglu_quant_refusals():
    def call(I=64, h=FAKE, hs=FAKE, groups=2, off=FAKE):
        return B.lib.mxfp4_grouped_gemm_swiglu_quant(0, groups, 4, I, 64, off, FAKE, FAKE, FAKE, FAKE, None, h, hs,
                                                     None, None)
    assert call(I=72) == 2 and call(h=None) == 1 and call(hs=FAKE + 8) == 1 and call(groups=0) == 2
    assert call(off=None) == 1


def test_no_rows_is_no_work():
    """rows == 0 returns before the device is looked for."""
    assert _q(rows=0, x=None, x_rows=0, codes=None, scales=None) == 0
    assert B.lib.mxfp4_gemm(0, 0, 16, 64, None, None, None, None, None, None, 16, None, None) == 0
    assert _linear(rows=0, x=None, x_rows=0, y=None, ws=None, ws_bytes=0) == 0


def test_python_argument_checks():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = {"codes": torch.zeros(16, 32, dtype=torch.uint8), "scales": torch.zeros(512, dtype=torch.uint8), "N": 16,
         "K": 64, "E": 1}
    off = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: B.mxfp4_quantize(x), lambda: B.mxfp4_linear(x, w), lambda: B.mxfp4_linear(x.float(), w),
                 lambda: B.mxfp4_grouped_linear(x, off, w), lambda: B.mxfp4_grouped_mlp_swiglu(x, off, w, w),
                 lambda: B.mxfp4_dequantize(w["codes"], w["scales"]), lambda: B.mxfp4_gemm(w["codes"], w["scales"], w),
                 lambda: B.mxfp4_quantize(None)):
        with pytest.raises(TypeError):
            call()


def test_header_and_binding_agree():
    assert ctypes.c_longlong(B.lib.mxfp4_scale_bytes(128, 128)).value == 512
    assert B.MXFP4_MAX_GROUPS == O.MAX_GROUPS
