"""MXFP4 operators on the GPU where they could go wrong unnoticed: the ends of
the range, waits beside a slow kernel."""
import time

import numpy as np
import pytest
import torch

import bit_w4a4_diffusion_b200 as B
from oracle import formats as F
from oracle import mxfp4 as O
from tests import mxfp4_cases as C
from tests.helpers import nibbles

pytestmark = pytest.mark.gpu


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


# ------------------------------------------------------------------ SwiGLU --

@pytest.mark.parametrize("kernel", ["pair", "narrow"])
@pytest.mark.parametrize("rows,K", [(70, 32), (5, 1024), (300, 96)])
def test_swiglu_of_gates_whose_exponential_leaves_the_range(monkeypatch, kernel, rows, K):
    """Gates around -87.3, where exp(-g) passes 2^126, and -88.7, where it
    passes the largest fp32 value: h = g sigmoid(g) u is then far from zero if u
    is large.  Error of h: as in the ordinary range (exp's argument |g| 2^-24,
    the exponential, the quotient and the products 2^-21 each), and that of an
    exponential below 2^-126, whose last place is 2^-149: a few of them times
    |g u|."""
    monkeypatch.setenv("SVDQ_MXFP4_GEMM_KERNEL", kernel)
    rng = np.random.default_rng(rows)
    width = 512
    # x is 1 everywhere; a gate is minus the sum of 32 weights out of 1.5 .. 4
    codes = np.zeros((2, width, K), np.uint8)
    codes[0, :, :32] = 8 + rng.integers(3, 7, (width, 32))
    codes[0] = codes[0][np.argsort(O.values(codes[0], np.full((width, K // 32), 127)).sum(1))]   # like values in a block
    codes[1, :, 0] = rng.integers(4, 8, width)
    codes[1, :, 0] |= (8 * rng.integers(0, 2, width)).astype(np.uint8)
    scales = np.full((2, width, K // 32), 127, np.uint8)
    scales[1] = 127 + 90
    w = {"codes": cuda(O.pack(codes)), "scales": cuda(np.stack([O.tile(s, K) for s in scales])), "N": width, "K": K,
         "E": 2}
    off = cuda([0, rows], torch.int32)
    q = B.mxfp4_quantize(torch.ones(rows, K, dtype=torch.bfloat16, device="cuda"), offsets=off)
    hc, hs = B.mxfp4_grouped_gemm_swiglu_quant(*q, off, w)
    got_c, got_s = nibbles(hc.cpu().numpy()), B.mxfp4_scales_to_rowmajor(hs.cpu().numpy()[:B.mxfp4_scale_bytes(rows, width)],
                                                                         rows, width)
    g, u = (O.values(codes[i], scales[i]).sum(1) for i in (0, 1))
    assert (g < -89).sum() > 50 and ((g > -88.5) & (g < -87.5)).sum() > 10 and (g > -87).sum() > 50
    h = O.swiglu(g, u)
    delta = np.abs(h) * (np.abs(g) * 2.0 ** -23 + 2.0 ** -19) + np.abs(g * u) * 2.0 ** -147
    top = lambda v: np.max(v.reshape(-1, 32), axis=1)                 # noqa: E731
    byte = lambda t: np.maximum(np.frexp(t)[1] - 3, -127) + 127       # noqa: E731
    lo, hi = byte(np.maximum(top(np.abs(h) - delta), 0)), byte(top(np.abs(h) + delta))
    assert ((got_s >= lo) & (got_s <= hi)).all()
    s = np.repeat(np.ldexp(1.0, got_s.astype(np.int64) - 127), 32, axis=1)
    low, high = (F.E2M1_VALUE[O._encode64((h + d) / s)] for d in (-delta, delta))
    got = F.e2m1_decode(got_c)
    assert ((got >= low) & (got <= high)).all()


# ------------------------------------------------------- -------------- waits --

def random_weight(lead, N, K, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    E = int(np.prod(lead))
    return {"codes": torch.randint(0, 256, (*lead, N, K // 2), dtype=torch.uint8, device="cuda", generator=g),
            "scales": torch.randint(110, 118, (*lead, B.mxfp4_scale_bytes(N, K)), dtype=torch.uint8, device="cuda",
                                    generator=g), "N": N, "K": K, "E": E}


def test_waiting_for_the_kernel_before_is_no_timeout():
    """The products of an MLP start while the kernels before them still run.
    Here the quantizer takes long: its rows come from pinned host memory, over
    a link that a copy keeps busy (0.3 ms).  The products must not count that
    against the limit of their own waits, which take a few microseconds."""
    E, rows, K, width = 2, 128, 32768, 256
    x = C.rows(np.random.default_rng(0), rows, K, torch.bfloat16)
    off = cuda([0, 80, rows], torch.int32)
    up, down = random_weight((E, 2), width, K), random_weight((E,), K, width, 1)
    want = B.mxfp4_grouped_mlp_swiglu(x.cuda(), off, up, down)
    host = x.pin_memory()
    y = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.mxfp4_mlp_workspace_bytes(E, rows, K, width), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream, other = torch.cuda.current_stream().cuda_stream, torch.cuda.Stream()
    src, dst = torch.empty(1 << 29, dtype=torch.uint8, pin_memory=True), torch.empty(1 << 29, dtype=torch.uint8, device="cuda")
    old = B.get_timeout_ns()
    try:
        B.set_timeout_ns(4000)
        for _ in range(3):
            torch.cuda.synchronize()
            with torch.cuda.stream(other):
                dst.copy_(src, non_blocking=True)     # 10 ms
            time.sleep(0.002)
            assert B.lib.mxfp4_grouped_mlp_swiglu(
                0, E, rows, K, width, host.data_ptr(), K, None, rows, off.data_ptr(), up["codes"].data_ptr(),
                up["scales"].data_ptr(), None, down["codes"].data_ptr(), down["scales"].data_ptr(), None, y.data_ptr(),
                K, ws.data_ptr(), ws.numel(), status.data_ptr(), stream) == 0
            torch.cuda.synchronize()
            assert int(status) == 0
            assert torch.equal(y, want)
    finally:
        B.set_timeout_ns(old)
