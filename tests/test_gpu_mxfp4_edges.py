"""MXFP4 operators on the GPU where they could go wrong unnoticed: the ends of
the range, waits beside a slow kernel, a second driver context; and what the
smoke run reaches."""
import os
import subprocess
import sys
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

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


# ---------------------------------------------------------------- contexts --

CONTEXTS = r"""
import ctypes, os, sys
import numpy as np
sys.path.insert(0, sys.argv[1])
import bit_w4a4_diffusion_b200 as B
from oracle import mxfp4 as O
from tests import mxfp4_cases as C

cu = ctypes.CDLL("libcuda.so.1")
def ok(e): assert e == 0, f"driver error {e}"
def lib(e): assert e == 0, (e, B.lib.svdq_last_error())
ok(cu.cuInit(0))
held = []
def put(a):
    a = np.ascontiguousarray(a)
    p = ctypes.c_uint64()
    ok(cu.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(a.nbytes)))
    ok(cu.cuMemcpyHtoD_v2(p, a.ctypes.data_as(ctypes.c_void_p), ctypes.c_size_t(a.nbytes)))
    held.append(p)
    return p.value
def get(p, shape, dtype):
    a = np.empty(shape, dtype)
    ok(cu.cuCtxSynchronize())
    ok(cu.cuMemcpyDtoH_v2(a.ctypes.data_as(ctypes.c_void_p), ctypes.c_uint64(p), ctypes.c_size_t(a.nbytes)))
    return a

rng = np.random.default_rng(0)
M, N, K = 300, 256, 320
a, sa = C.operand(rng, M, K, -3)
w, sw = C.operand(rng, N, K, -2)
want = C.rounded(O.product(O.values(a, sa), O.values(w, sw)), C.torch.bfloat16).view(C.torch.int16).numpy()
vals = O.values(a, sa).astype(np.float32)
off = np.array([0, M], np.int32)

def run():
    '''Every kernel that asks for more shared memory than it gets by itself.'''
    qa, qs, dw, ds, do = put(O.pack(a)), put(O.tile(sa, K)), put(O.pack(w)), put(O.tile(sw, K)), put(off)
    y = put(np.zeros((M, N), np.int16))
    for kernel in ("narrow", "pair256", "pair384"):
        os.environ["SVDQ_MXFP4_GEMM_KERNEL"] = kernel
        lib(B.lib.mxfp4_gemm(0, M, N, K, qa, qs, dw, ds, None, y, N, None, None))
        assert np.array_equal(get(y, (M, N), np.int16), want), kernel
    h = []
    gs = put(np.zeros(B.mxfp4_scale_bytes(M, K, 1), np.uint8))
    x, codes = put(vals), put(np.zeros((M, K // 2), np.uint8))
    lib(B.lib.mxfp4_quantize(2, M, K, x, K, None, M, 1, do, codes, gs, None, None))
    for kernel in ("narrow", "pair"):
        os.environ["SVDQ_MXFP4_GEMM_KERNEL"] = kernel
        hc, hs = put(np.zeros((M, N // 4), np.uint8)), put(np.zeros(B.mxfp4_scale_bytes(M, N // 2, 1), np.uint8))
        lib(B.lib.mxfp4_grouped_gemm_swiglu_quant(0, 1, M, N // 2, K, do, codes, gs, dw, put(np.concatenate(
            [O.tile(s, K) for s in (sw[:N // 2], sw[N // 2:])])), None, hc, hs, None, None))
        h.append(get(hc, (M, N // 4), np.uint8))
    assert np.array_equal(h[0], h[1]) and h[0].any()
    del os.environ["SVDQ_MXFP4_GEMM_KERNEL"]
    lib(B.lib.mxfp4_linear(0, 4, N, K, put((vals.view(np.uint32)[:4] >> 16).astype(np.uint16)), K, dw, ds, None, y, N,
                           None, 0, None, None))
    out = put(np.zeros((M, K), np.float32))
    lib(B.lib.mxfp4_dequantize(2, M, K, qa, qs, 0, None, out, K, None, None))
    assert np.array_equal(get(out, (M, K), np.float32), vals)

dev = ctypes.c_int()
ok(cu.cuDeviceGet(ctypes.byref(dev), 0))
ctxs = []
for _ in range(2):
    c = ctypes.c_void_p()
    ok(cu.cuCtxCreate_v2(ctypes.byref(c), 0, dev))
    ctxs.append(c)
for c in (ctxs[0], ctxs[1], ctxs[0]):
    ok(cu.cuCtxSetCurrent(c))
    run()
for c in ctxs:
    ok(cu.cuCtxDestroy_v2(c))
print("contexts ok")
"""


def test_calls_in_two_driver_contexts():
    """What a kernel was granted in one context of a device does not hold in
    another (or after a reset): every call looks at the context it is in."""
    r = subprocess.run([sys.executable, "-c", CONTEXTS, ROOT], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "contexts ok" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]


# ------------------------------------------------------------ stream handles --

@pytest.mark.parametrize("handle", [0, 1, None])
def test_the_default_stream_by_its_handle(handle):
    """stream=0, which is what torch.cuda.current_stream().cuda_stream mostly is
    (or 1, the default stream's other handle): behind the work that is queued
    there, before the work that follows."""
    if handle is None:
        handle = torch.cuda.current_stream().cuda_stream
        assert handle == 0
    rng = np.random.default_rng(3)
    w = random_weight((), 264, 320)
    xs = [C.rows(rng, 40, 320, torch.bfloat16).cuda() for _ in range(2)]
    want = [B.mxfp4_linear(x, w) for x in xs]
    x, y = torch.empty_like(xs[0]), torch.empty_like(want[0])
    busy = torch.randn(4096, 4096, device="cuda")
    got = []
    for i in range(6):
        torch.mm(busy, busy)                          # the copy waits for it
        x.copy_(xs[i % 2])
        assert B.mxfp4_linear(x, w, y=y, stream=handle) is y
        got.append(y.clone())
        got.append(B.mxfp4_linear(x, w, stream=handle).clone())
    for i, g in enumerate(got):
        assert torch.equal(g, want[i // 2 % 2]), i


# ----------------------------------------------------------------- repeats --

@pytest.mark.parametrize("T,E,K,width", [(1, 6, 256, 128), (40, 6, 1312, 96), (300, 20, 896, 960), (2000, 3, 320, 1312)])
def test_layers_repeat_bit_for_bit(T, E, K, width):
    """Whatever the memory that a call gets held before: NaN bytes, large and
    small values, what another call left."""
    rng = np.random.default_rng(T)
    x, other = (C.rows(rng, T, K, torch.bfloat16).cuda() for _ in range(2))
    rows = 2 * T
    off = cuda(np.concatenate([[0], np.sort(rng.integers(0, rows, E - 1)), [rows]]), torch.int32)
    index = cuda(rng.integers(0, T, rows), torch.int32)
    w, up, down = random_weight((E,), width, K), random_weight((E, 2), width, K), random_weight((E,), K, width)
    one = {**w, "codes": w["codes"][0], "scales": w["scales"][0], "E": 1}

    def calls(x):
        return (B.mxfp4_linear(x, one), B.mxfp4_grouped_linear(x, off, w, row_index=index),
                B.mxfp4_grouped_mlp_swiglu(x, off, up, down, row_index=index))

    first = calls(x)
    for fill in (0xFF, 0x7F, 0x01, None, 0xF5):
        if fill is None:
            calls(other)
        else:
            blocks = [torch.full((1 << n,), fill, dtype=torch.uint8, device="cuda") for n in range(9, 26) for _ in (0, 1)]
            del blocks
        for got, want in zip(calls(x), first):
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))


# ------------------------------------------------------- codes and padding --

@pytest.mark.parametrize("kernel", ["pair256", "pair384", "narrow"])
def test_every_code_pair_at_every_place(monkeypatch, kernel):
    """One-element rows: at each of the 256 places of a K slice all 256 pairs
    of E2M1 codes, scales over a wide range.  Row n of the weight and row n of
    the activations have their element at k = n; others meet in no place."""
    monkeypatch.setenv("SVDQ_MXFP4_GEMM_KERNEL", kernel)
    K, at = 256, np.arange(256)
    rng = np.random.default_rng(0)
    sa, sw = ((127 + rng.integers(-40, 41, (256, 8))).astype(np.uint8) for _ in range(2))
    da, dw = cuda(O.tile(sa, K)), cuda(O.tile(sw, K))
    scale = np.ldexp(1.0, sa[at, at // 32].astype(np.int64) + sw[at, at // 32] - 254)
    got, want = [], []
    for shift in range(256):
        pair = (at + shift) % 256
        a, w = np.zeros((2, 256, K), np.uint8)
        a[at, at], w[at, at] = pair % 16, pair // 16
        y = B.mxfp4_gemm(cuda(O.pack(a)), da, {"codes": cuda(O.pack(w)), "scales": dw, "N": 256, "K": K})
        got.append(y)
        want.append(np.diag(F.E2M1_VALUE[pair % 16] * F.E2M1_VALUE[pair // 16] * scale))
    got = torch.stack(got).double().cpu()              # at most 6 significant bits: exact in bf16
    assert torch.equal(got, torch.from_numpy(np.stack(want)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 32), (5, 96), (33, 160), (128, 1056), (129, 320), (300, 2080)])
def test_quantizer_writes_zero_padding(M, K, dtype):
    """Scale bytes of the blocks past K are 0 in every real row, whatever the
    buffer held, of a whole matrix and of row groups."""
    x = C.rows(np.random.default_rng(M), M, K, dtype).cuda()
    codes = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda")
    want = O.quantize(x.double().cpu().numpy())[1]
    padded = -(-K // 128) * 4
    r, g = np.meshgrid(np.arange(M), np.arange(padded), indexing="ij")
    full = np.zeros((M, padded), np.uint8)
    full[:, :K // 32] = want
    scales = torch.full((B.mxfp4_scale_bytes(M, K),), 0xFF, dtype=torch.uint8, device="cuda")
    B.mxfp4_quantize(x, out=(codes, scales))
    assert np.array_equal(scales.cpu().numpy()[O.scale_place(r, g, K)], full)
    off = [0, 0, M // 3, M // 2, M]
    scales = torch.full((B.mxfp4_scale_bytes(M, K, 4),), 0xFF, dtype=torch.uint8, device="cuda")
    B.mxfp4_quantize(x, offsets=cuda(off, torch.int32), out=(codes, scales))
    got = scales.cpu().numpy()
    for e in range(4):
        rows = r[:off[e + 1] - off[e]]
        at = (off[e] // 128 + e) * (padded // 4) * 512 + O.scale_place(rows, g[:len(rows)], K)
        assert np.array_equal(got[at], full[off[e]:off[e + 1]])


def test_wrong_tensors_are_refused():
    """Types, devices and sizes of CUDA tensors, one wrong at a time."""
    x = torch.zeros(20, 64, dtype=torch.bfloat16, device="cuda")
    off = cuda([0, 12, 20], torch.int32)
    w = random_weight((2,), 32, 64)
    up = random_weight((2, 2), 32, 64)
    down = random_weight((2,), 64, 32)
    one = {**w, "codes": w["codes"][0], "scales": w["scales"][0], "E": 1}
    codes, scales = B.mxfp4_quantize(x)
    index = torch.zeros(20, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def calls(x=x, off=off, w=w, up=up, down=down, one=one, codes=codes, scales=scales, index=index, status=status):
        return [lambda: B.mxfp4_quantize(x, offsets=off, row_index=index, dev_status=status),
                lambda: B.mxfp4_dequantize(codes, scales, dev_status=status),
                lambda: B.mxfp4_gemm(codes, scales, one, dev_status=status),
                lambda: B.mxfp4_linear(x, one, dev_status=status),
                lambda: B.mxfp4_grouped_linear(x, off, w, row_index=index, dev_status=status),
                lambda: B.mxfp4_grouped_mlp_swiglu(x, off, up, down, row_index=index, dev_status=status)]

    for call in calls():
        call()
    quantize, dequantize, gemm, linear, grouped, mlp = range(6)
    as_int8 = lambda t: {**t, "codes": t["codes"].view(torch.int8)}       # noqa: E731
    on_host = lambda t: {**t, "scales": t["scales"].cpu()}                # noqa: E731
    short = lambda t: {**t, "scales": t["scales"].reshape(-1)[:-1]}       # noqa: E731
    wider = lambda t: {**t, "N": t["N"] + 8}                              # noqa: E731
    for kw, which, error in [
            (dict(x=x.double()), (quantize, linear, grouped, mlp), TypeError),
            (dict(x=x.float()), (linear, grouped, mlp), TypeError),
            (dict(x=x.cpu()), (quantize, linear, grouped, mlp), TypeError),
            (dict(x=x[0]), (quantize, linear, grouped, mlp), TypeError),
            (dict(off=off.long()), (quantize, grouped, mlp), TypeError),
            (dict(off=off.cpu()), (quantize, grouped, mlp), TypeError),
            (dict(off=off[:1]), (quantize, grouped, mlp), TypeError),
            (dict(index=index.long()), (quantize, grouped, mlp), TypeError),
            (dict(index=index.cpu()), (quantize, grouped, mlp), TypeError),
            (dict(codes=codes.view(torch.int8)), (dequantize, gemm), TypeError),
            (dict(scales=scales.view(torch.int8)), (dequantize, gemm), TypeError),
            (dict(scales=scales[:-1]), (dequantize, gemm), ValueError),
            (dict(one=as_int8(one), w=as_int8(w), up=as_int8(up)), (gemm, linear, grouped, mlp), TypeError),
            (dict(one=on_host(one), w=on_host(w), down=on_host(down)), (gemm, linear, grouped, mlp), TypeError),
            (dict(one=short(one), w=short(w), down=short(down)), (gemm, linear, grouped, mlp), ValueError),
            (dict(one=wider(one), w=wider(w), up=wider(up)), (gemm, linear, grouped, mlp), ValueError),
            (dict(w={**w, "E": 3}, up={**up, "E": 2}), (grouped, mlp), B.SvdqError),
            (dict(status=status.float()), range(6), TypeError),
            (dict(status=status.cpu()), range(6), TypeError)]:
        for i in which:
            with pytest.raises(error):
                calls(**kw)[i]()
    for call in calls():
        call()
    assert int(status) == 0


# ------------------------------------------------------------------- smoke --

def test_smoke_reaches_every_mxfp4_product():
    """The smoke run launches the narrow and the pair kernel of both products."""
    import __graft_entry__ as entry
    from torch.profiler import ProfilerActivity, profile
    with profile(activities=[ProfilerActivity.CUDA], acc_events=True) as prof:
        entry.smoke()
        torch.cuda.synchronize()
    names = " ".join(e.key for e in prof.key_averages())
    if "_kernel" not in names:
        pytest.skip("no kernels in the profile: another tool holds the profiling interface")
    for kernel in ("mxfp4_quantize_kernel", "mxfp4_gemm_narrow_kernel", "mxfp4_gemm_pair_kernel",
                   "mxfp4_gemm_pair_swiglu_kernel"):
        assert kernel in names, kernel
