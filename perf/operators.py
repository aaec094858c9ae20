"""What is measured of the MXFP4 operators: their cases, inputs, plain forms and exact values.

The operators work on the OCP microscaling format MXFP4: E2M1 elements that
share a power-of-two scale (E8M0, one byte) in blocks of 32 along K.

  quantize   x -> codes and scales, and back to the values they stand for
  linear     y = Q(x) deq(W)^T + b, both sides in MXFP4
  grouped    the same with one weight per expert, over rows sorted by expert
  mlp        down(SwiGLU(up(x))) per expert, the hidden rows in MXFP4 too

`own` selects the framework's calls; otherwise `run` computes the plain forms
from elementary torch operations in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

BLOCK = 32                       # elements that share one scale
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # A few rows in fp32 with an odd number of blocks: the tail of a batch.
        {"name": "quantize_7x1056_fp32", "op": "quantize", "M": 7, "K": 1056, "dtype": "fp32"},
        # The activations of one image or prompt of about a thousand tokens.
        {"name": "quantize_1001x4096_fp16", "op": "quantize", "M": 1001, "K": 4096, "dtype": "fp16"},
        # A whole weight, or the activations of a long packed batch.
        {"name": "quantize_16384x8192_bf16", "op": "quantize", "M": 16384, "K": 8192, "dtype": "bf16"},
        # One token through a square projection: the weight's bytes and the launch count.
        {"name": "linear_1_4096_4096", "op": "linear", "M": 1, "N": 4096, "K": 4096, "dtype": "bf16", "bias": False},
        # A small odd batch with odd widths: a text prompt through a projection.
        {"name": "linear_77_5000_2080", "op": "linear", "M": 77, "N": 5000, "K": 2080, "dtype": "fp16", "bias": True},
        # A long prompt through a large layer: bound by the tensor cores.
        {"name": "linear_8192_8192_8192", "op": "linear", "M": 8192, "N": 8192, "K": 8192, "dtype": "bf16",
         "bias": True},
        # Two tokens, four experts each of 32: most experts have no row.
        {"name": "grouped_2x4_of_32", "op": "grouped", "tokens": 2, "topk": 4, "E": 32, "N": 2048, "K": 2048,
         "dtype": "bf16", "bias": False, "gather": True},
        # A short prompt over few experts, odd widths, rows already in order.
        {"name": "grouped_555x2_of_12", "op": "grouped", "tokens": 555, "topk": 2, "E": 12, "N": 1544, "K": 1440,
         "dtype": "bf16", "bias": True, "gather": False},
        # A long batch over many experts.
        {"name": "grouped_8192x4_of_64", "op": "grouped", "tokens": 8192, "topk": 4, "E": 64, "N": 4096, "K": 2048,
         "dtype": "bf16", "bias": False, "gather": True},
        # One token through the experts' MLP: each chosen expert's weights once.
        {"name": "mlp_1x8_of_64", "op": "mlp", "tokens": 1, "topk": 8, "E": 64, "K": 2048, "I": 1024,
         "dtype": "bf16", "bias": False, "gather": True},
        # A served batch: a few dozen rows per expert.
        {"name": "mlp_300x4_of_32", "op": "mlp", "tokens": 300, "topk": 4, "E": 32, "K": 2080, "I": 1440,
         "dtype": "fp16", "bias": True, "gather": True},
        # A long batch through large experts: bound by the tensor cores.
        {"name": "mlp_8192x2_of_16", "op": "mlp", "tokens": 8192, "topk": 2, "E": 16, "K": 4096, "I": 2048,
         "dtype": "bf16", "bias": False, "gather": True},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["quantize", "linear", "grouped", "mlp"])
    if op == "quantize":
        return {"op": op, "M": _spread(rng, 1, 16384), "K": _spread(rng, 32, 8192, 32),
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    dtype, bias = rng.choice(["bf16", "fp16"]), rng.random() < 0.5
    if op == "linear":
        return {"op": op, "M": _spread(rng, 1, 8192), "N": _spread(rng, 8, 8192, 8), "K": _spread(rng, 32, 8192, 32),
                "dtype": dtype, "bias": bias}
    E = _spread(rng, 2, 64)
    topk = rng.randint(1, min(8, E))
    case = {"op": op, "tokens": _spread(rng, 1, 16384 // topk), "topk": topk, "E": E, "dtype": dtype, "bias": bias,
            "gather": rng.random() < 0.5}
    if op == "grouped":
        case.update(N=_spread(rng, 64, 4096, 8), K=_spread(rng, 64, 2048, 32))
    else:
        case.update(K=_spread(rng, 64, 2048, 32), I=_spread(rng, 64, 1024, 32))
    return case


# ------------------------------------------------------------------ inputs ---

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(g, rows, K, dtype):
    """Normal values with a few large channels, as hidden states have them."""
    x = torch.randn(rows, K, generator=g, device="cuda")
    x *= torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x.to(DTYPES[dtype])


def _tile_scales(scales):
    """Row-major scales [B, N, K/32] -> the tiled layout of the block-scaled
    product: 512-byte tiles of 128 rows x 4 blocks, both padded with zeros."""
    B, N, G = scales.shape
    n, g = -(-N // 128) * 128, -(-G // 4) * 4
    padded = torch.zeros(B, n, g, dtype=torch.uint8, device=scales.device)
    padded[:, :N, :G] = scales
    tiles = padded.view(B, n // 128, 4, 32, g // 4, 4).permute(0, 1, 4, 3, 2, 5)
    return tiles.reshape(B, -1).contiguous()


def _weight(g, B, N, K):
    """B weights [N, K], quantized: codes, scales, and the scales laid out
    once for the product (as a program that loads a checkpoint does)."""
    w = torch.randn(B, N, K, generator=g, device="cuda") * (1.0 / math.sqrt(K))
    codes, scales = _plain_quantize(w)
    return {"codes": codes, "rowmajor": scales, "scales": _tile_scales(scales), "N": N, "K": K, "E": B}


def _bias(g, shape, dtype, wanted):
    return (torch.randn(*shape, generator=g, device="cuda") * 0.1).to(dtype) if wanted else None


def prepare(case, seed):
    g = _generator(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    state = {"op": op, "dtype": dtype}
    if op == "quantize":
        state["x"] = _activations(g, case["M"], case["K"], case["dtype"])
        return state
    if op == "linear":
        state["x"] = _activations(g, case["M"], case["K"], case["dtype"])
        w = _weight(g, 1, case["N"], case["K"])
        state["w"] = {**w, "codes": w["codes"][0], "rowmajor": w["rowmajor"][0], "scales": w["scales"][0]}
        state["bias"] = _bias(g, (case["N"],), dtype, case["bias"])
        return state
    # A router's choice: topk different experts per token, some of them more
    # often than others; the rows in the order of their experts.
    T, topk, E = case["tokens"], case["topk"], case["E"]
    logits = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
    chosen = logits.topk(topk, dim=1).indices.reshape(-1)
    counts = torch.bincount(chosen, minlength=E)
    state["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    state["most"] = int(counts.max())
    x = _activations(g, T, case["K"], case["dtype"])
    rows = (torch.argsort(chosen, stable=True) // topk).to(torch.int32)
    state["row_index"] = rows if case["gather"] else None
    state["x"] = x if case["gather"] else x[rows.long()]
    if op == "grouped":
        state["w"] = _weight(g, E, case["N"], case["K"])
        state["bias"] = _bias(g, (E, case["N"]), dtype, case["bias"])
    else:
        # up: two matrices [I, K] per expert, the gate and the other factor
        state["up"] = _weight(g, 2 * E, case["I"], case["K"])
        state["down"] = _weight(g, E, case["K"], case["I"])
        state["up_bias"] = _bias(g, (E, 2 * case["I"]), dtype, case["bias"])
        state["down_bias"] = _bias(g, (E, case["K"]), dtype, case["bias"])
    return state


# ------------------------------------------------------------- plain forms ---

_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _plain_quantize(x):
    """Codes (two per byte, the even element in the low half) and E8M0 scales
    of x [..., K]: the scale of a block is 2^(floor(log2 max|x|) - 2), no less
    than 2^-127; each element over it goes to the nearest of E2M1, a tie to
    the even one, at most 6."""
    v = x.float().reshape(*x.shape[:-1], -1, BLOCK)
    top = v.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(min=-127)
    u = torch.ldexp(v, -e)
    a = u.abs()
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + torch.signbit(u) * 8).to(torch.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e[..., 0] + 127).to(torch.uint8)


def _plain_values(codes, scales):
    """The values, in 32 bits, that codes and scales stand for."""
    table = torch.tensor(_VALUES + tuple(-v for v in _VALUES), device=codes.device)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1)
    v = v.reshape(*scales.shape, BLOCK)
    return torch.ldexp(v, scales.int()[..., None] - 127).reshape(*codes.shape[:-1], -1)


def _plain_rounded(x):
    return _plain_values(*_plain_quantize(x))


def _plain_groups(state):
    """The expert of each row and the row's place among that expert's rows."""
    off = state["offsets"].long()
    rows = state["row_index"].numel() if state["row_index"] is not None else state["x"].shape[0]
    row = torch.arange(rows, device=off.device)
    expert = torch.searchsorted(off, row, right=True) - 1
    return expert, row - off[expert]


def _plain_experts(x, w, E, expert, place, most, bias):
    """Each row of x [R, K] (32 bits) times its own expert's weight (all the
    matrices of an expert one below the other)."""
    padded = x.new_zeros(E, most, x.shape[1])
    padded[expert, place] = _plain_rounded(x)
    values = _plain_values(w["codes"], w["rowmajor"]).view(E, -1, x.shape[1])
    y = torch.bmm(padded, values.transpose(1, 2))[expert, place]
    return y if bias is None else y + bias.float()[expert]


def _plain(state):
    op = state["op"]
    if op == "quantize":
        codes, scales = _plain_quantize(state["x"])
        return {"values": _plain_values(codes, scales).to(torch.bfloat16)}
    if op == "linear":
        w = state["w"]
        y = _plain_rounded(state["x"]) @ _plain_values(w["codes"], w["rowmajor"]).t()
        y = y if state["bias"] is None else y + state["bias"].float()
        return {"y": y.to(state["dtype"])}
    expert, place = _plain_groups(state)
    E = state["offsets"].numel() - 1
    x = state["x"].float() if state["row_index"] is None else state["x"].float()[state["row_index"].long()]
    if op == "grouped":
        y = _plain_experts(x, state["w"], E, expert, place, state["most"], state["bias"])
        return {"y": y.to(state["dtype"])}
    both = _plain_experts(x, state["up"], E, expert, place, state["most"], state["up_bias"])
    gate, other = both.chunk(2, 1)
    h = gate / (1.0 + torch.exp(-gate)) * other
    y = _plain_experts(h, state["down"], E, expert, place, state["most"], state["down_bias"])
    return {"y": y.to(state["dtype"])}


# ------------------------------------------------------------------- calls ---

def run(state):
    if not own:
        return _plain(state)
    import bit_w4a4_diffusion_b200 as B
    op = state["op"]
    if op == "quantize":
        return {"values": B.mxfp4_dequantize(*B.mxfp4_quantize(state["x"]))}
    if op == "linear":
        return {"y": B.mxfp4_linear(state["x"], state["w"], bias=state["bias"])}
    if op == "grouped":
        return {"y": B.mxfp4_grouped_linear(state["x"], state["offsets"], state["w"], row_index=state["row_index"],
                                            bias=state["bias"])}
    return {"y": B.mxfp4_grouped_mlp_swiglu(state["x"], state["offsets"], state["up"], state["down"],
                                            row_index=state["row_index"], up_bias=state["up_bias"],
                                            down_bias=state["down_bias"])}


# -------------------------------------------------------------------- work ---

def _quantized_bytes(rows, K):
    return rows * (K / 2 + K / 32)


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    op, K = case["op"], case["K"]
    if op == "quantize":
        M = case["M"]
        # x in; codes and scales out and in again; the values (bf16) out
        return {"bytes": M * K * size + 2 * _quantized_bytes(M, K) + M * K * 2, "flops": M * K * 4}
    if op == "linear":
        M, N = case["M"], case["N"]
        return {"bytes": M * K * size + _quantized_bytes(N, K) + M * N * size + (N * size if case["bias"] else 0),
                "flops": 2 * M * N * K}
    T, E = case["tokens"], case["E"]
    rows = T * case["topk"]
    used = E * (1.0 - (1.0 - case["topk"] / E) ** T)     # experts with rows, where all are chosen alike
    x = (T if case["gather"] else rows) * K * size + rows * 4
    if op == "grouped":
        N = case["N"]
        return {"bytes": x + used * _quantized_bytes(N, K) + rows * N * size, "flops": 2 * rows * N * K}
    width = case["I"]
    return {"bytes": x + used * (_quantized_bytes(2 * width, K) + _quantized_bytes(K, width)) + rows * K * size,
            "flops": 6 * rows * K * width}


# ------------------------------------------------------------------- exact ---

def _exact_values64(x):
    """x [..., K] rounded to MXFP4, in 64 bits, by the format's definition:
    the spacing of E2M1 is 1/2 below 2, 1 from 2 to 4 and 2 above."""
    shape = x.shape
    v = x.double().reshape(-1, BLOCK)
    top = v.abs().max(dim=1, keepdim=True).values
    # frexp: top = m 2^e with m in [1/2, 1), so floor(log2(top)) = e - 1
    scale = torch.ldexp(torch.ones_like(top), (torch.frexp(top).exponent - 3).clamp(min=-127))
    scale[top == 0] = 2.0 ** -127
    a = v.abs() / scale
    step = torch.full_like(a, 0.5)
    step[a >= 2] = 1.0
    step[a >= 4] = 2.0
    a = torch.round(a / step).mul_(step).clamp_(max=6.0)      # torch.round: ties to even
    return (torch.copysign(a, v) * scale).reshape(shape)


def _exact_weight64(codes, scales):
    """A weight [N, K] from its codes and scales, in 64 bits."""
    both = torch.stack([codes.int() % 16, codes.int() // 16], dim=2).flatten(1)
    mag, sign = both % 8, 1 - 2 * (both // 8)
    exponent, mantissa = mag // 2, mag % 2
    v = torch.where(exponent == 0, mantissa * 0.5, (1 + mantissa * 0.5) * torch.exp2((exponent - 1).double()))
    scale = torch.ldexp(torch.ones_like(scales, dtype=torch.float64), scales.int() - 127)
    return sign * v * scale.repeat_interleave(BLOCK, dim=1)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return {"values": torch.cat([_exact_values64(part) for part in state["x"].split(2048)])}
    if op == "linear":
        w = state["w"]
        y = _exact_values64(state["x"]) @ _exact_weight64(w["codes"], w["rowmajor"]).t()
        return {"y": y if state["bias"] is None else y + state["bias"].double()}
    x = state["x"].double() if state["row_index"] is None else state["x"].double()[state["row_index"].long()]
    off = state["offsets"].tolist()

    def expert_product(h, w, bias, e):
        codes, scales = (w[k].view(case["E"], -1, w[k].shape[-1])[e] for k in ("codes", "rowmajor"))
        y = _exact_values64(h) @ _exact_weight64(codes, scales).t()
        return y if bias is None else y + bias[e].double()

    parts = []
    for e in range(case["E"]):
        h = x[off[e]:off[e + 1]]
        if h.shape[0] == 0:
            continue
        if op == "grouped":
            parts.append(expert_product(h, state["w"], state["bias"], e))
            continue
        h = expert_product(h, state["up"], state["up_bias"], e)
        h = h[:, :case["I"]] * torch.sigmoid(h[:, :case["I"]]) * h[:, case["I"]:]
        parts.append(expert_product(h, state["down"], state["down_bias"], e))
    return {"y": torch.cat(parts)}
