"""Constants of the MXFP4 part of include/svdq.h, in Python and in the library."""
import os
import re

import bit_w4a4_diffusion_b200 as B
from oracle import mxfp4 as O

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "svdq.h")


def defines():
    return {name: int(value) for name, value in re.findall(r"^#define\s+(\w+)\s+(\d+)\b", open(HEADER).read(), re.M)}


def test_binding_has_the_header_s_constants():
    d = defines()
    for name in ("MXFP4_MAX_GROUPS", "MXFP4_FUSED_ROWS", "MXFP4_FUSED_GROUPED_ROWS"):
        assert getattr(B, name) == d[name], name
    assert O.MAX_GROUPS == d["MXFP4_MAX_GROUPS"]


def test_library_goes_by_the_header_s_constants():
    d = defines()
    most = d["MXFP4_MAX_GROUPS"]
    assert B.lib.mxfp4_grouped_scale_bytes(most, 1, 32) > 0 > B.lib.mxfp4_grouped_scale_bytes(most + 1, 1, 32)
    for groups, rows in ((0, d["MXFP4_FUSED_ROWS"]), (3, d["MXFP4_FUSED_GROUPED_ROWS"])):
        assert B.lib.mxfp4_workspace_bytes(groups, rows, 64) == 0
        assert B.lib.mxfp4_workspace_bytes(groups, rows + 1, 64) > 0


def test_types_are_the_header_s():
    text = re.search(r"typedef enum \{([^}]*)\} mxfp4_dtype;", open(HEADER).read()).group(1)
    assert dict(re.findall(r"(MXFP4_\w+) = (\d)", text)) == {"MXFP4_BF16": "0", "MXFP4_FP16": "1", "MXFP4_FP32": "2"}
    out = [B.lib.mxfp4_dequantize(t, 0, 64, None, None, 0, None, None, 64, None, None) for t in range(4)]
    assert out == [0, 1, 0, 1]      # bf16 and fp32 only
