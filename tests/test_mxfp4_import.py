"""The package without its extension module, which is built against one torch
and one Python: only the MXFP4 calls need it."""
import os
import shutil
import subprocess
import sys

import bit_w4a4_diffusion_b200 as B

PKG = os.path.dirname(os.path.abspath(B.__file__))

USE = """
import numpy as np, torch
import bit_w4a4_diffusion_b200 as B
assert B.__file__.startswith({root!r}), B.__file__
assert B.act_scale_bytes("nvfp4", 4096, 3072) == 4096 * 192
assert B.mxfp4_pack_weights(np.zeros((4, 64), np.uint16))["codes"].shape == (4, 32)
for call in (lambda: B.mxfp4_quantize(torch.zeros(4, 64)), lambda: B.mxfp4_linear(torch.zeros(4, 64), dict())):
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e) and {why!r} in str(e), e
    else:
        raise AssertionError("an MXFP4 call went through without its module")
print("fine")
"""


def use_package(tmp_path, why, **files):
    """Imports a copy of the package with `files` in place of the module."""
    pkg = tmp_path / "bit_w4a4_diffusion_b200"
    pkg.mkdir()
    shutil.copy(os.path.join(PKG, "__init__.py"), pkg)
    os.symlink(os.path.join(PKG, "lib"), pkg / "lib")
    for name, text in files.items():
        (pkg / (name + ".py")).write_text(text)
    env = {k: v for k, v in os.environ.items() if k != "PYTHONPATH"}
    r = subprocess.run([sys.executable, "-c", USE.format(root=str(tmp_path), why=why)], cwd=tmp_path, env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_the_other_calls_need_no_extension_module(tmp_path):
    use_package(tmp_path, "_mxfp4")


def test_a_module_that_does_not_load(tmp_path):
    use_package(tmp_path, "undefined symbol", _mxfp4="raise ImportError('undefined symbol')")
