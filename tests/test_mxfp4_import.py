"""The package without its extension module, which is built against one torch
and one Python: only the MXFP4 calls need it."""
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

import bit_w4a4_diffusion_b200 as B

PKG = os.path.dirname(os.path.abspath(B.__file__))

USE = """
import numpy as np, torch
import bit_w4a4_diffusion_b200 as B
assert B.__file__.startswith({root!r}), B.__file__
assert B.act_scale_bytes("nvfp4", 4096, 2048) == 4096 * 128
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


def run_in_copy(tmp_path, program, **files):
    """Runs a program beside a copy of the package with `files` in place of
    the module."""
    pkg = tmp_path / "bit_w4a4_diffusion_b200"
    pkg.mkdir()
    shutil.copy(os.path.join(PKG, "__init__.py"), pkg)
    os.symlink(os.path.join(PKG, "lib"), pkg / "lib")
    for name, text in files.items():
        (pkg / (name + ".py")).write_text(text)
    env = {k: v for k, v in os.environ.items() if k != "PYTHONPATH"}
    r = subprocess.run([sys.executable, "-c", program], cwd=tmp_path, env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def use_package(tmp_path, why, **files):
    run_in_copy(tmp_path, USE.format(root=str(tmp_path), why=why), **files)


def test_the_other_calls_need_no_extension_module(tmp_path):
    use_package(tmp_path, "_mxfp4")


def test_a_module_that_does_not_load(tmp_path):
    use_package(tmp_path, "undefined symbol", _mxfp4="raise ImportError('undefined symbol')")


def test_a_module_of_another_torch(tmp_path):
    use_package(tmp_path, "built for torch 0.0.1", _mxfp4="built_for_torch = '0.0.1'\n"
                "def set_error(e): pass\ndef quantize(*a): return 1\ndef linear(*a): return 1\n")


def test_a_module_that_does_not_say_what_it_was_built_for(tmp_path):
    """One of an earlier build."""
    use_package(tmp_path, "built for torch", _mxfp4="def set_error(e): pass\ndef quantize(*a): return 1\n"
                "def linear(*a): return 1\n")


def test_the_build_follows_the_installed_torch(tmp_path, monkeypatch):
    """Another torch is another module, also where the installer keeps old
    file times; the same one is built once."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    torch = tmp_path / "torch"
    torch.mkdir()

    def install(version):
        (torch / "version.py").write_text(f"__version__ = {version!r}\n")
        os.utime(torch / "version.py", (0, 0))

    built = []

    def run(cmd, verbose):
        built.append(cmd)
        with open(build.BIND, "w") as f:
            f.write("module")

    class Spec:
        origin = str(torch / "__init__.py")

    monkeypatch.setattr(build, "BIND", str(tmp_path / "_mxfp4.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "PKG", str(tmp_path / "elsewhere"))
    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: Spec)
    for version, count in (("9.9.0", 1), ("9.9.0", 1), ("9.9.1", 2), ("9.9.1", 2), ("9.9.0", 3)):
        install(version)
        build._build_bind([], False)
        assert len(built) == count, (version, len(built))


def test_the_module_is_named_for_its_interpreter():
    assert os.path.basename(B._mxfp4.__file__).split(".", 1)[1] == sysconfig.get_config_var("EXT_SUFFIX")[1:]


RELOAD = """
import importlib, os, torch
import bit_w4a4_diffusion_b200 as B
try:
    B._mxfp4.quantize
    raise AssertionError("there is no module yet")
except ImportError:
    pass
with open(os.path.join(os.path.dirname(B.__file__), "_mxfp4.py"), "w") as f:
    f.write(f"built_for_torch = {str(torch.__version__)!r}\\ndef set_error(e): pass\\ndef quantize(*a): return 7\\n")
importlib.invalidate_caches()
importlib.reload(B)
assert B.mxfp4_quantize(torch.zeros(4, 64)) == 7
print("fine")
"""


def test_a_module_built_later_is_found_by_a_reload(tmp_path):
    run_in_copy(tmp_path, RELOAD)


def test_build_entry_needs_the_module(monkeypatch):
    """The package imports without its module; a build that left none is no
    build."""
    import __graft_entry__ as entry

    class Nothing:
        @staticmethod
        def build(verbose):
            pass

    monkeypatch.setattr(entry, "_build_module", lambda: Nothing)
    monkeypatch.setattr(entry.importlib, "reload", lambda module: module)
    entry.build()
    monkeypatch.setattr(B, "_mxfp4", B._Unavailable("left out"))
    with pytest.raises(ImportError):
        entry.build()
