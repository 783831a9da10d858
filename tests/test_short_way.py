"""CPU tests of the short way of the norm's and 4-bit calls, the extension module _calls: the package
needs neither it nor what it is built with, and takes none that was built for another torch."""
import glob
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "activation_sparse_decode_rank_amd"
HERE = os.path.join(ROOT, NAME)


def package(tmp_path, **files):
    """The package's Python files and HIP library elsewhere, and other files beside them."""
    to = tmp_path / NAME
    to.mkdir()
    for f in glob.glob(os.path.join(HERE, "*.py")):
        shutil.copy(f, to)
    os.symlink(os.path.join(HERE, "libsparse_ffn.so"), to / "libsparse_ffn.so")
    for name, text in files.items():
        (to / name).write_text(text)


def run(tmp_path, code):
    code = f"import sys; sys.path.insert(0, {str(tmp_path)!r})\n" + code
    return subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=120)


USE = f"""
import warnings
with warnings.catch_warnings(record=True) as told:
    warnings.simplefilter("always")
    import {NAME} as P
assert P.__file__.startswith({{at!r}}), P.__file__
import torch
assert callable(P.i8_matmul) and callable(P.SparseFFN) and P.mx4._calls.norm(1, 2) is None
for call in (lambda: P.rms_norm(torch.zeros(2, 64)), lambda: P.quantize_mx4(torch.zeros(2, 64))):
    try:
        call()
    except ValueError as e:
        assert "device" in str(e)
    else:
        raise AssertionError
print(sum("_calls" in str(w.message) for w in told))
"""


@pytest.mark.parametrize("files", [
    {}, {"_calls.py": "raise ImportError('undefined symbol')\n"},
    {"_calls.py": "def norm(*a): raise SystemError\ndef bind(*a): raise SystemError\n"},
    {"_calls.py": "built_for = '1.0.0'\ndef norm(*a): raise SystemError\ndef bind(*a): raise SystemError\n"}])
def test_the_package_works_without_the_module(tmp_path, files):
    """None there, one that does not load, one that does not say what it was built for, one built for
    another torch: the calls go through ctypes, and a warning says so."""
    package(tmp_path, **files)
    r = run(tmp_path, USE.format(at=str(tmp_path)))
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "1"


def test_what_is_built_is_for_this_python_and_torch():
    import torch
    from activation_sparse_decode_rank_amd import _calls, mx4
    import sysconfig
    assert mx4._calls is _calls and _calls.built_for == torch.__version__
    assert _calls.__file__.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


def build_script():
    spec = importlib.util.spec_from_file_location("_sffn_build_test", os.path.join(HERE, "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("missing", ["compiler", "headers"])
def test_the_build_goes_on_without_the_module(tmp_path, monkeypatch, capsys, missing):
    """A module that cannot be built is told of and left out, and an old one does not stay."""
    m = build_script()
    monkeypatch.setattr(m, "CALLS", str(tmp_path / "_calls.new.so"))
    for old in ("_calls.so", "_calls.new.so", "_calls.cpython-27.so"):
        (tmp_path / old).write_text("")
    (tmp_path / "libsparse_ffn.so").write_text("")
    if missing == "compiler":
        monkeypatch.setattr(m, "CXX", str(tmp_path / "no-such-compiler"))
    else:
        monkeypatch.setattr(m.importlib.util, "find_spec", lambda name: None)
    assert m.build_calls() is False
    assert "_calls" in capsys.readouterr().err
    assert sorted(os.listdir(tmp_path)) == ["libsparse_ffn.so"]


def test_the_module_refuses_what_is_no_argument():
    """A wrong number of arguments is a TypeError, as from any function, and a stream that is no address is
    refused before anything is looked at."""
    import torch
    from activation_sparse_decode_rank_amd import _calls
    for name in ("norm", "quantize", "dequantize", "matmul"):
        for args in ((), (1,), (None,) * 20):
            with pytest.raises(TypeError):
                getattr(_calls, name)(*args)
    x = torch.zeros((2, 64))
    for stream, error in ((1 << 80, OverflowError), ("0", TypeError), (None, TypeError)):
        for call in (lambda: _calls.norm(x, None, None, 1e-6, -1, None, 0, stream),
                     lambda: _calls.quantize(x, 0, stream), lambda: _calls.dequantize(x, x, None, 0, 0, stream),
                     lambda: _calls.matmul(x, x, x, None, None, -1, 0, stream)):
            with pytest.raises(error):
                call()
    for cols in (1 << 64, -1 << 70):  # left to the function, which says what the blocks hold
        assert _calls.dequantize(x, x, cols, 0, 0, 0) is None


def test_the_package_works_with_a_torch_without_devices(tmp_path):
    """A torch that was built without device support has no _cuda_getDevice: importing the package does
    not look for it, and the calls say that they need device tensors."""
    package(tmp_path)
    code = "import torch\nfor name in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n    delattr(torch._C, name)\n"
    r = run(tmp_path, code + USE.format(at=str(tmp_path)))
    assert r.returncode == 0, r.stderr
