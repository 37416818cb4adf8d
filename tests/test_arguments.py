"""The binding's native argument checks (csrc/arguments.cpp): they pass what the
Python functions behind them pass, with the same address, and leave the rest to
them."""
import os
import subprocess
import sys

import pytest
import torch

from vision_transformer_shifted_gb300 import _arguments
from vision_transformer_shifted_gb300 import binding as sw

BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


class Handle:
    C = 8


def test_in_their_places_once_loaded():
    sw.load()
    assert sw._arg is _arguments.arg and sw._rows is _arguments.rows


@pytest.mark.parametrize("call", [
    lambda x: sw._arg("x", x, BF, x.shape, 0),                        # (on the CPU)
    lambda x: sw._arg("x", x, F32, x.shape, 0),
    lambda x: sw._arg("x", x, BF, (4, 9), 0),
    lambda x: sw._arg("x", x, BF, (4,), 0),
    lambda x: sw._arg("x", x.t(), BF, (8, 4), 0),
    lambda x: sw._rows(Handle, x, BF, "x"),
    lambda x: sw._rows(Handle, x[:, :4], BF, "x"),
    lambda x: sw._rows(Handle, x.float(), BF, "x"),
])
def test_refusals_are_the_python_functions(call):
    sw.load()
    with pytest.raises(ValueError):
        call(torch.zeros(4, 8, dtype=BF))


def test_other_objects_and_counts_of_arguments():
    sw.load()
    for bad in (None, 3, "x"):
        with pytest.raises(AttributeError):
            sw._arg("x", bad, BF, (4, 8), 0)
        with pytest.raises(AttributeError):
            sw._rows(Handle, bad, BF, "x")
    with pytest.raises(TypeError):
        sw._arg("x", torch.zeros(1))
    with pytest.raises(TypeError):
        _arguments.setup(1)


class Sub(torch.Tensor):
    pass


THREADS = """
import sys, threading
import torch
from vision_transformer_shifted_gb300 import binding as sw
sys.setswitchinterval(1e-6)
class Sub(torch.Tensor):
    pass
x = torch.zeros(4, 8, dtype=torch.bfloat16)
gate, seen = threading.Barrier(16), []
def work():
    gate.wait()
    sw.load()
    try:   # (CPU tensors: their device is -1)
        assert sw._arg("x", x.as_subclass(Sub), torch.bfloat16, (4, 8), -1) == x.data_ptr()
        sw._arg("x", x, torch.bfloat16, (4, 8), 0)
    except Exception as e:
        seen.append(type(e).__name__)
threads = [threading.Thread(target=work) for _ in range(16)]
for t in threads:
    t.start()
for t in threads:
    t.join()
print(sorted(set(seen)), len(seen))
"""


def test_first_load_from_many_threads():
    """What the native checks leave to the Python functions reaches them, whoever
    loaded the library and however often."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(3):
        done = subprocess.run([sys.executable, "-c", THREADS], cwd=root, capture_output=True, text=True, timeout=300)
        assert done.returncode == 0 and done.stdout.strip() == "['ValueError'] 16", done.stdout + done.stderr[-2000:]



WITHOUT = """
import sys, types
import torch
import vision_transformer_shifted_gb300 as pkg
from vision_transformer_shifted_gb300 import binding as sw
def setup(*a):
    raise SystemExit("not to be asked")
for other in (None, types.SimpleNamespace(setup=setup), types.SimpleNamespace(setup=setup, torch_version="0.1")):
    sys.modules[pkg.__name__ + "._arguments"] = other
    if other is not None:
        pkg._arguments = other
    sw._lib = None
    assert sw.load().swin_block_rms_destroy(None) == sw.OK
    assert sw._arg is sw._arg_python and sw._rows is sw._rows_python
    try:
        sw._arg("x", torch.zeros(4, 8), torch.bfloat16, (4, 8), -1)
    except ValueError:
        print("refused")
"""


def test_library_works_without_the_native_checks():
    """Not there (not built, another Python), of a build that does not say its PyTorch,
    of another PyTorch: the Python functions stay in their places."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", WITHOUT], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and done.stdout.split() == ["refused"] * 3, done.stdout + done.stderr[-2000:]


def test_native_checks_are_of_this_python_and_torch(monkeypatch):
    import sysconfig

    from vision_transformer_shifted_gb300 import build
    assert _arguments.torch_version == str(torch.__version__) == build.torch_version()
    assert _arguments.__file__ == build.ARGUMENTS and build.ARGUMENTS.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(build, "_newer", lambda *a: True)
    assert build.arguments_current()
    monkeypatch.setattr(build, "torch_version", lambda: "0.1")
    assert not build.arguments_current()   # (built anew)


def test_build_without_a_compiler_for_the_checks_keeps_the_library(monkeypatch, capsys):
    from vision_transformer_shifted_gb300 import build

    def no_compiler(*a, **kw):
        raise FileNotFoundError("g++")

    monkeypatch.setattr(build, "arguments_current", lambda: False)
    monkeypatch.setattr(build, "_library_current", lambda: True)
    monkeypatch.setattr(build.subprocess, "run", no_compiler)
    assert build.build() == build.LIB
    assert "arguments.cpp" in capsys.readouterr().err


@pytest.mark.gpu
def test_addresses_on_the_gpu():
    sw.load()
    x = torch.zeros(6, 3, 8, dtype=BF, device="cuda")
    for t in (x, x[2:], x[1, 1:], torch.nn.Parameter(x), x.as_subclass(Sub), x[:0], x.view(torch.int16).view(BF)):
        assert sw._arg("t", t, BF, t.shape, 0) == t.data_ptr()
        assert sw._arg("t", t, BF, tuple(t.shape), 0) == t.data_ptr()
        assert sw._rows(Handle, t, BF, "t") == (t.numel() // 8, t.shape, 0, t.data_ptr())
    for dtype in (F32, E4M3):
        t = torch.zeros(5, 8, device="cuda").to(dtype)
        assert sw._arg("t", t, dtype, (5, 8), 0) == t.data_ptr()
    for t, dtype, shape, dev in ((x.float(), BF, x.shape, 0), (x, F32, x.shape, 0), (x, BF, (6, 24), 0), (x, BF, [6, 3, 8, 1], 0),
                                 (x.transpose(0, 1), BF, (3, 6, 8), 0), (x[:, :2], BF, (6, 2, 8), 0), (x, BF, x.shape, 1),
                                 (x.cpu(), BF, x.shape, 0), (x.half(), torch.float32, x.shape, 0)):
        with pytest.raises(ValueError):
            sw._arg("t", t, dtype, shape, dev)
    assert sw._arg("t", x.half(), torch.half, x.shape, 0)   # (a type that only the Python function knows)
    for t in (x[..., :4], x.transpose(0, 1), x.float(), x.cpu()):
        with pytest.raises(ValueError):
            sw._rows(Handle, t, BF, "t")
    with torch.inference_mode():
        y = torch.zeros(4, 8, dtype=BF, device="cuda")
        assert sw._arg("y", y, BF, (4, 8), 0) == y.data_ptr()


@pytest.mark.gpu
def test_addresses_without_leaking():
    """A thousand calls leave the reference counts of what they were given."""
    import sys
    sw.load()
    x, shape = torch.zeros(4, 8, dtype=BF, device="cuda"), (4, 8)
    counts = lambda: [sys.getrefcount(o) for o in (x, shape, BF, Handle, Handle.C)]  # noqa: E731
    before = counts()
    for _ in range(1000):
        sw._arg("x", x, BF, shape, 0)
        sw._rows(Handle, x, BF, "x")
    assert counts() == before
