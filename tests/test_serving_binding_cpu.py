"""The serving binding without a GPU: a child process in which torch's two device queries are replaced, tensors are objects
with a tensor's attributes, and the library's functions are ones that report on their call; and its build."""
import importlib.machinery
import os
import subprocess
import sys
import sysconfig
import textwrap

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALLEE = """
#include <unistd.h>
static volatile int flag;
void set_flag(int v) { flag = v; }
int until_flag(void) {  /* at most three seconds */
  for (int i = 0; i < 3000 && !flag; ++i) usleep(1000);
  return flag ? 0 : 77;
}
int zero(void) { return 0; }
"""

CHILD = """
import ctypes, importlib.machinery, importlib.util, sys, threading, time
sys.path.insert(0, {root!r})
import torch
torch._C._cuda_getDevice = lambda: 0
torch._C._cuda_getCurrentRawStream = lambda device: 0
from fp8_quantized_exact_b200 import SageError, build
loader = importlib.machinery.ExtensionFileLoader("_sage_serving", build.SERVING)
m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_sage_serving", loader))
loader.exec_module(m)
callee = ctypes.CDLL({callee!r})
address = lambda f: ctypes.cast(f, ctypes.c_void_p).value

class Tensor:
    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, shape
    def stride(self):
        s = [1]
        for n in self.shape[:0:-1]:
            s.insert(0, s[0] * n)
        return tuple(s)
    def get_device(self): return 0
    def data_ptr(self): return 4096
    def element_size(self): return 1

i32, bf16 = torch.int32, torch.bfloat16
cache = (Tensor(torch.int8, 4, 2, 16, 64), Tensor(torch.float32, 4, 2, 16)) * 2
x, q = Tensor(bf16, 3, 5, 2, 64), Tensor(bf16, 3, 5, 4, 64)
table, lens, ws = Tensor(i32, 3, 2), Tensor(i32, 3), Tensor(torch.uint8, 1024)
calls = dict(rope=[q, x, q, x, None, Tensor(torch.float64, 32), 1.0, 0, None, False, None],
             append=[cache, x, x, table, lens, None, ws, None],
             read=[cache, table, lens, None, x, x, ws, None],
             attn=[q, cache, table, lens, None, None, q, None, 0.0, ws, None])
{body}
"""


@pytest.fixture(scope="module")
def build():
    from fp8_quantized_exact_b200 import build as b
    b.build()
    return b


def child(tmp_path, body):
    src, so = tmp_path / "callee.c", tmp_path / "callee.so"
    src.write_text(CALLEE)
    subprocess.check_call([os.environ.get("CC", "gcc"), "-O1", "-fPIC", "-shared", str(src), "-o", str(so)])
    code = CHILD.format(root=ROOT, callee=str(so), body=textwrap.dedent(body))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_calls_let_other_threads_run(build, tmp_path):
    """A launch may block; what it waits for may be a Python thread's to do."""
    child(tmp_path, """
        m.bind(*[address(callee.until_flag)] * 4, SageError)
        for name, args in calls.items():
            callee.set_flag(0)
            def free():
                time.sleep(0.1)
                callee.set_flag(1)
            t = threading.Thread(target=free)
            t.start()
            getattr(m, name)(*args)  # SageError(77) where the other thread could not set the flag
            t.join()
    """)


def test_wrong_arguments(build, tmp_path):
    """Too few or many arguments, None for a tensor that is not optional, and an object that is no tensor."""
    child(tmp_path, """
        m.bind(*[address(callee.zero)] * 4, SageError)
        optional = dict(rope={1, 4, 8, 10}, append={4, 5, 7}, read={2, 3, 4, 5, 7}, attn={4, 5, 7, 10})
        def refused(error, name, args):
            try:
                getattr(m, name)(*args)
            except error:
                return
            raise AssertionError((name, error, len(args)))
        for name, args in calls.items():
            assert getattr(m, name)(*args) is None
            for n in (0, 1, 2, 3, 4, len(args) - 1):
                refused(TypeError, name, args[:n])
            refused(TypeError, name, args + [None])
            for i, a in enumerate(args):
                if isinstance(a, Tensor):
                    for other in (3, "x", [1]) + (() if i in optional[name] else (None,)):
                        refused(ValueError, name, args[:i] + [other] + args[i + 1:])
        refused(ValueError, "append", [None] + calls["append"][1:])
        refused(ValueError, "append", [cache[:3] + (None,)] + calls["append"][1:])
        refused(ValueError, "append", [cache[:3]] + calls["append"][1:])
        refused(ValueError, "rope", calls["rope"][:3] + [None] + calls["rope"][4:])
        refused(ValueError, "read", calls["read"][:4] + [None, None] + calls["read"][6:])
    """)


def test_module_is_the_interpreters_own(build):
    """Its name has the ABI tag, so that another Python version builds and loads one of its own."""
    assert build.SERVING.endswith("_sage_serving" + sysconfig.get_config_var("EXT_SUFFIX"))
    assert sysconfig.get_config_var("EXT_SUFFIX") in importlib.machinery.EXTENSION_SUFFIXES
    from fp8_quantized_exact_b200 import serving
    assert os.path.samefile(serving._calls().__spec__.origin, build.SERVING)


def test_library_builds_without_python_headers(build, tmp_path, monkeypatch, capsys):
    """The library needs nvcc alone; the serving calls then say what is missing."""
    import fp8_quantized_exact_b200 as sage
    from fp8_quantized_exact_b200 import serving
    missing = str(tmp_path / "_sage_serving.so")
    monkeypatch.setattr(build, "SERVING", missing)
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build.build() == build.LIB
    assert not os.path.exists(missing) and "Python.h" in capsys.readouterr().err
    monkeypatch.setattr(serving, "_native", None)
    monkeypatch.setattr(serving, "_bound", None)
    with pytest.raises(RuntimeError, match="not built"):
        sage.sage_rope(None, None, None, None, None, None)
    assert sage.sage_workspace_bytes(sage.SAGE_OP_CACHE, 1, 1, 1, 64) > 0


@pytest.mark.parametrize("workspace", [torch.zeros(1024, dtype=torch.uint8), None])
def test_clear_status_refuses_what_is_no_device_workspace(build, workspace):
    import fp8_quantized_exact_b200 as sage
    with pytest.raises(ValueError):
        sage.sage_clear_device_status(workspace)
