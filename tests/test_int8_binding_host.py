"""The 8-bit calls' native module on the CPU: how it is found and built, and how it
calls the library.  Every test runs a child process, with stand-ins for torch's
tensors and the library where it calls."""
import os
import subprocess
import sys
import textwrap

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _child(code, **env):
    p = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300, env={**os.environ, **env})
    assert p.returncode == 0, p.stdout + p.stderr
    return p.stdout


# stand-ins: a tensor whose address is a number of microseconds, and usleep as the
# library's paro_quantize_activations_int8 (its first argument is x's address)
FAKES = """
    import ctypes, threading, time
    from types import SimpleNamespace
    import torch
    import rotation_int4_weight_b200 as paro

    class Tensor:
        def __init__(self, shape, dtype, at):
            self.shape, self.dtype, self.device, self.at = torch.Size(shape), dtype, "cuda:0", at
        def get_device(self): return 0
        def is_contiguous(self): return True
        def data_ptr(self): return self.at

    fake = SimpleNamespace(**{n: getattr(torch, n) for n in ("int8", "float32", "bfloat16", "float16", "int16",
                                                            "uint16", "uint8")},
                           empty=None, empty_like=None,
                           _C=SimpleNamespace(_cuda_getCurrentRawStream=lambda d: 0, _cuda_getDevice=lambda: 0))
    usleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    paro._binding.setup(fake, paro._check, (usleep,) * 7)
"""


def test_other_threads_run_while_the_library_is_called():
    # a launch that waits for room in the queue must not stop the process's other threads
    out = _child(FAKES + """
    ticks, stop = [], False
    def tick():
        while not stop:
            ticks.append(time.perf_counter())
            time.sleep(0.005)
    t = threading.Thread(target=tick); t.start()
    time.sleep(0.05)
    a = time.perf_counter()
    paro._binding.quantize(Tensor((2, 16), torch.bfloat16, 400000), Tensor((2, 16), torch.int8, 64),
                           Tensor((2,), torch.float32, 64))
    b = time.perf_counter()
    stop = True; t.join()
    print(b - a, sum(a < x < b - 0.01 for x in ticks))
    """)
    took, ticks = out.split()
    assert float(took) >= 0.4
    assert int(ticks) >= 5, "the call kept the interpreter's lock"


def test_the_module_is_named_for_the_interpreter_it_is_built_for():
    # a name without a tag would be loaded by any CPython, and count as built for it
    out = _child("""
    import importlib.machinery, importlib.util, os, sysconfig
    import rotation_int4_weight_b200 as paro
    spec = importlib.util.spec_from_file_location("b", os.path.join(os.path.dirname(paro.__file__), "_build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    print(sysconfig.get_config_var("EXT_SUFFIX"), b.BINDING, paro._binding.__file__)
    """)
    tag, built, loaded = out.split()
    assert tag not in (".so", ".abi3.so")
    assert built == loaded and built.endswith("_binding" + tag)


# the package as it is, and a Python that has no _binding for it
WITHOUT = """
    import sys
    class Finder:
        def find_spec(self, name, path=None, target=None):
            if name.endswith("._binding"):
                raise ModuleNotFoundError(f"No module named {name!r}", name=name)
    sys.meta_path.insert(0, Finder())
"""


def test_the_package_without_the_module_has_everything_but_the_8_bit_calls():
    _child(WITHOUT + """
    import torch
    import rotation_int4_weight_b200 as paro
    assert paro.paro_weight_layout_version() == 1
    assert paro.paro_workspace_bytes(1, 512) > 0
    assert paro.lib.paro_w8a8_linear is not None         # the C ABI has them
    x = torch.zeros(2, 16, dtype=torch.bfloat16)
    q, s = torch.zeros(2, 16, dtype=torch.int8), torch.ones(2)
    for call in (lambda: paro.paro_quantize_activations_int8(x), lambda: paro.paro_rms_norm_int8(x),
                 lambda: paro.paro_pack_weights_int8(x.float()), lambda: paro.paro_w8a8_linear(q, s, q, s),
                 lambda: paro.paro_w8a8_swiglu(q, s, q, s, q, s),
                 lambda: paro.paro_rotate_w8a8_linear(x, None, None, None, None, q, s)):
        try:
            call()
        except ImportError as e:
            assert "_build.py" in str(e) and isinstance(e.__cause__, ImportError)
        else:
            raise AssertionError("the call went on without its module")
    """)


def test_the_package_imports_with_a_torch_that_has_no_cuda():
    _child("""
    import torch
    del torch._C._cuda_getCurrentRawStream
    import rotation_int4_weight_b200 as paro
    assert paro.paro_workspace_bytes(1, 512) > 0
    try:
        paro.paro_quantize_activations_int8(torch.zeros(2, 16, dtype=torch.bfloat16))
    except ImportError as e:
        assert "_cuda_getCurrentRawStream" in str(e)
    else:
        raise AssertionError("the call went on")
    """)


def test_the_build_without_python_headers_leaves_the_module_out():
    out = _child("""
    import importlib.util, sys, sysconfig
    real = sysconfig.get_paths
    sysconfig.get_paths = lambda *a, **k: dict(real(*a, **k), include="/nonexistent")
    spec = importlib.util.spec_from_file_location("b", "rotation_int4_weight_b200/_build.py")
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    b._newer = lambda target, deps: False
    sys.stderr = sys.stdout
    assert b.build_binding() is None
    """)
    assert "Python.h" in out
