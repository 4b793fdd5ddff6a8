"""The binding's C module on objects that answer what it asks of a tensor (CPU), and the same together with the
host side of gdn_layer.h under AddressSanitizer and UndefinedBehaviorSanitizer."""
import os
import subprocess
import sys
import sysconfig

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CLANG = "/opt/rocm/llvm/bin/clang"


class T:
    def __init__(self, shape, stride, dtype="bf16", device=0, at=4096, contiguous=True):
        self.shape, self._stride, self.dtype, self._device, self._at, self._c = shape, stride, dtype, device, at, contiguous

    def stride(self):
        return self._stride

    def get_device(self):
        return self._device

    def data_ptr(self):
        return self._at

    def is_contiguous(self):
        return self._c


@pytest.fixture(scope="module")
def M():
    import gated_delta_rule_34_amd as G

    return G.layer._marshal


def test_rows(M):
    rows = lambda *a, n=4, w=32, **k: M.rows(T(*a, **k), n, w, 0, "bf16")
    assert rows((4, 32), (40, 1)) == (4096, 40)
    assert rows((4, 2, 16), (40, 16, 1)) == (4096, 40)
    assert rows((4, 32, 1), (40, 1, 7)) == (4096, 40)  # heads of one value: no stride among them
    assert rows((4, 1, 32), (40, 5, 1)) == (4096, 40) and rows((4, 1), (40, 9), w=1) == (4096, 40)
    assert rows((1, 32), (7, 1), n=1) == (4096, 32)  # no second row, no stride
    assert rows((0, 32), (0, 9), n=0) == (4096, 32)
    assert rows((4, 32), (0, 1)) == (4096, 0)  # (expanded rows are refused in the library)
    for shape, stride in (((4, 32), (40, 2)), ((4, 31), (40, 1)), ((5, 32), (40, 1)), ((4, 2, 16), (40, 20, 1)), ((4, 2, 16), (40, 16, 2)),
                          ((128,), (1,)), ((1, 4, 2, 16), (1, 32, 16, 1)), ((), ()), ((4, 32), (40,)), ([4, 32], (40, 1))):
        assert rows(shape, stride) is None, (shape, stride)
    assert rows((4, 32), (40, 1), dtype="f32") is None and rows((4, 32), (40, 1), device=1) is None and rows((4, 32), (40, 1), device=-1) is None


def test_array(M):
    assert M.array(T((2, 3), (3, 1)), (2, 3), 0, "bf16") == 4096
    for t in (T((2, 3), (3, 1), contiguous=False), T((3, 2), (2, 1)), T((2, 3), (3, 1), dtype="f32"), T((2, 3), (3, 1), device=1)):
        assert M.array(t, (2, 3), 0, "bf16") is None


def test_errors_come_through(M):
    class Broken(T):
        def data_ptr(self):
            raise RuntimeError("no storage")

        def get_device(self):
            return "0" if self._at == 1 else 0

    for f in (lambda t: M.rows(t, 4, 32, 0, "bf16"), lambda t: M.array(t, (4, 32), 0, "bf16")):
        with pytest.raises(RuntimeError):
            f(Broken((4, 32), (32, 1)))
        with pytest.raises(TypeError):
            f(Broken((4, 32), (32, 1), at=1))
        with pytest.raises(AttributeError):
            f(object())
    with pytest.raises(TypeError):
        M.rows(T((4, 32), (32, 1)), 4, 32, 0)
    with pytest.raises(TypeError):
        M.rows(T((4, 32), ("x", 1)), 4, 32, 0, "bf16")
    with pytest.raises(TypeError):
        M.rows(T((4, 32), (32, 1)), "4", 32, 0, "bf16")
    with pytest.raises(TypeError):
        M.array(T((4, 32), (32, 1)), (4, 32), 0)
    import gated_delta_rule_34_amd as G

    at, p = G.layer._at("gdn_gated_norm_fwd"), G.make_norm_problem(1, 8)
    for args in ((at,), (at, p, "x"), (at, p, 1 << 70), (at, 5, 1), ("x", p, 1), (at, p, *[0] * 29)):
        with pytest.raises((TypeError, OverflowError)):
            M.call(*args)
    for args in ((at,), ("x", p), (at, 5)):
        with pytest.raises(TypeError):
            M.size(*args)


def test_host_side_under_sanitizers(tmp_path):
    """-fsanitize=function is left out: m_call calls every function through one prototype of integers, by design."""
    r = subprocess.run([CLANG, "-print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True, text=True) if os.path.exists(CLANG) else None
    rt = r.stdout.strip() if r else ""
    if not (os.path.exists(HIPCC) and os.path.isabs(rt) and os.path.exists(rt)):
        pytest.skip("no hipcc / clang sanitizer runtime")
    csrc, san = os.path.join(ROOT, "gated_delta_rule_34_amd", "csrc"), os.path.join(ROOT, "tests", "sanitize")
    lib = str(tmp_path / "libgdn_sanitized.so")
    subprocess.run([HIPCC, "-xhip", "--offload-host-only", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                    "-Xarch_host", "-fno-sanitize=function", "-shared-libasan", "-fno-omit-frame-pointer", "-g", "-O1", "-std=c++17", "-fPIC",
                    "-shared", f"-I{ROOT}/include", f"-I{csrc}", os.path.join(csrc, "gdn_abi.cpp"), os.path.join(csrc, "layer", "layer_abi.cpp"),
                    os.path.join(san, "gdn_host_stubs.cpp"), os.path.join(san, "layer_host_stubs.cpp"), "-o", lib], check=True)
    mod = str(tmp_path / ("_marshal" + sysconfig.get_config_var("EXT_SUFFIX")))
    subprocess.run([CLANG, "-fsanitize=address,undefined", "-fno-sanitize=function", "-shared-libasan", "-fno-omit-frame-pointer", "-g", "-O1",
                    "-shared", "-fPIC", f"-I{sysconfig.get_paths()['include']}", os.path.join(csrc, "layer", "marshal.c"), "-o", mod], check=True)
    code = f"""
import importlib.util, sys
spec = importlib.util.spec_from_file_location("gated_delta_rule_34_amd._marshal", {mod!r})
sys.modules[spec.name] = importlib.util.module_from_spec(spec)
spec.loader.exec_module(sys.modules[spec.name])
import pytest
import gated_delta_rule_34_amd as G
maps = open("/proc/self/maps").read()
assert {lib!r} in maps and {mod!r} in maps and {os.path.basename(rt)!r} in maps and G.layer._marshal.__file__ == {mod!r}
sys.exit(pytest.main(["-q", "-p", "no:cacheprovider", "-m", "not gpu", "tests/test_layer_host.py", "tests/test_layer_marshal.py",
                      "-k", "not sanitizers"]))
"""
    env = dict(os.environ, LD_PRELOAD=rt, GDN_LIBRARY=lib, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", code], env=env, cwd=ROOT, capture_output=True, text=True, timeout=900)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert "ERROR: AddressSanitizer" not in tail and "runtime error" not in tail and " passed" in r.stdout, tail
