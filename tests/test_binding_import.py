"""The package without the binding's C++ extension: what does not use it still runs."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "selective_state_space_46_b200"


@pytest.fixture(scope="module", params=["missing", "of another torch"])
def package(request, tmp_path_factory):
    at = tmp_path_factory.mktemp("alone")
    (at / PKG).mkdir()
    shutil.copy(os.path.join(ROOT, PKG, "__init__.py"), at / PKG)
    os.symlink(os.path.join(ROOT, PKG, "libmssm.so"), at / PKG / "libmssm.so")
    if request.param != "missing":
        (at / PKG / "_marshal.so").write_bytes(b"not a shared object")
    return str(at)


def run(package, code):
    return subprocess.run([sys.executable, "-c", "import torch, selective_state_space_46_b200 as m\n" + code], cwd=package,
                          capture_output=True, text=True, timeout=120)


def test_the_other_operators_stay(package):
    r = run(package, """
print(m.mssm_version(), m.mssm_kernel_stats())
t = torch.zeros(2, 8, 32)
for call in (lambda: m.mssm_selective_scan_fwd(*[t] * 8, True, t, t), lambda: m.mssm_causal_conv1d_fwd(t, t[0], t[0, :, 0], t)):
    try:
        call()
    except (m.MssmError, ValueError, RuntimeError) as e:
        print(type(e).__name__, e)
""")
    assert r.returncode == 0, r.stderr
    assert "_marshal" not in r.stdout


def test_the_operators_that_need_it_say_so(package):
    r = run(package, """
x, v = torch.zeros(2, 8, 32), torch.zeros(8)
for call in (lambda: m.gated_scan_fwd(x, x, x, v), lambda: m.gated_scan_bwd(x, x, x, v, dout=x),
             lambda: m.gated_state_update(x[..., 0], x[..., 0], x[..., 0], x[..., 0], v),
             lambda: m.mssm_w4_linear(x[0], v, v, None, 32, None, x[0])):
    try:
        call()
    except ImportError as e:
        assert "_marshal.so" in str(e) and e.__cause__ is not None
    else:
        raise AssertionError("no error")
""")
    assert r.returncode == 0, r.stderr


def test_a_build_without_a_compiler_for_it_keeps_the_library(monkeypatch):
    import importlib.util
    spec = importlib.util.spec_from_file_location("_mssm_build", os.path.join(ROOT, PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    monkeypatch.setenv("CXX", "/bin/false")
    monkeypatch.setattr(build, "MARSHAL", os.path.join(ROOT, PKG, "_marshal_absent.so"))
    with pytest.warns(UserWarning, match="_marshal.so"):
        assert build.build() == build.LIB
    assert not os.path.exists(build.MARSHAL)
