"""What the library launches, without a GPU: its own host code against a runtime that records (tests/fake_cudart.cpp)."""
import importlib.util
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    spec = importlib.util.spec_from_file_location(
        "_mssm_build", os.path.join(ROOT, "selective_state_space_46_b200", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    so = str(tmp_path_factory.mktemp("fake") / "libfake.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc()))), "include")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-Wl,--no-undefined",
                    "-I" + cuda, os.path.join(ROOT, "tests", "fake_cudart.cpp"), *build.compile_objects(), "-o", so], check=True)
    return so


PRELUDE = """
import ctypes, json, sys
sys.path[:0] = [{tests!r}, {root!r}]
lib = ctypes.CDLL({so!r})
lib.fake_kernel.restype = lib.mssm_last_error.restype = ctypes.c_char_p
from test_abi_host import mk
F32, BF16, I32, U8 = 0, 1, 2, 3
V = ctypes.c_void_p

def ref(t):
    return None if t is None else ctypes.byref(t)

def last():
    v = (ctypes.c_uint * 5)()
    lib.fake_last(v)
    return dict(zip(("grid", "grid_y", "threads", "smem", "cluster"), v), kernel=lib.fake_kernel().decode(), count=lib.fake_launches())

def linear(M, K, N, group, dt=BF16, zeros=False):
    lib.mssm_w4_packed_sizes.argtypes = [ctypes.c_int64] * 3 + [ctypes.POINTER(ctypes.c_int64)] * 2
    lib.mssm_w4_linear.argtypes = [V] * 4 + [ctypes.c_int64] + [V] * 3
    q, s = ctypes.c_int64(), ctypes.c_int64()
    assert lib.mssm_w4_packed_sizes(N, K, group, q, s) == 0
    st = lib.mssm_w4_linear(ref(mk([M, K], dt)), ref(mk([q.value], I32)), ref(mk([s.value], dt)),
                            ref(mk([s.value], U8)) if zeros else None, group, None, ref(mk([M, N], dt)), None)
    return st
"""


def run(so, body):
    """`body`, which leaves a JSON-able `result`, in a process that has the recording library alone."""
    code = PRELUDE.format(tests=os.path.join(ROOT, "tests"), root=ROOT, so=so) + body + "\nprint(json.dumps(result))\n"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout.splitlines()[-1])


def test_linear_launches_after_shutdown_and_reset(fake):
    """A device reset drops the kernels' shared-memory limits; mssm_shutdown before it makes the library set them again."""
    got = run(fake, """
result = []
for device in (0, 3, 0):
    lib.fake_device(device)
    for again in range(2):
        result += [linear(3, 1001, 193, 32, F32), linear(24, 999, 300, 96, zeros=True), linear(1, 5120, 20480, 128)]
    result.append(last()["smem"] > 48 * 1024)
    lib.mssm_shutdown()
    lib.fake_reset()
""")
    assert got == ([0] * 6 + [True]) * 3


def test_a_forced_split_keeps_every_row(fake):
    """Rows times CTAs a row stay within a grid, and every row keeps its CTAs."""
    got = run(fake, """
result = []
lib.mssm_set_option.argtypes = [ctypes.c_int, ctypes.c_int64]
for D in (4, (1 << 28) - 1, (1 << 28) + 5, (1 << 29) + 8, (1 << 30) + 8, (1 << 31) - 1):
    wide = [mk([1, D, 1], BF16) for _ in range(4)]
    for k, t in enumerate(wide):
        t.data = (1 << 40) * (k + 1)
    lam = mk([D], F32, [0])
    for split in (0, 2, 8):
        assert lib.mssm_set_option(10, split) == 0
        st = lib.mssm_gated_scan_fwd(ref(wide[0]), ref(wide[1]), ref(wide[2]), ref(lam), None, None, None, None, ref(wide[3]), None, None)
        l = last()
        per = 4 if l["threads"] == 128 and l["cluster"] == 1 else 1
        result.append([st, l["grid"] % l["cluster"], l["grid"] // l["cluster"] * per >= D])
""")
    assert got == [[0, 0, True]] * 18


def test_linear_plan_counts_the_ctas_it_launches(fake):
    """Two tiles of outputs a CTA wherever one tile a CTA would give every SM one or more, in either type."""
    got = run(fake, """
result = []
for dt in (F32, BF16):
    for M in (1, 8, 16, 17, 24, 32, 33, 64, 100):
        for N in (64, 1536, 2048, 2352, 2368, 5120):
            assert linear(M, 2560, N, 128, dt) == 0
            l = last()
            tiles = (N + 15) // 16
            two = l["grid"] == (tiles + 1) // 2
            assert two or l["grid"] == tiles
            result.append([dt, M, N, two, tiles * l["grid_y"] >= 148])
""")
    assert [r for r in got if r[3] != r[4]] == []
