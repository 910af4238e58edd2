"""The packed sequences' walk of the gated scans, run on the host lane by lane (tests/host_warp.cpp): every window's masks
against the definition, and no read or step outside the arrays whatever the offsets hold."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WINDOW, STEPS = 256, 8
INT_MIN, INT_MAX = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("host") / "host_warp.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-fPIC", "-shared", "-fno-strict-aliasing",
                    "-I" + os.path.join(ROOT, "selective_state_space_46_b200", "csrc"),
                    os.path.join(ROOT, "tests", "host_warp.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


def walk(host, cu, L, off=0, stride=WINDOW, back=False):
    """The masks of the windows that cover a row of L steps and the ones behind it, by step."""
    cu = np.asarray(cu, np.int64).astype(np.int32)
    n = -(-(L + off) // stride) + 1
    first, step = (-off, stride) if not back else (-off + (n - 1) * stride, -stride)
    whole, valid, starts, ends = (np.zeros((n, 32), np.int32) for _ in range(4))
    seq = np.zeros((n, 32, STEPS), np.int32)
    p = [v.ctypes.data_as(ctypes.c_void_p) for v in (cu, whole, valid, starts, ends, seq)]
    assert host.walk_windows(p[0], len(cu) - 1, L, first, step, n, *p[1:]) == 0
    order = slice(None, None, -1) if back else slice(None)
    bits = [(v[order, :, None] >> np.arange(STEPS) & 1).reshape(n, WINDOW).astype(bool) for v in (valid, starts, ends)]
    assert all((v >> STEPS == 0).all() for v in (valid, starts, ends))
    t = (np.arange(n) * stride - off)[:, None] + np.arange(WINDOW)
    return t, whole[order, 0].astype(bool), *bits, seq[order].reshape(n, WINDOW)


def check_against_definition(host, cu, L, off, stride, back):
    t, whole, valid, starts, ends, seq = walk(host, cu, L, off, stride, back)
    cu = np.asarray(cu)
    inside = (t >= cu[0]) & (t < cu[-1])
    np.testing.assert_array_equal(valid, inside)
    np.testing.assert_array_equal(starts, inside & np.isin(t, cu[:-1]))
    np.testing.assert_array_equal(ends, inside & np.isin(t + 1, cu[1:]))
    np.testing.assert_array_equal(seq[inside], (np.searchsorted(cu, t, "right") - 1)[inside])
    one = inside.all(1) & ~starts.any(1) & ~ends.any(1)
    assert not (whole & ~one).any()


OFFSETS = {
    "one": [0, 2000],
    "inner": [300, 301, 1500],
    "empty": [0, 0, 0, 700, 700, 1800, 1800],
    "short": list(range(0, 900, 3)) + [900, 1900],
    "single steps": list(range(0, 600)) + [2000],
    "ends of windows": [0, 256, 512, 513, 1024, 2048],
}


@pytest.mark.parametrize("name", sorted(OFFSETS))
@pytest.mark.parametrize("back", [False, True])
def test_masks(host, name, back):
    cu = OFFSETS[name]
    for off in (0, 1, 7):
        for stride in (WINDOW, 4 * WINDOW):
            check_against_definition(host, cu, 2048 + 13, off, stride, back)


def test_masks_of_random_sequences(host):
    rng = np.random.default_rng(1)
    for n in (1, 2, 31, 32, 33, 64, 70):
        for _ in range(6):
            L = int(rng.integers(1, 5000))
            cu = np.sort(rng.integers(0, L + 1, n + 1))
            check_against_definition(host, cu, L, int(rng.integers(0, 8)), WINDOW, bool(rng.integers(2)))


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("S", [1, 30, 31, 32, 33, 63, 64, 65, 96])
def test_windows_inside_one_sequence_are_whole(host, S, back):
    """Every window without a boundary takes the way without masks, whichever sequence it lies in."""
    for stride in (WINDOW, 2 * WINDOW):
        cu = np.arange(S + 1) * 1000
        t, whole, valid, starts, ends, _ = walk(host, cu, int(cu[-1]), 0, stride, back)
        one = valid.all(1) & ~starts.any(1) & ~ends.any(1)
        assert one.sum() >= S // (stride // WINDOW)
        np.testing.assert_array_equal(whole, one)


WILD = [[0, INT_MIN], [0, INT_MIN, INT_MIN], [INT_MAX, INT_MAX], [INT_MAX, 50], [INT_MIN, INT_MAX], [INT_MAX, INT_MIN],
        [INT_MIN, 20, INT_MAX], [0, 60], [-3, 20, 50], [50, 40, 30, 20, 10, 0], [70, 80, 90], [0, INT_MAX, 0, INT_MIN, 50],
        [0] + [INT_MIN] * 40 + [50], [0] + [INT_MAX] * 40 + [50], list(range(70, 0, -1))]


@pytest.mark.parametrize("cu", WILD, ids=range(len(WILD)))
@pytest.mark.parametrize("back", [False, True])
def test_wrong_offsets_stay_inside_the_row(host, cu, back):
    """Whatever the offsets hold: no step outside the row, no sequence outside the array (states are indexed with it)."""
    for L in (1, 50, 300, 1000):
        for off in (0, 1, 7):
            t, _, valid, starts, ends, seq = walk(host, cu, L, off, back=back)
            assert not (valid & ((t < 0) | (t >= L))).any()
            assert not ((starts | ends) & ~valid).any()
            assert seq.min() >= 0 and seq.max() < len(cu) - 1
