"""The fp64 references of the gated recurrence and the 4-bit linear map: pinned to closed forms and finite
differences, on the CPU."""
import numpy as np
import pytest

import gated_ref as ref


def test_constant_decay_is_a_geometric_sum():
    p = ref.gated_inputs(1, 3, 40, gate=False, bias=False, seed=1)
    p["r"][:], p["i"][:], p["x"][:] = 0.3, -0.2, 1.0
    out = ref.forward(p, "f32")["out"][0]
    a = np.exp(-8 * np.log1p(np.exp(p["lam"])) / (1 + np.exp(-0.3)))
    gain = np.sqrt(1 - a * a) / (1 + np.exp(0.2))
    k = np.arange(1, 41)
    want = gain[:, None] * (1 - a[:, None] ** k) / (1 - a[:, None])
    assert np.allclose(out[0], want, rtol=1e-10)


def test_packed_sequences_are_separate_scans():
    cu = [0, 5, 5, 6, 30]
    p = ref.gated_inputs(1, 4, 30, h0=True, cu=cu, seed=2)
    full = ref.forward(p, "f32")
    for s in range(4):
        q = dict(p, cu=None, h0=p["h0"][s:s + 1])
        for k in ("x", "r", "i", "z"):
            q[k] = p[k][:, :, cu[s]:cu[s + 1]]
        one = ref.forward(q, "f32")
        assert np.array_equal(one["out"][0], full["out"][0][:, :, cu[s]:cu[s + 1]])
        assert np.array_equal(one["last_state"][0][0], full["last_state"][0][s])


@pytest.mark.parametrize("cu", [None, [1, 4, 4, 9]])
def test_gradients_against_differences(cu):
    """Every gradient against a central difference of the loss it is the gradient of."""
    p = ref.gated_inputs(1 if cu else 2, 3, 10, h0=True, cu=cu, seed=3)
    rng = np.random.default_rng(4)
    first = ref.forward(p, "f32")
    dout = rng.standard_normal(first["out"][0].shape)
    dlast = rng.standard_normal(first["last_state"][0].shape)
    if cu:  # nothing outside the sequences enters the loss
        dout[:, :, :cu[0]] = dout[:, :, cu[-1]:] = 0

    def loss(q):
        f = ref.forward(q, "f32")
        return np.sum(f["out"][0] * dout) + np.sum(f["last_state"][0] * dlast)

    g = ref.backward(p, dout, dlast, "f32")
    names = dict(dx="x", dr="r", di="i", dz="z", dlam="lam", dr_bias="r_bias", di_bias="i_bias", dh0="h0")
    assert set(g) == set(names)
    step = 1e-6
    for gn, n in names.items():
        flat = g[gn][0].reshape(-1)
        for at in rng.choice(flat.size, min(flat.size, 12), replace=False):
            both = []
            for sign in (1, -1):
                v = p[n].copy()
                v.reshape(-1)[at] += sign * step
                both.append(loss(dict(p, **{n: v})))
            diff = (both[0] - both[1]) / (2 * step)
            # the difference's own error: rounding 1e-16 |loss| / step and curvature step^2
            assert abs(diff - flat[at]) <= 1e-8 * (1 + abs(loss(p))) + 1e-7 * abs(flat[at]), (gn, at)


def test_w4_dequantise_by_hand():
    codes = np.array([[0x21, 0x03]], np.uint8)  # 1, 2, 3
    w = ref.w4_dequantise(codes, np.array([[0.5]]), None, 3, 32)
    assert np.array_equal(w, [[-3.5, -3.0, -2.5]])
    w = ref.w4_dequantise(codes, np.array([[2.0]]), np.array([[1]], np.uint8), 3, 32)
    assert np.array_equal(w, [[0.0, 2.0, 4.0]])


def test_bf16_rounding():
    v = np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -2.5, 1 + 2.0 ** -9])
    assert np.array_equal(ref.to_bf16(v), [1.0, 1.0, 1 + 2.0 ** -6, -2.5, 1.0])
