"""The gated recurrence at the edges of what its interface allows."""
import numpy as np
import pytest
import torch

import gated_ref as ref
from test_parity_gated import args, check_bwd, check_fwd, tensors

pytestmark = pytest.mark.gpu

INT_MIN, INT_MAX = -2 ** 31, 2 ** 31 - 1


class Guarded:
    """Views in the middle of a filled buffer, and whether anything around them was written."""

    def __init__(self, fill=3.0):
        self.fill, self.held = fill, []

    def view(self, *shape, dtype=torch.float32, gap=600):
        """A tensor whose rows (along the last axis) lie `gap` elements apart, with room in front and behind."""
        row = shape[-1] + gap
        n = row + gap
        for s in shape[:-1]:
            n *= s
        buf = torch.full((n + 2 * row,), self.fill, device="cuda", dtype=dtype)
        strides = [1]
        for s in reversed(shape[1:]):
            strides.insert(0, strides[0] * (s if len(strides) > 1 else row))
        v = buf.as_strided(shape, strides, row)
        self.held.append((buf, shape, strides, row))
        return v

    def untouched(self):
        for buf, shape, strides, at in self.held:
            rest = buf.clone()
            rest.as_strided(shape, strides, at).fill_(self.fill)
            if not bool((rest == self.fill).all()):
                return False
        return True


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", [50, 1000])
@pytest.mark.parametrize("warps", [0, 1, 8])
def test_wrong_offsets_write_nothing_around_the_outputs(cuda_device, io, L, warps):
    """Offsets far outside the row: reported, and every element around out, the gradients and the states is left."""
    import selective_state_space_46_b200 as m
    D = 4
    d = tensors(ref.gated_inputs(1, D, L, io, seed=30), io)
    dt = d["x"].dtype
    m.mssm_set_option(m.MSSM_OPT_GATED_WARPS, warps)
    try:
        for cu in ([0, INT_MIN], [INT_MAX, INT_MAX], [INT_MAX, L], [0, INT_MAX], [INT_MIN, 20, INT_MAX],
                   [0, INT_MAX, 0, INT_MIN, L], [0] + [INT_MIN] * 40 + [L]):
            n = len(cu) - 1
            g = Guarded()
            cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
            h0, dlast = torch.randn(n, D, device="cuda"), torch.randn(n, D, device="cuda")
            m.mssm_get_error()
            m.gated_scan_fwd(*args(d), h0=h0, cu_seqlens=cu_t, out=g.view(1, D, L, dtype=dt), last_state=g.view(n, D))
            with pytest.raises(m.MssmError):
                m.mssm_get_error()
            wide = [g.view(1, D, L, dtype=dt) for _ in range(4)]
            m.mssm_gated_scan_bwd(*args(d), d["x"], dlast, *wide, *[g.view(D) for _ in range(3)], g.view(n, D), h0=h0,
                                  cu_seqlens=cu_t)
            with pytest.raises(m.MssmError):
                m.mssm_get_error()
            assert g.untouched(), cu
    finally:
        m.mssm_set_option(m.MSSM_OPT_GATED_WARPS, 0)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [False, True])
def test_rates_beyond_every_decay(cuda_device, io, packed):
    """Rates that leave no memory (a = 0, beta = 1), up to the largest numbers and infinity: the same bits as a rate of
    10^4, no NaN, and no gradient for r and lam."""
    import selective_state_space_46_b200 as m
    L = 700
    p = ref.gated_inputs(1, 6, L, io, h0=True, cu=[0, 300, 301, 690] if packed else None, seed=31)
    p["r"] = np.abs(p["r"])  # r >= 1/2: y >= 5000
    p["r_bias"][:] = 0.0
    d = tensors(p, io)
    n = 3 if packed else 1
    dlast = torch.randn(n, 6, device="cuda")
    keep = slice(0, 690 if packed else L)

    def run(lam):
        d["lam"] = torch.full((6,), lam, device="cuda")
        out, last = m.gated_scan_fwd(*args(d), h0=d["h0"], cu_seqlens=d["cu"])
        g = m.gated_scan_bwd(*args(d), dout=d["x"], h0=d["h0"], cu_seqlens=d["cu"], dlast_state=dlast)
        return [out[..., keep], last] + [v[..., keep] if v.dim() == 3 else v for v in g.values()], g

    want, g = run(1250.0)
    assert all(bool(torch.isfinite(v).all()) for v in want)
    assert not g["dr"][..., keep].any() and not g["dlam"].any() and not g["dr_bias"].any() and not g["dh0"].any()
    for lam in (1e11, 1.5e11, 1e20, 1e30, 1e34, 4e37, 3e38, float("inf")):
        got, _ = run(lam)
        for a, b in zip(got, want):
            assert torch.equal(a, b), lam


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_largest_rates_behind_gates_that_are_almost_shut(cuda_device, io):
    """Rates around 2^40 and far above it, with gates as small as their reciprocals, so that every decay is met."""
    p = ref.gated_inputs(1, 8, 500, io, h0=True, seed=32)
    rates = np.array([2.0 ** 39, 2.0 ** 40, 2.0 ** 40.1, 2.0 ** 41, 1e20, 1e28, 1e31, 1e33])
    p["lam"] = np.float32(rates / p["c"]).astype(np.float64)
    p["r_bias"] = np.float32(-np.log(p["lam"] * p["c"])).astype(np.float64)
    check_fwd(p, io)
    check_bwd(p, io, dlast=True)
