"""The gated recurrence at the edges of what its interface allows."""
import pytest
import torch

import gated_ref as ref
from test_parity_gated import args, tensors

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
