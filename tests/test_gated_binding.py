"""The binding of the gated recurrence and the 4-bit linear map: what a failed call leaves behind."""
import gc

import pytest
import torch

pytestmark = pytest.mark.gpu

MB = 1 << 20


@pytest.fixture
def little_memory(cuda_device):
    """limit(bytes): that much more memory for torch than it holds now."""
    def limit(nbytes):
        gc.collect()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        total = torch.cuda.get_device_properties(cuda_device).total_memory
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + nbytes) / total, cuda_device)

    yield limit
    torch.cuda.set_per_process_memory_fraction(1.0, cuda_device)
    torch.cuda.empty_cache()


def inputs(Bt, D, L):
    x = torch.randn(Bt, D, L, device="cuda")
    return x, torch.zeros(D, device="cuda")


@pytest.mark.parametrize("room", [0.5, 1.5, 2.5, 3.5])
def test_a_backward_that_runs_out_of_memory_keeps_nothing(little_memory, room):
    """Each gradient of 64 MB; `room` says how many of the four fit."""
    import selective_state_space_46_b200 as m
    x, lam = inputs(2, 64, 1 << 17)
    size = x.numel() * 4
    little_memory(int(room * size) // (2 * MB) * (2 * MB))
    before = torch.cuda.memory_allocated()
    for _ in range(2):
        with pytest.raises(torch.cuda.OutOfMemoryError):
            m.gated_scan_bwd(x, x, x, lam, z=x, dout=x, h0=lam.expand(2, 64))
        gc.collect()
        assert torch.cuda.memory_allocated() == before


def test_a_scan_that_runs_out_of_memory_keeps_nothing(little_memory):
    """`out` of 2 MB fits, last_state of 64 MB does not."""
    import selective_state_space_46_b200 as m
    x, lam = inputs(1, 16, 1 << 15)
    cu = torch.zeros(2 ** 20 + 1, device="cuda", dtype=torch.int32)
    cu[-1] = x.shape[2]
    little_memory(32 * MB)
    before = torch.cuda.memory_allocated()
    with pytest.raises(torch.cuda.OutOfMemoryError):
        m.gated_scan_fwd(x, x, x, lam, cu_seqlens=cu)
    gc.collect()
    assert torch.cuda.memory_allocated() == before


def test_a_refused_call_keeps_nothing(cuda_device):
    import selective_state_space_46_b200 as m
    x, lam = inputs(2, 64, 4096)
    gc.collect()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(3):
        with pytest.raises(m.MssmError):
            m.gated_scan_bwd(x, x, x, lam[:5], dout=x)
        with pytest.raises(m.MssmError):
            m.gated_scan_fwd(x, x, x, lam, c=-1.0)
        with pytest.raises(m.MssmError):
            m.gated_state_update(x[..., 0], x[..., 0], x[..., 0], x[..., 0], lam[:3])
    gc.collect()
    assert torch.cuda.memory_allocated() == before
