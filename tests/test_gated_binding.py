"""The binding of the gated recurrence and the 4-bit linear map: what a failed call leaves behind."""
import gc

import numpy as np
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


def streams():
    side = torch.cuda.Stream()
    return (None, side, side.cuda_stream, np.int64(side.cuda_stream), torch.cuda.default_stream(), 0)


def test_errors_are_the_same_on_every_stream(cuda_device):
    import selective_state_space_46_b200 as m
    x, lam = inputs(2, 8, 64)
    flat = x[..., 0].contiguous()
    codes, scales = torch.zeros(16, 32, device="cuda", dtype=torch.uint8), torch.ones(16, 1, device="cuda")
    weight = m.w4_pack(codes, scales, group_size=64)
    for s in streams():
        for bad in (x[0], x[None], lam):
            with pytest.raises(ValueError, match="Bt, D, L"):
                m.gated_scan_fwd(bad, x, x, lam, stream=s)
            with pytest.raises(ValueError, match="Bt, D, L"):
                m.gated_scan_bwd(bad, x, x, lam, dout=x, stream=s)
        with pytest.raises(TypeError, match="expected a tensor"):
            m.gated_state_update(flat, [1.0], flat, flat, lam, stream=s)
        with pytest.raises(TypeError, match="expected a tensor"):
            m.gated_scan_fwd(x, x, x, lam, cu_seqlens=[0, 64], stream=s)
        with pytest.raises(ValueError, match="CUDA"):
            m.gated_scan_fwd(x.cpu(), x, x, lam, stream=s)
        with pytest.raises(m.MssmError):
            m.gated_state_update(flat, x[..., 0, None], flat, flat, lam, stream=s)
        with pytest.raises(m.MssmError):
            m.gated_scan_bwd(x, x, x, lam, stream=s)
        with pytest.raises(m.MssmError):
            m.w4_linear(torch.zeros(2, 64, device="cuda"), weight, bias=lam, stream=s)


def test_outputs_belong_to_the_stream_of_the_call(cuda_device):
    """What a call allocates lies in its stream's part of the memory, so that freeing it orders with the call."""
    import selective_state_space_46_b200 as m
    x, lam = inputs(2, 40, 1 << 16)
    flat = torch.randn(1, 1 << 22, device="cuda")
    codes, scales = torch.zeros(1 << 21, 32, device="cuda", dtype=torch.uint8), torch.ones(1 << 21, 1, device="cuda")
    weight = m.w4_pack(codes, scales, group_size=64)
    tokens = torch.randn(1, 64, device="cuda")
    torch.cuda.synchronize()

    def owner(t):
        for seg in torch.cuda.memory_snapshot():
            if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
                return seg["stream"]
        raise AssertionError("not in the allocator's memory")

    for s in streams():
        raw = 0 if s is None else s.cuda_stream if isinstance(s, torch.cuda.Stream) else int(s)
        out, last = m.gated_scan_fwd(x, x, x, lam, stream=s)
        g = m.gated_scan_bwd(x, x, x, lam, z=x, dout=x, h0=torch.zeros(2, 40, device="cuda"), stream=s)
        step = m.gated_state_update(torch.zeros_like(flat), flat, flat, flat, flat[0], stream=s)
        y = m.w4_linear(tokens, weight, stream=s)
        packed = m.w4_pack(codes, scales, group_size=64, stream=s)
        torch.cuda.synchronize()
        made = [out, last, y, step, packed.qweight, packed.qscales] + [v for v in g.values() if v is not None]
        assert {owner(t) for t in made} == {raw}
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
