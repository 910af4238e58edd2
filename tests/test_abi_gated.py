"""Argument checks of the gated recurrence and the 4-bit linear map: refused on the host, no GPU needed (the
descriptors carry fake device pointers that nothing reads)."""
import ctypes

import pytest
import torch

import selective_state_space_46_b200 as m
from test_abi_host import INVALID, UNSUPPORTED, T, last_error, lib, mk  # noqa: F401  (lib: fixture)

F32, BF16, I32, U8 = 0, 1, 2, 3


class Ext(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("decay_scale", ctypes.c_float), ("h0", ctypes.POINTER(T)),
                ("cu_seqlens", ctypes.POINTER(T))]


def ref(t):
    return None if t is None else ctypes.byref(t)


def gated_args(Bt=2, D=8, L=32, S=None, dt=BF16):
    S = Bt if S is None else S
    a = {k: mk([Bt, D, L], dt) for k in ("x", "r", "i", "z", "out", "dout", "dx", "dr", "di", "dz")}
    a.update({k: mk([D], F32) for k in ("lam", "r_bias", "i_bias", "dlam", "dr_bias", "di_bias")})
    a.update({k: mk([S, D], F32) for k in ("last_state", "dlast_state", "dh0")})
    a["workspace"] = mk([3, Bt, D], F32)
    a["ext"] = Ext(ctypes.sizeof(Ext), 8.0, None, None)
    return a


def fwd(lib, a):  # noqa: F811
    return lib.mssm_gated_scan_fwd(*[ref(a[k]) for k in ("x", "r", "i", "lam", "r_bias", "i_bias", "z", "ext", "out",
                                                         "last_state")], None)


def bwd(lib, a):  # noqa: F811
    return lib.mssm_gated_scan_bwd(*[ref(a[k]) for k in (
        "x", "r", "i", "lam", "r_bias", "i_bias", "z", "ext", "dout", "dlast_state", "dx", "dr", "di", "dz", "dlam",
        "dr_bias", "di_bias", "dh0", "workspace")], None)


def strided(shape, dtype, stride):
    return mk(shape, dtype, stride=stride)


COMMON = [
    ("x", None, INVALID), ("lam", None, INVALID), ("r", mk([2, 8, 31], BF16), INVALID),
    ("i", mk([2, 8, 32], F32), INVALID), ("lam", mk([8], BF16), INVALID), ("r_bias", mk([7], F32), INVALID),
    ("x", strided([2, 8, 32], BF16, [512, 64, 2]), UNSUPPORTED),
    ("ext", Ext(4, 8.0, None, None), INVALID), ("ext", Ext(ctypes.sizeof(Ext), 0.0, None, None), INVALID),
    ("ext", Ext(ctypes.sizeof(Ext), -1.0, None, None), INVALID),
    ("ext", Ext(ctypes.sizeof(Ext), float("nan"), None, None), INVALID),
    ("ext", Ext(ctypes.sizeof(Ext), float("inf"), None, None), INVALID),
    ("ext", Ext(ctypes.sizeof(Ext), 8.0, ctypes.pointer(mk([3, 8], F32)), None), INVALID),
    ("ext", Ext(ctypes.sizeof(Ext), 8.0, None, ctypes.pointer(mk([3], I32))), INVALID),  # packed, but Bt = 2
]


@pytest.mark.parametrize("name,value,expect", COMMON + [
    ("out", None, INVALID), ("out", strided([2, 8, 32], BF16, [0, 32, 1]), INVALID),
    ("last_state", mk([2, 8], BF16), INVALID), ("last_state", mk([3, 8], F32), INVALID),
])
def test_forward_refuses(lib, name, value, expect):  # noqa: F811
    a = gated_args()
    a[name] = value
    assert fwd(lib, a) == expect, last_error(lib)
    assert last_error(lib)


@pytest.mark.parametrize("name,value,expect", COMMON + [
    ("dout", None, INVALID), ("dx", mk([2, 8, 32], F32), INVALID), ("dz", None, INVALID), ("dr_bias", None, INVALID),
    ("di_bias", None, INVALID), ("dlam", None, INVALID), ("dlam", strided([8], F32, [2]), UNSUPPORTED),
    ("dh0", mk([2, 9], F32), INVALID), ("workspace", None, INVALID), ("workspace", mk([3, 2, 7], F32), INVALID),
    ("workspace", strided([3, 2, 8], F32, [32, 8, 1]), UNSUPPORTED), ("dx", strided([2, 8, 32], BF16, [256, 0, 1]), INVALID),
])
def test_backward_refuses(lib, name, value, expect):  # noqa: F811
    a = gated_args()
    a[name] = value
    assert bwd(lib, a) == expect, last_error(lib)
    assert last_error(lib)


def test_aliases_are_refused(lib):  # noqa: F811
    a = gated_args()
    a["out"].data = a["x"].data + 64  # dense tensors whose bytes meet
    assert fwd(lib, a) == INVALID and "alias" in last_error(lib)
    a = gated_args()
    a["dr"].data = a["dx"].data
    assert bwd(lib, a) == INVALID and "alias" in last_error(lib)


def test_sizes_beyond_the_index_types_are_refused(lib):  # noqa: F811
    assert fwd(lib, gated_args(1 << 16, 1 << 15, 1)) == UNSUPPORTED
    assert fwd(lib, gated_args(1, 1, (1 << 31) - 100)) == UNSUPPORTED
    assert bwd(lib, gated_args(1, 1, (1 << 23) + 1)) == UNSUPPORTED


@pytest.mark.parametrize("call", [fwd, bwd])
def test_more_sequences_than_the_kernels_count_are_refused(lib, call):  # noqa: F811
    """The loops over the offsets add their stride to an index of 31 bits."""
    S = (1 << 31) - (1 << 16)
    a = gated_args(1, 1, 32, S)
    a["ext"] = Ext(ctypes.sizeof(Ext), 8.0, None, ctypes.pointer(mk([S + 1], I32)))
    assert call(lib, a) == UNSUPPORTED, last_error(lib)


def test_nothing_to_do_is_no_error(lib):  # noqa: F811
    for shape in ((0, 8, 32), (2, 0, 32)):
        assert fwd(lib, gated_args(*shape)) == 0
    assert bwd(lib, gated_args(2, 0, 32)) == 0


def test_step_refuses(lib):  # noqa: F811
    f = lib.mssm_gated_state_update
    f.argtypes = [ctypes.c_void_p] * 8 + [ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p]

    def call(scale=8.0, **over):
        a = dict(state=mk([4, 8], F32), lam=mk([8], F32), r_bias=mk([8], F32), i_bias=mk([8], F32),
                 **{k: mk([4, 8], BF16) for k in ("x", "r", "i", "z", "out")})
        a.update(over)
        return f(*[ref(a[k]) for k in ("state", "x", "r", "i", "lam", "r_bias", "i_bias", "z")], scale, ref(a["out"]),
                 None)

    assert call(state=mk([4, 8], BF16)) == INVALID
    assert call(state=strided([4, 8], F32, [0, 1])) == INVALID
    assert call(r=mk([4, 7], BF16)) == INVALID
    assert call(z=mk([4, 8], F32)) == INVALID
    assert call(scale=0.0) == INVALID
    x = mk([4, 8], BF16)
    assert call(x=x, out=x) == INVALID
    assert call(**{k: mk([1 << 16, 1 << 15], BF16) for k in ("x", "r", "i", "z", "out")}, state=mk([1 << 16, 1 << 15], F32),
                **{k: mk([1 << 15], F32) for k in ("lam", "r_bias", "i_bias")}) == UNSUPPORTED


def test_w4_refuses(lib):  # noqa: F811
    sizes = lib.mssm_w4_packed_sizes
    sizes.argtypes = [ctypes.c_int64] * 3 + [ctypes.POINTER(ctypes.c_int64)] * 2
    q, s = ctypes.c_int64(), ctypes.c_int64()
    assert sizes(17, 65, 128, q, s) == 0
    assert (q.value, s.value) == (2 * 2 * 128, 2 * 1 * 16)
    assert sizes(17, 65, 32, q, s) == 0
    assert (q.value, s.value) == (2 * 2 * 128, 2 * 4 * 16)
    for bad in ((0, 64, 32), (16, 0, 32)):
        assert sizes(*bad, q, s) == INVALID
    for bad in ((16, 64, 0), (16, 64, 48), (16, 64, -32), (1 << 31, 64, 32), (16, 1 << 31, 32)):
        assert sizes(*bad, q, s) == UNSUPPORTED

    pack = lib.mssm_w4_pack
    pack.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_int64] * 2 + [ctypes.c_void_p] * 4

    def call_pack(k=65, group=32, **over):
        a = dict(codes=mk([17, 33], U8), scales=mk([17, 3], BF16), zeros=mk([17, 3], U8), qweight=mk([512], I32),
                 qscales=mk([128], BF16), qzeros=mk([128], U8))
        a.update(over)
        return pack(ref(a["codes"]), ref(a["scales"]), ref(a["zeros"]), k, group, ref(a["qweight"]), ref(a["qscales"]),
                    ref(a["qzeros"]), None)

    assert call_pack(codes=mk([17, 32], U8)) == INVALID
    assert call_pack(codes=mk([17, 33], I32)) == INVALID
    assert call_pack(scales=mk([17, 2], BF16)) == INVALID
    assert call_pack(scales=mk([17, 3], U8)) == INVALID
    assert call_pack(qzeros=None) == INVALID
    assert call_pack(zeros=None) == INVALID
    assert call_pack(qweight=mk([511], I32)) == INVALID
    assert call_pack(qscales=mk([128], F32)) == INVALID
    assert call_pack(group=40) == UNSUPPORTED

    lin = lib.mssm_w4_linear
    lin.argtypes = [ctypes.c_void_p] * 4 + [ctypes.c_int64] + [ctypes.c_void_p] * 3

    def call_lin(group=32, **over):
        a = dict(x=mk([3, 65], BF16), qweight=mk([512], I32), qscales=mk([128], F32), qzeros=mk([128], U8),
                 bias=mk([17], F32), out=mk([3, 17], BF16))
        a.update(over)
        return lin(ref(a["x"]), ref(a["qweight"]), ref(a["qscales"]), ref(a["qzeros"]), group, ref(a["bias"]),
                   ref(a["out"]), None)

    assert call_lin(x=None) == INVALID
    assert call_lin(x=mk([3, 130], BF16)) == INVALID      # another K than the packed one
    assert call_lin(out=mk([3, 33], BF16)) == INVALID     # another N
    assert call_lin(out=mk([4, 17], BF16)) == INVALID
    assert call_lin(out=mk([3, 17], F32)) == INVALID
    assert call_lin(group=64) == INVALID                  # another group
    assert call_lin(bias=mk([17], BF16)) == INVALID
    assert call_lin(x=strided([3, 65], BF16, [130, 2])) == UNSUPPORTED
    assert call_lin(out=strided([3, 17], BF16, [0, 1])) == INVALID
    odd = mk([512], I32)
    odd.data += 4
    assert call_lin(qweight=odd) == UNSUPPORTED
    assert call_lin(x=mk([1 << 20, 65], BF16), out=mk([1 << 20, 17], BF16)) == UNSUPPORTED
    assert call_lin(x=mk([0, 65], BF16), out=mk([0, 17], BF16)) == 0


def test_cpu_tensors_are_refused():
    x, v, s = torch.zeros(2, 8, 32), torch.zeros(8), torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        m.gated_scan_fwd(x, x, x, v)
    with pytest.raises(ValueError, match="CUDA"):
        m.gated_scan_bwd(x, x, x, v, dout=x)
    with pytest.raises(ValueError, match="CUDA"):
        m.gated_state_update(s, s, s, s, v)
    with pytest.raises(ValueError, match="CUDA"):
        m.w4_pack(torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(16, 1), group_size=64)


def test_plan_options(lib):  # noqa: F811
    for opt, good, bad in ((9, (1, 2, 4, 8, 0), (-1, 3, 16)), (10, (1, 2, 4, 8, 0), (-1, 3, 16)), (11, (2, 8, 16, 0), (-1, 1, 4)),
                           (12, (1, 2, 0), (-1, 3, 4))):
        lib.mssm_set_option.argtypes = [ctypes.c_int, ctypes.c_int64]
        for v in bad:
            assert lib.mssm_set_option(opt, v) == INVALID
        for v in good:
            assert lib.mssm_set_option(opt, v) == 0


def test_kernel_kinds(lib):  # noqa: F811
    """The kinds that mssm_kernel_stats fills stay five; the newer ones are counted by mssm_kernel_stats_all."""
    guard = (ctypes.c_int64 * 9)(*[77] * 9)
    assert lib.mssm_kernel_stats(guard, None, None, 0) == 0
    assert list(guard)[5:] == [77] * 4
    assert lib.mssm_kernel_stats_all(9, guard, None, None, 0) == 0
    assert 77 not in list(guard)
    assert lib.mssm_kernel_stats_all(10, guard, None, None, 0) == INVALID
    assert set(m.mssm_kernel_stats()) == set(m.KERNEL_KINDS) and len(m.KERNEL_KINDS) == 9
