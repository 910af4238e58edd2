"""GPU parity of the gated linear recurrence (scan, backward, decode step) with its fp64 reference, within
the bounds that the reference derives for the kernels' arithmetic (tests/gated_ref.py)."""
import numpy as np
import pytest
import torch

import gated_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(v, io=None):
    if v is None:
        return None
    t = torch.from_numpy(np.array(v)).cuda()
    return t if v.dtype == np.int32 else t.to(TYPES[io or "f32"])


def tensors(p, io):
    d = {k: dev(p[k], io) for k in ("x", "r", "i", "z")}
    d.update({k: dev(p[k]) for k in ("lam", "r_bias", "i_bias", "h0", "cu")})
    return d


def args(d):
    return [d[k] for k in ("x", "r", "i", "lam", "r_bias", "i_bias", "z")]


def within(got, want, name, mask=None):
    v, bound = want
    g = got.detach().double().cpu().numpy()
    assert g.shape == v.shape, name
    err = np.abs(g - v)
    bad = ~(err <= bound)
    if mask is not None:
        bad &= mask
    if bad.any():
        at = tuple(int(k) for k in np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} out of bounds, first at {at}: "
                             f"got {g[at]!r}, want {v[at]!r} +- {np.broadcast_to(bound, v.shape)[at]:.3e}")


def run_fwd(p, io, **kw):
    import selective_state_space_46_b200 as m
    d = tensors(p, io)
    out, last = m.gated_scan_fwd(*args(d), c=p["c"], h0=d["h0"], cu_seqlens=d["cu"], **kw)
    torch.cuda.synchronize()
    m.mssm_get_error()
    return out, last


def check_fwd(p, io):
    out, last = run_fwd(p, io)
    want = ref.forward(p, io)
    mask = inside(p)
    within(out, want["out"], "out", mask)
    within(last, want["last_state"], "last_state")


def inside(p):
    if p["cu"] is None:
        return np.ones((1, 1, 1), bool)
    mask = np.zeros((1, 1, p["x"].shape[2]), bool)
    mask[..., p["cu"][0]:p["cu"][-1]] = True
    return mask


def check_bwd(p, io, dlast=False, seed=9):
    import selective_state_space_46_b200 as m
    rng = np.random.default_rng(seed)
    dout = rng.standard_normal(p["x"].shape)
    dout = ref.to_bf16(dout) if io == "bf16" else np.float32(dout).astype(np.float64)
    seqs = p["x"].shape[0] if p["cu"] is None else len(p["cu"]) - 1
    dl = np.float32(rng.standard_normal((seqs, p["x"].shape[1]))).astype(np.float64) if dlast else None
    d = tensors(p, io)
    g = m.gated_scan_bwd(*args(d), dout=dev(dout, io), c=p["c"], h0=d["h0"], cu_seqlens=d["cu"], dlast_state=dev(dl))
    torch.cuda.synchronize()
    m.mssm_get_error()
    want = ref.backward(p, dout, dl, io)
    mask = inside(p)
    assert {k for k, v in g.items() if v is not None} == set(want)
    for k, w in want.items():
        within(g[k], w, k, mask if w[0].ndim == 3 else None)


LENGTHS = [0, 1, 2, 7, 8, 9, 31, 64, 65, 255, 256, 257, 1000, 1023, 1024, 1025, 2049, 4097]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", LENGTHS)
def test_scan_lengths(cuda_device, L, io):
    check_fwd(ref.gated_inputs(2, 5, L, io, gate=L % 2 == 1, h0=L % 3 == 0, seed=L), io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", LENGTHS)
def test_bwd_lengths(cuda_device, L, io):
    check_bwd(ref.gated_inputs(2, 5, L, io, gate=L % 2 == 1, h0=L % 3 != 1, seed=L), io, dlast=L % 3 != 2)


@pytest.mark.parametrize("shape", [(1, 1, 20000), (1, 3, 40001), (3, 700, 300), (1, 2048, 600), (2, 1200, 520),
                                   (1, 300, 9000), (40, 64, 33), (500, 9, 16)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_shapes(cuda_device, shape, io):
    check_fwd(ref.gated_inputs(*shape, io, seed=sum(shape)), io)


@pytest.mark.parametrize("shape", [(1, 1, 20000), (1, 3, 40001), (3, 700, 300), (1, 2048, 600), (2, 1200, 520),
                                   (1, 300, 9000), (40, 64, 33), (500, 9, 16)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_bwd_shapes(cuda_device, shape, io):
    check_bwd(ref.gated_inputs(*shape, io, seed=sum(shape)), io)


OFFSETS = {
    "ragged": [0, 5, 5, 6, 14, 22, 85, 86, 150, 1177, 1177, 1180, 3000],
    "inner": [3, 3, 40, 41, 299, 300],       # steps before and behind the sequences
    "singles": list(range(0, 70)),
    "one": [0, 777],
    "empty": [0, 0, 0],
    "empty_then_all": [0, 0, 2100, 2100],
}


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("name", sorted(OFFSETS))
@pytest.mark.parametrize("h0", [False, True])
@pytest.mark.parametrize("dim", [3, 1900])
def test_packed(cuda_device, name, io, h0, dim):
    cu = OFFSETS[name]
    T = cu[-1] + (9 if name in ("inner", "empty") else 0)
    if dim > 1000 and T > 1000:
        T, cu = 300, [min(c, 300) for c in cu]
    p = ref.gated_inputs(1, dim, T, io, gate=name != "one", h0=h0, cu=cu, seed=T + dim)
    check_fwd(p, io)
    check_bwd(p, io, dlast=h0)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", [6000, 70001])
def test_packed_long_rows(cuda_device, L, io):
    """Few packed rows, long: the row is split the way long plain rows are."""
    cu = [0, 1, 9, 9, L // 3, L // 3 + 1, L // 2, L - 1, L]
    p = ref.gated_inputs(1, 2, L, io, h0=True, cu=cu, seed=L)
    check_fwd(p, io)
    check_bwd(p, io, dlast=True)


def test_steps_outside_the_sequences_are_left(cuda_device):
    import selective_state_space_46_b200 as m
    p = ref.gated_inputs(1, 6, 100, "bf16", cu=[7, 30, 30, 64], seed=3)
    d = tensors(p, "bf16")
    out = torch.full((1, 6, 100), 7.0, device="cuda", dtype=torch.bfloat16)
    m.gated_scan_fwd(*args(d), cu_seqlens=d["cu"], out=out)
    grads = [torch.full((1, 6, 100), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    vec = [torch.empty(6, device="cuda") for _ in range(3)]
    m.mssm_gated_scan_bwd(*args(d), d["x"], None, *grads, *vec, None, None, cu_seqlens=d["cu"])
    torch.cuda.synchronize()
    for t in [out] + grads:
        assert (t[..., :7] == 7).all() and (t[..., 64:] == 7).all()
        assert not (t[..., 7:64] == 7).all()


def test_values_outside_and_in_other_sequences_do_not_leak(cuda_device):
    """NaN and infinities behind the last sequence and in another sequence stay there, both ways."""
    import selective_state_space_46_b200 as m
    p = ref.gated_inputs(1, 4, 600, "f32", h0=True, cu=[5, 200, 311, 590], seed=4)
    d = tensors(p, "f32")
    dout = torch.randn(1, 4, 600, device="cuda")
    dl = torch.randn(3, 4, device="cuda")

    def both():
        out, last = m.gated_scan_fwd(*args(d), h0=d["h0"], cu_seqlens=d["cu"])
        g = m.gated_scan_bwd(*args(d), dout=dout, h0=d["h0"], cu_seqlens=d["cu"], dlast_state=dl)
        torch.cuda.synchronize()
        return [out, last, g["dx"], g["dr"], g["di"], g["dz"], g["dh0"]]

    clean = both()
    for v in (float("nan"), float("inf"), -float("inf")):
        for k in ("x", "r", "i", "z"):
            d[k][..., :5] = v
            d[k][..., 590:] = v
        d["x"][..., 200:311] = v
        d["h0"][1] = v
        dl[1] = v
        dout[..., 200:311] = v
        dirty = both()
        for a, b in zip(clean, dirty):
            if a.dim() == 3:
                assert torch.equal(a[..., 5:200], b[..., 5:200]) and torch.equal(a[..., 311:590], b[..., 311:590])
            else:
                assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
        assert not torch.isfinite(dirty[0][..., 200:311]).any()


def test_values_do_not_leak_between_rows(cuda_device):
    import selective_state_space_46_b200 as m
    p = ref.gated_inputs(3, 5, 300, "f32", seed=5)
    d = tensors(p, "f32")
    clean, _ = m.gated_scan_fwd(*args(d))
    d["x"][1, 2, 250] = float("nan")
    dirty, last = m.gated_scan_fwd(*args(d))
    same = torch.ones(3, 5, 300, dtype=torch.bool, device="cuda")
    same[1, 2, 250:] = False
    assert torch.equal(clean[same], dirty[same]) and dirty[~same].isnan().all()
    assert last.isnan().sum() == 1 and last[1, 2].isnan()


EXTREMES = [0.0, -0.0, 20.0, -20.0, 60.0, -60.0, 88.0, -88.0, 200.0, -200.0]


def extreme_inputs(io):
    p = ref.gated_inputs(1, 7, 100, io, bias=False, seed=6)
    p["lam"] = np.array([-30.0, -10.0, -3.0, 0.0, 1.0, 5.0, 40.0])
    p["r"] = np.tile(np.array(EXTREMES), 10)[None, None, :].repeat(7, 1)
    p["i"] = np.repeat(np.array(EXTREMES), 10)[None, None, :].repeat(7, 1)
    return p


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_extreme_gates_and_rates(cuda_device, io):
    """Saturated gates, decays from 1 to 0 and their gradients, which stay finite where a is 1."""
    p = extreme_inputs(io)
    if io == "bf16":
        p["r"], p["i"] = ref.to_bf16(p["r"]), ref.to_bf16(p["i"])
    check_fwd(p, io)
    check_bwd(p, io)


def test_infinite_gates(cuda_device):
    """r = -inf keeps the state, r = inf decays at the full rate, i = +-inf opens and closes the input."""
    import selective_state_space_46_b200 as m
    p = ref.gated_inputs(1, 2, 64, "f32", gate=False, bias=False, h0=True, seed=7)
    p["r"][:] = np.where(np.arange(64) % 2, np.inf, -np.inf)
    p["i"][:] = np.where(np.arange(64) % 4 < 2, np.inf, -np.inf)
    out, _ = run_fwd(p, "f32")
    q = dict(p, r=np.clip(p["r"], -300, 300), i=np.clip(p["i"], -300, 300))
    within(out, ref.forward(q, "f32")["out"], "out")
    d = tensors(p, "f32")
    g = m.gated_scan_bwd(*args(d), dout=torch.ones_like(d["x"]), h0=d["h0"])
    assert all(torch.isfinite(v).all() for v in g.values() if v is not None)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("how", ["offset", "odd_rows", "mixed", "chunks", "transposed_batch", "broadcast"])
def test_strides_and_alignment(cuda_device, io, how):
    """Views of every kind: equally and unequally misaligned rows, slices of one tensor, broadcast inputs."""
    import selective_state_space_46_b200 as m
    B, D, L = 3, 6, 700 if how != "odd_rows" else 701
    p = ref.gated_inputs(B, D, L, io, seed=8)
    d = tensors(p, io)
    names = ("x", "r", "i", "z")
    if how in ("offset", "mixed"):
        for n, k in enumerate(names):
            off = 3 if how == "offset" else n + 1
            big = torch.zeros(B, D, L + 20, device="cuda", dtype=TYPES[io])
            big[..., off:off + L] = d[k]
            d[k] = big[..., off:off + L]
    elif how == "chunks":
        cat = torch.cat([d[k] for k in names], 1)
        d.update(zip(names, cat.chunk(4, 1)))
    elif how == "transposed_batch":
        for k in names:
            d[k] = d[k].transpose(0, 1).contiguous().transpose(0, 1)
        d["lam"] = torch.stack([d["lam"], d["lam"]], 1)[:, 0]
    elif how == "broadcast":
        p["r"][:] = p["r"][:1]
        d["r"] = d["r"][:1].expand(B, D, L)
        p["i"][:] = p["i"][:, :1]
        d["i"] = d["i"][:, :1].expand(B, D, L)
    out, last = m.gated_scan_fwd(*args(d))
    want = ref.forward(p, io)
    within(out, want["out"], "out")
    within(last, want["last_state"], "last_state")
    dout = torch.ones(B, D, L, device="cuda", dtype=TYPES[io])
    g = m.gated_scan_bwd(*args(d), dout=dout)
    for k, w in ref.backward(p, np.ones((B, D, L)), None, io).items():
        within(g[k], w, k)
    # outputs that are slices of one tensor, rows off every boundary
    cat = torch.full((B, 3 * D, L + 3), 5.0, device="cuda", dtype=TYPES[io])
    o1, o2, o3 = (cat[:, k * D:(k + 1) * D, 1:L + 1] for k in range(3))
    vec = [torch.empty(D, device="cuda") for _ in range(3)]
    m.gated_scan_fwd(*args(d), out=o1)
    within(o1, want["out"], "out")  # not bit by bit: the steps are grouped from another boundary
    dz = torch.empty(B, D, L, device="cuda", dtype=TYPES[io])
    m.mssm_gated_scan_bwd(*args(d), dout, None, o1, o2, o3, dz, *vec, None,
                          torch.empty(3, B, D, device="cuda"))
    for a, k in ((o1, "dx"), (o2, "dr"), (o3, "di"), (dz, "dz")):
        within(a, ref.backward(p, np.ones((B, D, L)), None, io)[k], k)
    assert (cat[..., 0] == 5).all() and (cat[..., L + 1:] == 5).all()


PLANS = [(1, 1), (2, 1), (4, 1), (8, 1), (8, 2), (8, 4), (8, 8)]


@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 300, 2049, 7001, 33000])
def test_every_plan(cuda_device, plan, io, L):
    """Every way of sharing a row among warps and CTAs, whatever the automatic choice is."""
    import selective_state_space_46_b200 as m
    try:
        m.mssm_set_option(m.MSSM_OPT_GATED_WARPS, plan[0])
        m.mssm_set_option(m.MSSM_OPT_GATED_SPLIT, plan[1])
        p = ref.gated_inputs(2, 3, L, io, h0=True, seed=L)
        check_fwd(p, io)
        check_bwd(p, io, dlast=True)
        cu = sorted({0, 1, L // 3, L // 2, L - 1, L}) + [L]
        p = ref.gated_inputs(1, 3, L, io, h0=True, gate=False, cu=cu, seed=L + 1)
        check_fwd(p, io)
        check_bwd(p, io, dlast=True)
    finally:
        m.mssm_set_option(m.MSSM_OPT_GATED_WARPS, 0)
        m.mssm_set_option(m.MSSM_OPT_GATED_SPLIT, 0)


def test_many_sequences_in_a_window(cuda_device):
    """More sequences than one look at the offsets takes, several in a thread's window."""
    rng = np.random.default_rng(17)
    cu = np.concatenate([[2], 2 + np.cumsum(rng.integers(0, 4, 900))])
    p = ref.gated_inputs(1, 3, int(cu[-1]) + 5, "f32", h0=True, cu=cu, seed=18)
    check_fwd(p, "f32")
    check_bwd(p, "f32", dlast=True)


def test_pieces_reproduce_the_whole(cuda_device):
    """A sequence processed in two pieces, the state handed on, and its gradient handed back."""
    import selective_state_space_46_b200 as m
    p = ref.gated_inputs(2, 5, 900, "f32", h0=True, seed=10)
    d = tensors(p, "f32")
    dout = torch.randn(2, 5, 900, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    cut = 333
    halves = []
    for lo, hi in ((0, cut), (cut, 900)):
        halves.append({**d, **{k: d[k][..., lo:hi] for k in ("x", "r", "i", "z")}})
    o1, l1 = m.gated_scan_fwd(*args(halves[0]), h0=d["h0"])
    o2, l2 = m.gated_scan_fwd(*args(halves[1]), h0=l1)
    want = ref.forward(p, "f32")
    within(torch.cat([o1, o2], -1), want["out"], "out")
    within(l2, want["last_state"], "last_state")
    g2 = m.gated_scan_bwd(*args(halves[1]), dout=dout[..., cut:], h0=l1)
    g1 = m.gated_scan_bwd(*args(halves[0]), dout=dout[..., :cut], h0=d["h0"], dlast_state=g2["dh0"])
    grads = ref.backward(p, dout.double().cpu().numpy(), None, "f32")
    for k in ("dx", "dr", "di", "dz"):
        within(torch.cat([g1[k], g2[k]], -1), grads[k], k)
    for k in ("dlam", "dr_bias", "di_bias"):
        within(g1[k] + g2[k], grads[k], k)
    within(g1["dh0"], grads["dh0"], "dh0")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bias,gate", [(True, True), (False, False)])
def test_steps_reproduce_the_scan(cuda_device, io, bias, gate):
    import selective_state_space_46_b200 as m
    B, D, L = 3, 37, 20
    p = ref.gated_inputs(B, D, L, io, bias=bias, gate=gate, h0=True, seed=11)
    d = tensors(p, io)
    state = d["h0"].clone()
    outs = []
    for t in range(L):
        step = [None if d[k] is None else (d[k][..., t] if d[k].dim() == 3 else d[k])
                for k in ("x", "r", "i", "lam", "r_bias", "i_bias", "z")]
        outs.append(m.gated_state_update(state, *step, c=p["c"]))
    want = ref.forward(p, io)
    within(torch.stack(outs, -1), want["out"], "out")
    within(state, want["last_state"], "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (5, 1), (3, 2560), (256, 129), (2, 1 << 16), (700, 8), (1, 4097)])
@pytest.mark.parametrize("how", ["dense", "strided", "offset"])
def test_step_shapes_and_strides(cuda_device, io, shape, how):
    import selective_state_space_46_b200 as m
    B, D = shape
    p = ref.gated_inputs(B, D, 1, io, h0=True, seed=B + D)
    d = tensors(p, io)
    v = {k: d[k][..., 0] for k in ("x", "r", "i", "z")}
    state, out = d["h0"].clone(), torch.empty(B, D, device="cuda", dtype=TYPES[io])
    hold = None
    if how == "strided":
        v = {k: t.t().contiguous().t() for k, t in v.items()}
        hold = torch.full((B, 2 * D + 1), 3.0, device="cuda")
        hold[:, 1::2] = state
        state = hold[:, 1::2]
    elif how == "offset":
        for k, t in v.items():
            big = torch.zeros(B, D + 5, device="cuda", dtype=TYPES[io])
            big[:, 3:D + 3] = t
            v[k] = big[:, 3:D + 3]
        hold = torch.full((B, D + 3), 3.0, device="cuda")
        hold[:, 1:D + 1] = state
        state = hold[:, 1:D + 1]
    m.gated_state_update(state, v["x"], v["r"], v["i"], d["lam"], d["r_bias"], d["i_bias"], v["z"], out=out)
    want = ref.forward(p, io)
    within(out[..., None], want["out"], "out")
    within(state, want["last_state"], "state")
    if how == "strided":
        assert (hold[:, 0::2] == 3).all()
    elif how == "offset":
        assert (hold[:, 0] == 3).all() and (hold[:, D + 1:] == 3).all()


def test_step_extremes(cuda_device):
    p = extreme_inputs("f32")
    import selective_state_space_46_b200 as m
    d = tensors(p, "f32")
    flat = [d[k].transpose(1, 2).reshape(100, 7) for k in ("x", "r", "i")]
    state = torch.zeros(100, 7, device="cuda")
    out = m.gated_state_update(state, *flat, d["lam"])
    q = dict(p, z=None, x=p["x"].transpose(2, 1, 0), r=p["r"].transpose(2, 1, 0), i=p["i"].transpose(2, 1, 0))
    within(out[..., None], ref.forward(q, "f32")["out"], "out")


def test_same_inputs_give_the_same_bits(cuda_device):
    import selective_state_space_46_b200 as m
    for shape, cu in (((4, 300, 3000), None), ((1, 60, 30000), [0, 11, 20000, 30000])):
        d = tensors(ref.gated_inputs(*shape, "bf16", h0=True, cu=cu, seed=12), "bf16")
        runs = []
        for _ in range(3):
            o = m.gated_scan_fwd(*args(d), h0=d["h0"], cu_seqlens=d["cu"])
            g = m.gated_scan_bwd(*args(d), dout=d["x"], h0=d["h0"], cu_seqlens=d["cu"])
            runs.append([*o, *[v for v in g.values() if v is not None]])
        for a, b, c in zip(*runs):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_bad_offsets_are_reported(cuda_device):
    """Offsets that decrease or leave the row touch nothing outside the tensors and are reported."""
    import selective_state_space_46_b200 as m
    d = tensors(ref.gated_inputs(1, 4, 50, "f32", seed=13), "f32")
    for cu in ([0, 60], [-3, 20, 50], [0, 30, 20, 50], [10, 5], [70, 80, 90], [50, 40, 30, 20, 10, 0]):
        cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
        n = len(cu) - 1
        guard = torch.full((n + 4, 4), 3.0, device="cuda")
        m.mssm_get_error()
        m.gated_scan_fwd(*args(d), cu_seqlens=cu_t, last_state=guard[2:n + 2])
        with pytest.raises(m.MssmError) as e:
            m.mssm_get_error()
        assert e.value.status == m.MSSM_ERR_INVALID_ARG
        m.gated_scan_bwd(*args(d), dout=d["x"], cu_seqlens=cu_t)
        with pytest.raises(m.MssmError):
            m.mssm_get_error()
        assert (guard[:2] == 3).all() and (guard[n + 2:] == 3).all()
    m.mssm_get_error()


def test_streams_and_graphs(cuda_device):
    """Two streams at once and a captured, replayed graph give what the eager calls give."""
    import selective_state_space_46_b200 as m
    d = tensors(ref.gated_inputs(2, 64, 5000, "bf16", h0=True, seed=14), "bf16")
    e = tensors(ref.gated_inputs(3, 32, 4000, "bf16", h0=True, seed=15), "bf16")

    def work(t, stream=None):
        o, l = m.gated_scan_fwd(*args(t), h0=t["h0"], stream=stream)
        g = m.gated_scan_bwd(*args(t), dout=t["x"], h0=t["h0"], stream=stream)
        return [o, l] + [v for v in g.values() if v is not None]

    want = [work(d), work(e)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [work(d, s[0]), work(e, s[1].cuda_stream)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got1 = work(d)
    with torch.cuda.graph(graph2):
        got2 = work(e)
    for _ in range(2):
        with torch.cuda.stream(s[0]):
            graph.replay()
        with torch.cuda.stream(s[1]):
            graph2.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want[0], got1))
        assert all(torch.equal(x, y) for x, y in zip(want[1], got2))
        for t in got1 + got2:
            t.zero_()


def test_launches_are_counted(cuda_device):
    import selective_state_space_46_b200 as m
    before = {k: v["launches"] for k, v in m.mssm_kernel_stats().items()}
    d = tensors(ref.gated_inputs(2, 8, 100, "f32", seed=16), "f32")
    m.gated_scan_fwd(*args(d))
    m.gated_scan_bwd(*args(d), dout=d["x"])
    after = {k: v["launches"] for k, v in m.mssm_kernel_stats().items()}
    assert after["gated_scan"] == before["gated_scan"] + 1 and after["gated_bwd"] == before["gated_bwd"] + 1


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [False, True])
def test_spikes_among_ordinary_gates(cuda_device, io, packed):
    """Now and then a gate so far from zero that its window is computed with more care, over many tiles."""
    L = 9001
    cu = [0, 700, 701, 4096, 8000, L] if packed else None
    p = ref.gated_inputs(1 if packed else 2, 5, L, io, h0=True, cu=cu, seed=21)
    rng = np.random.default_rng(22)
    for k in ("r", "i", "z"):
        at = rng.random(p[k].shape) < 2e-3
        p[k] = np.where(at, rng.choice([-80.0, -50.0, 50.0, 80.0], p[k].shape), p[k])
    check_fwd(p, io)
    check_bwd(p, io, dlast=True)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_rates_around_the_polynomials_ends(cuda_device, io):
    """Rates just below and above 1/8 and 1/4 with gates that take them whole."""
    p = ref.gated_inputs(2, 9, 3000, io, h0=True, seed=23)
    rates = np.array([1e-4, 0.1, 0.1249, 0.1251, 0.2, 0.2499, 0.2501, 1.0, 30.0])
    p["lam"] = np.float32(np.log(np.expm1(rates / p["c"]))).astype(np.float64)
    p["r"][:, :, ::3] = 12.0
    check_fwd(p, io)
    check_bwd(p, io, dlast=True)


def test_offsets_past_32_bits(cuda_device):
    """Rows and batches more than 2^31 elements apart."""
    import selective_state_space_46_b200 as m
    far = 2 ** 31 + 8
    buf = torch.zeros(far + 4096, device="cuda", dtype=torch.bfloat16)
    p = ref.gated_inputs(1, 2, 600, "bf16", seed=24)
    d = tensors(p, "bf16")
    views = [buf.as_strided((1, 2, 600), (far, far, 1), 640 * n) for n in range(5)]
    for v, k in zip(views, ("x", "r", "i", "z")):
        v.copy_(d[k])
    out, last = m.gated_scan_fwd(*views[:3], d["lam"], d["r_bias"], d["i_bias"], views[3], out=views[4])
    want = m.gated_scan_fwd(*args(d))
    assert out.data_ptr() == views[4].data_ptr() and torch.equal(views[4], want[0]) and torch.equal(last, want[1])
    dout = torch.randn_like(d["x"])
    views[4].copy_(dout)
    g = m.gated_scan_bwd(*views[:3], d["lam"], d["r_bias"], d["i_bias"], views[3], dout=views[4])
    h = m.gated_scan_bwd(*args(d), dout=dout)
    assert all(torch.equal(g[k], h[k]) for k in g if g[k] is not None)
    rows = [buf.as_strided((2, 128), (far, 1), 640 * n) for n in range(4)]
    state = torch.randn(2, 128, device="cuda")
    other = state.clone()
    lam = torch.randn(128, device="cuda")
    o = m.gated_state_update(state, *rows[:3], lam, z=rows[3])
    assert torch.equal(o, m.gated_state_update(other, *[v.contiguous() for v in rows[:3]], lam, z=rows[3].contiguous()))
    assert torch.equal(state, other)


def test_outputs_given_and_left_out(cuda_device):
    """The caller's outputs are the ones returned; inputs that require gradients make no outputs that do."""
    import selective_state_space_46_b200 as m
    d = tensors(ref.gated_inputs(2, 6, 333, "f32", h0=True, seed=25), "f32")
    d["x"].requires_grad_(True)
    out, last = torch.empty(2, 6, 333, device="cuda"), torch.empty(2, 6, device="cuda")
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        got = m.gated_scan_fwd(*args(d), h0=d["h0"], out=out, last_state=last, stream=stream)
        torch.cuda.synchronize()
        assert got[0] is out and got[1] is last
        new, none = m.gated_scan_fwd(*args(d), h0=d["h0"], return_last_state=False, stream=stream)
        torch.cuda.synchronize()
        assert none is None and torch.equal(new, out) and not new.requires_grad
        state = d["h0"].clone()
        step = [d[k][..., 0] for k in ("x", "r", "i")]
        o = torch.empty(2, 6, device="cuda")
        assert m.gated_state_update(state, *step, d["lam"], out=o, stream=stream) is o
        state2 = d["h0"].clone()
        o2 = m.gated_state_update(state2, *step, d["lam"], stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(state, state2) and not o2.requires_grad
    with pytest.raises(m.MssmError):
        m.gated_scan_fwd(*args(d), out=torch.empty(2, 6, 334, device="cuda"))
    with pytest.raises(m.MssmError):
        m.gated_state_update(state, *step, d["lam"][:5])
    with pytest.raises(TypeError):
        m.gated_state_update(state, *step, [1.0] * 6)
    with pytest.raises(ValueError):
        m.gated_scan_fwd(d["x"][0], d["r"], d["i"], d["lam"])


@pytest.mark.parametrize("rows", [1, 2])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 4), (7, 12), (5, 13), (64, 260)])
def test_every_step_plan(cuda_device, rows, io, shape):
    """The decode step with 1 and 2 batch rows a thread, whatever the automatic choice is, and replayed."""
    import selective_state_space_46_b200 as m
    p = ref.gated_inputs(*shape, 1, io, h0=True, seed=rows)
    d = tensors(p, io)
    flat = [d[k][..., 0].contiguous() for k in ("x", "r", "i")] + [d[k] for k in ("lam", "r_bias", "i_bias")]
    z = d["z"][..., 0].contiguous()
    want = ref.forward(p, io)
    try:
        m.mssm_set_option(m.MSSM_OPT_GATED_STEP_ROWS, rows)
        state = d["h0"].clone()
        out = m.gated_state_update(state, *flat, z=z)
        within(out[..., None], want["out"], "out")
        within(state, want["last_state"], "state")
        again = d["h0"].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            replayed = m.gated_state_update(again, *flat, z=z)
        again.copy_(d["h0"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(replayed, out) and torch.equal(again, state)
    finally:
        m.mssm_set_option(m.MSSM_OPT_GATED_STEP_ROWS, 0)
