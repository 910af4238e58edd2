"""GPU parity of the 4-bit linear map with its fp64 reference (tests/gated_ref.py derives the bounds), and a
recurrent block's decode step made of the operators together."""
import numpy as np
import pytest
import torch

import gated_ref as ref
from test_parity_gated import TYPES, within

pytestmark = pytest.mark.gpu


def weight(n, k, group, scale_io, zeros, seed):
    rng = np.random.default_rng(seed)
    g = -(-k // group)
    codes = rng.integers(0, 256, (n, (k + 1) // 2), dtype=np.uint8)
    scales = rng.uniform(0.5, 1.5, (n, g)) * rng.choice([1.0, -1.0], (n, g)) / np.sqrt(k)
    scales = ref.to_bf16(scales) if scale_io == "bf16" else np.float32(scales).astype(np.float64)
    z = rng.integers(0, 16, (n, g), dtype=np.uint8) if zeros else None
    return codes, scales, z


def packed(w, k, group, scale_io):
    import selective_state_space_46_b200 as m
    codes, scales, z = w
    return m.w4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda().to(TYPES[scale_io]),
                     None if z is None else torch.from_numpy(z).cuda(), in_features=k, group_size=group)


def tokens(m_, k, io, seed):
    x = np.random.default_rng(seed).standard_normal((m_, k))
    return ref.to_bf16(x) if io == "bf16" else np.float32(x).astype(np.float64)


def check(m_, n, k, group, io="bf16", scale_io=None, zeros=False, bias=False, seed=0):
    import selective_state_space_46_b200 as m
    scale_io = scale_io or io
    w = weight(n, k, group, scale_io, zeros, seed)
    x = tokens(m_, k, io, seed + 1)
    b = np.float32(np.random.default_rng(seed + 2).standard_normal(n)).astype(np.float64) if bias else None
    y = m.w4_linear(torch.from_numpy(x).cuda().to(TYPES[io]), packed(w, k, group, scale_io),
                    None if b is None else torch.from_numpy(b).cuda().float())
    within(y, ref.w4_linear(x, *w, b, group, io), "y")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("m_", [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 32, 33, 70])
def test_token_counts(cuda_device, m_, io):
    check(m_, 50, 300, 64, io, zeros=m_ % 2 == 0, bias=m_ % 3 == 0, seed=m_)


@pytest.mark.parametrize("k", [1, 2, 7, 31, 32, 33, 63, 64, 65, 127, 128, 129, 1001, 4100])
@pytest.mark.parametrize("group", [32, 64, 96, 128, 4096])
def test_inputs_and_groups(cuda_device, k, group):
    io = "f32" if k % 2 else "bf16"
    check(3, 33, k, group, io, zeros=k % 3 == 0, seed=k + group)


@pytest.mark.parametrize("n", [1, 2, 8, 15, 16, 17, 193, 2049])
@pytest.mark.parametrize("io,scale_io", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("zeros", [False, True])
def test_outputs_and_types(cuda_device, n, io, scale_io, zeros):
    check(2, n, 520, 128, io, scale_io, zeros, bias=True, seed=n)


@pytest.mark.parametrize("shape", [(1, 5120, 2560), (1, 192, 5120), (4, 10240, 1536), (1, 16, 16384), (2, 20000, 64),
                                   (16, 2560, 5120), (256, 512, 1536)])
def test_model_sizes(cuda_device, shape):
    check(*shape, 128, zeros=True, seed=sum(shape))


def test_strides(cuda_device):
    """Rows of x off the 16-byte boundaries, an output that is a transposed slice, codes and scales as views."""
    import selective_state_space_46_b200 as m
    n, k, group = 40, 200, 32
    codes, scales, z = weight(n, k, group, "f32", True, 3)
    wide = torch.zeros(n, 2 * codes.shape[1], dtype=torch.uint8, device="cuda")
    wide[:, ::2] = torch.from_numpy(codes).cuda()
    st = torch.from_numpy(scales).cuda().float().t().contiguous().t()
    zt = torch.from_numpy(z).cuda().t().contiguous().t()
    w = m.w4_pack(wide[:, ::2], st, zt, in_features=k, group_size=group)
    for io in ("bf16", "f32"):
        x = tokens(5, k, io, 4)
        big = torch.full((5, k + 9), float("nan"), device="cuda", dtype=TYPES[io])
        big[:, 3:k + 3] = torch.from_numpy(x).cuda().to(TYPES[io])
        hold = torch.full((n + 2, 5), 9.0, device="cuda", dtype=TYPES[io])
        y = m.w4_linear(big[:, 3:k + 3], w, out=hold[1:n + 1].t())
        within(y, ref.w4_linear(x, codes, scales, z, None, group, io), "y")
        assert (hold[0] == 9).all() and (hold[n + 1] == 9).all()


def test_nan_and_infinite_tokens_stay_in_their_rows(cuda_device):
    import selective_state_space_46_b200 as m
    for io in ("bf16", "f32"):
        w = weight(40, 130, 32, io, False, 5)
        wp = packed(w, 130, 32, io)
        x = torch.from_numpy(tokens(11, 130, io, 6)).cuda().to(TYPES[io])
        clean = m.w4_linear(x, wp)
        for v in (float("nan"), float("inf"), torch.finfo(TYPES[io]).max):
            bad = x.clone()
            bad[4, 77] = v
            y = m.w4_linear(bad, wp)
            keep = torch.arange(11, device="cuda") != 4
            assert torch.equal(y[keep], clean[keep])
            col = ref.w4_dequantise(*w, 130, 32)[:, 77]
            if v == float("inf"):  # the sign of the infinity is the weight's
                want = torch.from_numpy(np.where(col > 0, np.inf, np.where(col < 0, -np.inf, np.nan))).cuda()
                assert torch.equal(y[4].double().nan_to_num(7.0, 1.0, -1.0), want.nan_to_num(7.0, 1.0, -1.0))
            elif v != v:
                assert y[4].isnan().all()


def test_wide_range_of_fp32_tokens(cuda_device):
    """Tokens of very different sizes: fp32 keeps all of its 24 bits."""
    import selective_state_space_46_b200 as m
    w = weight(20, 256, 32, "f32", True, 7)
    x = tokens(4, 256, "f32", 8) * np.exp2(np.random.default_rng(9).integers(-60, 60, (4, 256)))
    y = m.w4_linear(torch.from_numpy(x).cuda().float(), packed(w, 256, 32, "f32"))
    within(y, ref.w4_linear(x, *w, None, 32, "f32"), "y")


def test_same_inputs_give_the_same_bits_and_replay(cuda_device):
    import selective_state_space_46_b200 as m
    w = weight(300, 3000, 128, "bf16", True, 10)
    wp = packed(w, 3000, 128, "bf16")
    x = torch.from_numpy(tokens(5, 3000, "bf16", 11)).cuda().bfloat16()
    y = m.w4_linear(x, wp)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(3):
        z = m.w4_linear(x, wp, stream=s if k % 2 else s.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(y, z)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z = m.w4_linear(x, wp)
    for _ in range(2):
        z.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, z)


def test_no_tokens(cuda_device):
    import selective_state_space_46_b200 as m
    w = packed(weight(20, 64, 32, "bf16", False, 12), 64, 32, "bf16")
    assert m.w4_linear(torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), w).shape == (0, 20)
    with pytest.raises(ValueError):
        m.w4_linear(torch.empty(1, 65, device="cuda", dtype=torch.bfloat16), w)
    with pytest.raises(ValueError):
        m.w4_linear(torch.empty(1, 64, device="cuda", dtype=torch.bfloat16), w, out=torch.empty(1, 21, device="cuda"))


def test_recurrent_block_decodes_as_it_prefills(cuda_device):
    """Projections with 4-bit weights, the causal conv, the gated recurrence and the output projection: a prompt
    in one call each, then token by token from the states it left, against the fp64 composition."""
    import selective_state_space_46_b200 as m
    B, E, D, L, extra, group = 2, 96, 80, 21, 5, 32
    io = "f32"
    rng = np.random.default_rng(13)
    w_in, w_out = weight(4 * D, E, group, io, True, 14), weight(E, D, group, io, False, 15)
    p_in, p_out = packed(w_in, E, group, io), packed(w_out, D, group, io)
    conv_w, conv_b = np.float32(rng.standard_normal((D, 4)) / 2), np.float32(rng.standard_normal(D) / 4)
    vecs = {k: np.float32(rng.standard_normal(D)).astype(np.float64) for k in ("lam", "r_bias", "i_bias")}
    tok = np.float32(rng.standard_normal((B, L + extra, E))).astype(np.float64)
    # fp64: every projection, conv and recurrence in turn
    wi, wo = ref.w4_dequantise(*w_in, E, group), ref.w4_dequantise(*w_out, D, group)
    branches = np.split((tok @ wi.T).transpose(0, 2, 1), 4, axis=1)  # x, r, i, z: [B, D, L + extra]
    padded = np.concatenate([np.zeros((B, D, 3)), branches[0]], -1)
    conv = sum(conv_w[:, k, None].astype(np.float64) * padded[..., k:k + L + extra] for k in range(4))
    conv = conv + conv_b[:, None]
    conv = conv * ref.sigmoid(conv)
    prob = dict(x=conv, r=branches[1], i=branches[2], z=branches[3], h0=None, cu=None, c=8.0, **vecs)
    y = ref.forward(prob, io)["out"][0].transpose(0, 2, 1) @ wo.T

    def to(v):
        return torch.from_numpy(np.asarray(v)).cuda().float()

    cw, cb, lam, rb, ib = to(conv_w), to(conv_b), to(vecs["lam"]), to(vecs["r_bias"]), to(vecs["i_bias"])
    t = to(tok)
    h = m.w4_linear(t[:, :L].reshape(-1, E), p_in).reshape(B, L, 4, D).permute(2, 0, 3, 1).contiguous()
    x, r, i, z = h
    u = m.causal_conv1d(x, cw, cb)
    out, state = m.gated_scan_fwd(u, r, i, lam, rb, ib, z)
    got = [m.w4_linear(out.transpose(1, 2).reshape(-1, D), p_out).reshape(B, L, E)]
    window = x[..., -3:].contiguous()
    for k in range(L, L + extra):
        x, r, i, z = m.w4_linear(t[:, k].contiguous(), p_in).reshape(B, 4, D).unbind(1)
        u = m.causal_conv1d_update(window, x, cw, cb)
        o = m.gated_state_update(state, u, r, i, lam, rb, ib, z)
        got.append(m.w4_linear(o, p_out)[:, None])
    got = torch.cat(got, 1).double().cpu().numpy()
    # four stages of at most some hundred fp32 roundings each, on values of order one: 4 * 256 * 2^-24 of the scale
    assert np.abs(got - y).max() <= 4 * 256 * 2.0 ** -24 * (1 + np.abs(y).max())


@pytest.mark.parametrize("plan", [2, 8, 16])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 16, 64, 32), (5, 33, 1000, 96), (13, 100, 4096, 128), (40, 48, 2100, 64)])
def test_every_plan(cuda_device, plan, io, shape):
    """One or two tiles and 8 or 16 warps a CTA, whatever the automatic choice is: fewer blocks than warps, odd tiles."""
    import selective_state_space_46_b200 as m
    m_, n, k, group = shape
    try:
        m.mssm_set_option(m.MSSM_OPT_W4_PLAN, plan)
        for zeros in (False, True):
            check(m_, n, k, group, io, zeros=zeros, bias=zeros, seed=plan)
            check(m_, n, k - 1, group, io, scale_io="f32", zeros=zeros, seed=plan + 1)
    finally:
        m.mssm_set_option(m.MSSM_OPT_W4_PLAN, 0)


def test_scales_of_a_group_wider_than_the_input(cuda_device):
    check(3, 20, 100, 224, zeros=True, seed=31)
    check(3, 20, 100, 2 ** 20, "f32", seed=32)
