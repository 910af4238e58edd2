"""The gated linear recurrence and the 4-bit linear map in fp64 numpy, each with a bound on what the fp32
kernels may lose.

The bounds are running error analyses of the kernels' arithmetic, derived from its unit roundings:
u = 2^-24 for an fp32 operation, 2^-22 for an SFU exponential, reciprocal square root or reciprocal, and
half a step of the storage type (2^-8 relative for bf16) at the end.  A gate's argument v is rounded
to u |v|, which its exponential turns into a relative error, hence the terms in |v|.
"""
import numpy as np

U = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "f32": U}
TINY = 1e-35  # results the kernels flush to zero


def sigmoid(v):
    with np.errstate(over="ignore"):
        return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def gate_error(v):
    """Relative error of sigmoid(v).  Below the smallest normal number the kernels flush it to zero."""
    return U * (3 * np.abs(v) + 16) + (sigmoid(v) < 2.0 ** -125)


def terms(p):
    """Everything a step computes from its own inputs, and the relative errors."""
    col = (None, slice(None), None)
    vr = p["r"] + (p["r_bias"][col] if p["r_bias"] is not None else 0.0)
    vi = p["i"] + (p["i_bias"][col] if p["i_bias"] is not None else 0.0)
    lam = p["lam"][col]
    t = dict(r=sigmoid(vr), r1=sigmoid(-vr), i=sigmoid(vi), i1=sigmoid(-vi), eg_r=gate_error(vr), eg_i=gate_error(vi),
             eg_r1=gate_error(-vr), eg_i1=gate_error(-vi), x=p["x"])
    t["y"] = p["c"] * np.logaddexp(0.0, lam) * t["r"]
    t["a"] = np.exp(-t["y"])
    t["beta"] = np.sqrt(-np.expm1(-2 * t["y"]))
    # rate r: three roundings of softplus and two products; the series and the exponential of it
    t["e_y"] = t["eg_r"] + 6 * U
    t["e_a"] = 1.3 * t["y"] * (t["e_y"] + 4 * U) + np.where(t["y"] < 0.25, 2, 8) * U
    t["e_beta"] = 0.5 * t["e_y"] + 20 * U + (t["r"] < 2.0 ** -125)
    t["e_b"] = t["e_beta"] + t["eg_i"] + 3 * U
    t["b"] = t["beta"] * t["i"] * t["x"]
    if p["z"] is not None:
        z = p["z"]
        sz = sigmoid(z)
        t.update(z=z, sz=sz, silu=z * sz, dsilu=sz * (1 + z * sigmoid(-z)), dsilu_abs=sz * (1 + np.abs(z) * sigmoid(-z)),
                 eg_z=gate_error(z))
    return t


def spans(p):
    """(sequence, batch row, first step, end step) of every sequence."""
    if p["cu"] is None:
        return [(b, b, 0, p["x"].shape[2]) for b in range(p["x"].shape[0])]
    return [(s, 0, int(p["cu"][s]), int(p["cu"][s + 1])) for s in range(len(p["cu"]) - 1)]


def states(p, t):
    """h before and after every step with their error bounds, and the last states."""
    shape = p["x"].shape
    h, e, mag = (np.zeros(shape) for _ in range(3))
    before, e_before, mag_before = (np.zeros(shape) for _ in range(3))
    sp = spans(p)
    last, e_last = np.zeros((len(sp), shape[1])), np.zeros((len(sp), shape[1]))
    for s, b, t0, t1 in sp:
        hv = p["h0"][s].copy() if p["h0"] is not None else np.zeros(shape[1])
        ev, mv = np.zeros(shape[1]), np.abs(hv)
        for k in range(t0, t1):
            before[b, :, k], e_before[b, :, k], mag_before[b, :, k] = hv, ev, mv
            a, bb = t["a"][b, :, k], t["b"][b, :, k]
            mn = a * mv + np.abs(bb)
            ev = a * ev + t["e_a"][b, :, k] * a * mv + t["e_b"][b, :, k] * np.abs(bb) + 4 * U * mn
            hv = a * hv + bb
            mv = mn
            h[b, :, k], e[b, :, k], mag[b, :, k] = hv, ev, mv
        last[s], e_last[s] = hv, ev
    return dict(h=h, e=e, mag=mag, before=before, e_before=e_before, mag_before=mag_before, last=last, e_last=e_last)


def stored(ref, err, io):
    return err + HALF_STEP[io] * (np.abs(ref) + err) + TINY


def forward(p, io):
    """{"out": (value, bound), "last_state": (value, bound)}."""
    t = terms(p)
    st = states(p, t)
    out, e = st["h"], st["e"]
    if p["z"] is not None:
        e = e * np.abs(t["silu"]) + (st["mag"] + e) * np.abs(t["silu"]) * (t["eg_z"] + 4 * U)
        out = out * t["silu"]
    return {"out": (out, stored(out, e, io)), "last_state": (st["last"], st["e_last"] + TINY)}


def backward(p, dout, dlast, io):
    """Every gradient with its bound."""
    t = terms(p)
    st = states(p, t)
    shape = p["x"].shape
    g = {}
    q, e_q = dout, np.zeros(shape)
    if p["z"] is not None:
        dz = dout * st["h"] * t["dsilu"]
        e = np.abs(dout) * t["dsilu_abs"] * (st["e"] + st["mag"] * (2 * t["eg_z"] + 8 * U))
        g["dz"] = (dz, stored(dz, e, io))
        q = dout * t["silu"]
        e_q = np.abs(q) * (t["eg_z"] + 5 * U)
    s, e_s, m_s = (np.zeros(shape) for _ in range(3))
    sp = spans(p)
    dh0, e_h0 = np.zeros((len(sp), shape[1])), np.zeros((len(sp), shape[1]))
    for n, b, t0, t1 in sp:
        cv = dlast[n].copy() if dlast is not None else np.zeros(shape[1])
        ev, mv = np.zeros(shape[1]), np.abs(cv)
        for k in range(t1 - 1, t0 - 1, -1):
            sv, mn = q[b, :, k] + cv, np.abs(q[b, :, k]) + mv
            es = e_q[b, :, k] + ev + 4 * U * mn
            s[b, :, k], e_s[b, :, k], m_s[b, :, k] = sv, es, mn
            a = t["a"][b, :, k]
            cv, mv = a * sv, a * mn
            ev = a * es + (t["e_a"][b, :, k] + 4 * U) * mv
        dh0[n], e_h0[n] = cv, ev
    if p["h0"] is not None:
        g["dh0"] = (dh0, e_h0 + TINY)
    x, ax = t["x"], np.abs(t["x"])
    bi = t["beta"] * t["i"]
    dx = s * bi
    g["dx"] = (dx, stored(dx, e_s * bi + m_s * bi * (t["e_beta"] + t["eg_i"] + 6 * U), io))
    di = dx * x * t["i1"]
    e_di = (e_s + m_s * (t["e_beta"] + t["eg_i"] + t["eg_i1"] + 8 * U)) * bi * ax * t["i1"]
    g["di"] = (di, stored(di, e_di, io))
    # w = s a (i x rho - y h_before), rho = a y / beta
    with np.errstate(divide="ignore", invalid="ignore"):
        rho = np.where(t["beta"] > 0, t["a"] * t["y"] / t["beta"], 0.0)
    w = s * t["a"] * (t["i"] * x * rho - t["y"] * st["before"])
    in_abs = t["i"] * ax * rho + t["y"] * st["mag_before"]
    e_rho = t["e_a"] + t["e_y"] + t["e_beta"] + 20 * U
    e_w = t["a"] * (e_s * in_abs + m_s * (t["i"] * ax * rho * (t["eg_i"] + e_rho + 4 * U)
                                          + t["y"] * (t["e_y"] * st["mag_before"] + st["e_before"])
                                          + in_abs * (t["e_a"] + 8 * U)))
    m_w = m_s * t["a"] * in_abs
    dr = t["r1"] * w
    e_dr = t["r1"] * (e_w + m_w * (t["eg_r1"] + 2 * U))
    g["dr"] = (dr, stored(dr, e_dr, io))
    valid = np.zeros(shape[2] if p["cu"] is not None else 1, bool)
    for _, _, t0, t1 in sp:
        if p["cu"] is not None:
            valid[t0:t1] = True
    mask = valid[None, None, :] if p["cu"] is not None else np.ones((1, 1, shape[2]))
    n_add = shape[2] / 16 + 64 + shape[0]

    def total(v, e, m):
        v, e, m = (np.sum(k * mask, axis=(0, 2)) for k in (v, e, m))
        return v, e + n_add * U * m

    lam = p["lam"]
    with np.errstate(under="ignore", invalid="ignore", divide="ignore"):
        spl = np.logaddexp(0.0, lam)
        ratio = np.where(spl > 0, sigmoid(lam) / spl, 1.0)
    v, e = total(w, e_w, m_w)
    g["dlam"] = (v * ratio, ratio * (e + 10 * U * np.abs(v)) + TINY)
    v, e = total(dr, e_dr, t["r1"] * m_w)
    if p["r_bias"] is not None:
        g["dr_bias"] = (v, e + TINY)
    v, e = total(di, e_di, m_s * bi * ax * t["i1"])
    if p["i_bias"] is not None:
        g["di_bias"] = (v, e + TINY)
    return g


# ---------------------------------------------------------------- 4-bit linear map

def w4_dequantise(codes, scales, zeros, k, group):
    col = np.arange(k)
    code = (codes[:, col // 2] >> (4 * (col % 2))) & 15
    zero = 8.0 if zeros is None else zeros.astype(np.float64)[:, col // group]
    return scales.astype(np.float64)[:, col // group] * (code.astype(np.float64) - zero)


def w4_linear(x, codes, scales, zeros, bias, group, io):
    """(value, bound): the products and their sum inside a group are exact to the tensor cores' fp32
    accumulation (one truncation, 2 u, per product added), the groups' sums are scaled and added in fp32."""
    w = w4_dequantise(codes, scales, zeros, x.shape[1], group)
    y = x @ w.T
    mag = np.abs(x) @ np.abs(w).T
    if bias is not None:
        y = y + bias
        mag = mag + np.abs(bias)
    groups = -(-x.shape[1] // 32)
    return y, stored(y, mag * U * (2 * 64 + 8 + groups), io)


# ---------------------------------------------------------------- inputs

def to_bf16(v):
    """fp64 values rounded to the nearest bf16 number (ties to even)."""
    b = np.asarray(v, np.float32).view(np.uint32)
    b = (b + 0x7fff + ((b >> 16) & 1)) & np.uint32(0xffff0000)
    return b.view(np.float32).astype(np.float64)


def gated_inputs(batch, dim, length, io="f32", gate=True, bias=True, h0=False, cu=None, seed=0, lam=None, c=8.0):
    rng = np.random.default_rng(seed)
    store = to_bf16 if io == "bf16" else (lambda v: np.asarray(v, np.float32).astype(np.float64))

    def f32(*shape, std=1.0):
        return np.float32(std * rng.standard_normal(shape)).astype(np.float64)

    if lam is None:  # decays from long memories (1 - a of 1e-3) to short ones (a of 0.05)
        lam = np.float32(np.log(np.expm1(np.exp(rng.uniform(np.log(2e-3), np.log(3.0), dim)) / c))).astype(np.float64)
    shape = (batch, dim, length)
    seqs = batch if cu is None else len(cu) - 1
    return dict(x=store(rng.standard_normal(shape)), r=store(2 * rng.standard_normal(shape)),
                i=store(2 * rng.standard_normal(shape)), z=store(rng.standard_normal(shape)) if gate else None,
                lam=lam, r_bias=f32(dim, std=0.5) if bias else None, i_bias=f32(dim, std=0.5) if bias else None,
                h0=f32(seqs, dim) if h0 else None, cu=None if cu is None else np.asarray(cu, np.int32), c=c)
