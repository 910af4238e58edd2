"""The gated linear recurrence (scan, backward, decode step) and the linear map with 4-bit weights:
cases at real sizes, their plain forms, and the calls a program makes of this library.

``run`` computes an operator in elementary torch operations in 32 bits, or, when ``own`` is true,
through ``selective_state_space_46_b200``; ``exact`` computes it in 64 bits from the definition.

    r = sigmoid(r_raw + r_bias), i = sigmoid(i_raw + i_bias), a = exp(-c softplus(lam) r)
    h_t = a_t h_(t-1) + sqrt(1 - a_t^2) i_t x_t,  out_t = h_t silu(z_t)        (z optional)
    y[m, n] = sum_k x[m, k] scale[n, k / g] (code[n, k] - zero[n, k / g]) + bias[n]
"""
import math

import torch

own = False

C = 8.0  # the recurrence's decay scale

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def _scan(name, op, dtype, batch, dim, length, gate, state, sequences=0):
    """A scan or backward case; sequences > 0: that many packed sequences of `length` steps in all."""
    return dict(name=name, op=op, dtype=dtype, batch=batch, dim=dim, length=length, gate=gate, state=state,
                sequences=sequences)


def _step(name, dtype, batch, dim, gate):
    return dict(name=name, op="step", dtype=dtype, batch=batch, dim=dim, gate=gate)


def _w4(name, dtype, tokens, k, n, group, zeros, bias):
    return dict(name=name, op="w4", dtype=dtype, tokens=tokens, k=k, n=n, group=group, zeros=zeros, bias=bias)


def listed():
    return [
        # an ordinary prefill: two prompts of a small model, gated output
        _scan("scan_prefill_bf16_2x1536x2048", "scan", "bf16", 2, 1536, 2048, True, False),
        # one very long context: few rows, the length has to be split
        _scan("scan_long_bf16_1x2048x131072", "scan", "bf16", 1, 2048, 131072, True, False),
        # continuous batching: 32 prompts packed without padding, each resumed from its own state
        _scan("scan_packed_bf16_1536x27048", "scan", "bf16", 1, 1536, 27048, False, True, 32),
        # odd sizes in fp32, resumed from a state (rows that start on no 16-byte boundary)
        _scan("scan_odd_f32_3x257x1001", "scan", "f32", 3, 257, 1001, False, True),
        # a training step's backward of an ordinary batch
        _scan("bwd_train_bf16_2x1536x2048", "bwd", "bf16", 2, 1536, 2048, True, False),
        # a training step's backward of a large model's batch
        _scan("bwd_large_bf16_8x5120x4096", "bwd", "bf16", 8, 5120, 4096, True, False),
        # packed training sequences in fp32, states and their gradients carried across pieces
        _scan("bwd_packed_f32_513x10007", "bwd", "f32", 1, 513, 10007, False, True, 13),
        # decoding, one token for each of 256 sequences
        _step("step_bf16_256x5120", "bf16", 256, 5120, True),
        # decoding one sequence: latency
        _step("step_f32_1x1536", "f32", 1, 1536, False),
        # one token through a large model's input projection
        _w4("w4_bf16_1x5120x20480", "bf16", 1, 5120, 20480, 128, False, False),
        # a small batch through an output projection, with zero points and a bias
        _w4("w4_bf16_16x5120x2560", "bf16", 16, 5120, 2560, 64, True, True),
        # odd sizes, fp32 activations and scales, the last group short
        _w4("w4_f32_3x1001x193", "f32", 3, 1001, 193, 32, True, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "bwd", "bwd", "step", "w4", "w4"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("scan", "bwd"):
        packed = rng.random() < 0.35
        batch = 1 if packed else _log_int(rng, 1, 8)
        dim = _log_int(rng, 1, 5120)
        # at most the elements of the long prefill (fp32: half), a quarter of that for the backward pass
        most = 2 ** 28 // (2 if dtype == "f32" else 1) // (4 if op == "bwd" else 1)
        length = _log_int(rng, 1, max(1, min(131072, most // (batch * dim))))
        return dict(op=op, dtype=dtype, batch=batch, dim=dim, length=length, gate=rng.random() < 0.5,
                    state=rng.random() < 0.5, sequences=_log_int(rng, 1, 64) if packed else 0)
    if op == "step":
        return dict(op=op, dtype=dtype, batch=_log_int(rng, 1, 512), dim=_log_int(rng, 1, 8192),
                    gate=rng.random() < 0.5)
    return dict(op=op, dtype=dtype, tokens=_log_int(rng, 1, 32), k=_log_int(rng, 32, 16384),
                n=_log_int(rng, 1, 20480), group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5,
                bias=rng.random() < 0.5)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "w4":
        m, k, n = case["tokens"], case["k"], case["n"]
        groups = -(-k // case["group"])
        nbytes = n * k / 2 + n * groups * (es + (0.5 if case["zeros"] else 0)) + m * (k + n) * es
        nbytes += 4 * n if case["bias"] else 0
        return {"bytes": nbytes, "flops": 2.0 * m * n * k}
    z = int(case["gate"])
    if case["op"] == "step":
        e = case["batch"] * case["dim"]
        return {"bytes": e * (8 + es * (4 + z)) + 12 * case["dim"], "flops": e * (20.0 + 5 * z)}
    e = case["batch"] * case["dim"] * case["length"]
    states = (case["sequences"] or case["batch"]) * case["dim"]
    s = int(case["state"])
    if case["op"] == "scan":
        # x, r, i, (z) -> out; h0 -> last_state; lam and the biases
        return {"bytes": e * es * (4 + z) + 4 * states * (1 + s) + 12 * case["dim"], "flops": e * (20.0 + 5 * z)}
    # x, r, i, dout, (z) -> dx, dr, di, (dz); h0, dlast_state -> dh0; lam and the biases and their gradients
    return {"bytes": e * es * (7 + 2 * z) + 12 * states * s + 24 * case["dim"], "flops": e * (50.0 + 15 * z)}


# ---------------------------------------------------------------- inputs

def _offsets(total, sequences, gen):
    """Offsets of packed sequences: ragged lengths, now and then an empty one."""
    cuts = torch.randint(0, total + 1, (sequences - 1,), generator=gen)
    return torch.tensor([0] + sorted(cuts.tolist()) + [total], dtype=torch.int32)


def _inputs(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=dtype) * std)

    if case["op"] == "w4":
        m, k, n, group = case["tokens"], case["k"], case["n"], case["group"]
        groups = -(-k // group)
        codes = torch.randint(0, 256, (n, (k + 1) // 2), generator=g, device=dev, dtype=torch.uint8)
        # group scales about those of a weight of standard deviation 1 / sqrt(k)
        scales = (torch.rand(n, groups, generator=g, device=dev) + 0.5) / (4.6 * math.sqrt(k))
        zeros = None
        if case["zeros"]:
            zeros = torch.randint(4, 13, (n, groups), generator=g, device=dev, dtype=torch.uint8)
        return dict(x=normal(m, k), codes=codes, scales=scales.to(dt), zeros=zeros,
                    bias=normal(n, dtype=torch.float32, std=0.1) if case["bias"] else None)
    dim = case["dim"]
    # decay rates: exp(-c softplus(lam)) uniform in [0.9, 0.999], a memory of tens to thousands of steps
    u = torch.rand(dim, generator=g, device=dev, dtype=torch.float64) * 0.099 + 0.9
    lam = torch.log(torch.expm1(-torch.log(u) / C)).float()
    d = dict(lam=lam, r_bias=normal(dim, dtype=torch.float32, std=0.5), i_bias=normal(dim, dtype=torch.float32, std=0.5))
    shape = (case["batch"], dim) if case["op"] == "step" else (case["batch"], dim, case["length"])
    for name in ("x", "r", "i"):
        d[name] = normal(*shape)
    d["z"] = normal(*shape) if case["gate"] else None
    if case["op"] == "step":
        d["state"] = normal(*shape, dtype=torch.float32)
        return d
    seqs = case["sequences"]
    d["cu"] = None
    if seqs:
        d["cu"] = _offsets(case["length"], seqs, torch.Generator().manual_seed(seed)).to(dev)
    states = (seqs or case["batch"], dim)
    d["h0"] = normal(*states, dtype=torch.float32) if case["state"] else None
    if case["op"] == "bwd":
        d["dout"] = normal(*shape)
        d["dlast"] = normal(*states, dtype=torch.float32) if case["state"] else None
    return d


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if case["op"] == "w4" and own:
        import selective_state_space_46_b200 as mssm
        # the weight as a program keeps it: laid out once when the model is loaded
        state["weight"] = mssm.w4_pack(state["codes"], state["scales"], state["zeros"], in_features=case["k"],
                                       group_size=case["group"])
    return state


# ---------------------------------------------------------------- the library's operators

def _run_own(s):
    import selective_state_space_46_b200 as mssm
    op = s["case"]["op"]
    if op == "w4":
        return mssm.w4_linear(s["x"], s["weight"], s["bias"])
    args = (s["x"], s["r"], s["i"], s["lam"], s["r_bias"], s["i_bias"], s["z"])
    if op == "step":
        out = mssm.gated_state_update(s["state"], *args, c=C)
        return {"out": out, "state": s["state"]}
    if op == "scan":
        out, last = mssm.gated_scan_fwd(*args, c=C, h0=s["h0"], cu_seqlens=s["cu"])
        return {"out": out, "last_state": last}
    return mssm.gated_scan_bwd(*args, dout=s["dout"], c=C, h0=s["h0"], cu_seqlens=s["cu"], dlast_state=s["dlast"])


# ---------------------------------------------------------------- plain forms

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _gates(s):
    """r, i, log a, a, beta and x in 32 bits; the channel axis is axis 1."""
    tail = (1,) * (s["x"].dim() - 2)
    per = {k: s[k].view(1, -1, *tail) for k in ("lam", "r_bias", "i_bias")}
    r = _sigmoid(s["r"].float() + per["r_bias"])
    i = _sigmoid(s["i"].float() + per["i_bias"])
    rate = C * (torch.clamp(per["lam"], min=0) + torch.log1p(torch.exp(-per["lam"].abs())))
    la = -rate * r
    return r, i, la, torch.exp(la), torch.sqrt(-torch.expm1(2 * la)), s["x"].float()


def _doubling(a, b):
    """h_t = a_t h_(t-1) + b_t from h = 0 along the last axis, by doubling strides."""
    n, k = a.shape[-1], 1
    while k < n:
        b = torch.cat([b[..., :k], b[..., k:] + a[..., k:] * b[..., :-k]], -1)
        if 2 * k < n:
            a = torch.cat([a[..., :k], a[..., k:] * a[..., :-k]], -1)
        k *= 2
    return b


def _bounds(s):
    """First steps, last steps and sequence numbers of the non-empty packed sequences."""
    cu = s["cu"].long()
    keep = (cu[1:] > cu[:-1]).nonzero().flatten()
    return cu[:-1][keep], cu[1:][keep] - 1, keep


def _states(s, a, b):
    """The states of every step, and a with its sequence starts cut."""
    b, cut = b.clone(), a.clone()
    if s["cu"] is None:
        if s["h0"] is not None:
            b[..., 0] += a[..., 0] * s["h0"]
        cut[..., 0] = 0
    else:
        first, _, seq = _bounds(s)
        if s["h0"] is not None:
            b[0][:, first] += a[0][:, first] * s["h0"][seq].T
        cut[..., first] = 0
    return _doubling(cut, b), cut


def _plain_scan(s):
    _, i, _, a, beta, x = _gates(s)
    h, _ = _states(s, a, beta * i * x)
    if s["cu"] is None:
        last = h[..., -1].contiguous()
    else:
        _, end, seq = _bounds(s)
        n = s["cu"].numel() - 1
        last = torch.zeros(n, x.shape[1], device=x.device) if s["h0"] is None else s["h0"].clone()
        last[seq] = h[0][:, end].T
    if s["z"] is not None:
        z = s["z"].float()
        h = h * z * _sigmoid(z)
    return {"out": h.to(s["x"].dtype), "last_state": last}


def _plain_bwd(s):
    r, i, la, a, beta, x = _gates(s)
    h, cut = _states(s, a, beta * i * x)
    q = s["dout"].float()
    g = {}
    dt = s["x"].dtype
    if s["z"] is not None:
        z = s["z"].float()
        sz = _sigmoid(z)
        g["dz"] = (q * h * sz * (1 + z * (1 - sz))).to(dt)
        q = q * z * sz
    if s["cu"] is None:
        first, end = [0], [x.shape[2] - 1]
        if s["dlast"] is not None:
            q = q.clone()
            q[..., -1] += s["dlast"]
    else:
        first, end, seq = _bounds(s)
        if s["dlast"] is not None:
            q = q.clone()
            q[0][:, end] += s["dlast"][seq].T
    # the adjoint runs backwards with the next step's decay, cut at the sequences' ends
    nxt = torch.cat([cut[..., 1:], torch.zeros_like(cut[..., :1])], -1)
    adj = _doubling(nxt.flip(-1), q.flip(-1)).flip(-1)
    before = torch.cat([torch.zeros_like(h[..., :1]), h[..., :-1]], -1)
    if s["cu"] is None:
        if s["h0"] is not None:
            before[..., 0] = s["h0"]
            g["dh0"] = a[..., 0] * adj[..., 0]
    else:
        before[..., first] = 0
        if s["h0"] is not None:
            before[0][:, first] = s["h0"][seq].T
            g["dh0"] = s["dlast"].clone()
            g["dh0"][seq] = (a[0][:, first] * adj[0][:, first]).T
    ratio = torch.where(beta > 0, -la / beta, torch.zeros_like(la))
    w = adj * (la * a * before + a * a * i * x * ratio)
    dr = (1 - r) * w
    di = adj * beta * x * i * (1 - i)
    lam = s["lam"]
    sp = torch.clamp(lam, min=0) + torch.log1p(torch.exp(-lam.abs()))

    def total(v):
        return v.sum((0, 2), dtype=torch.float64)

    g.update(dx=(adj * beta * i).to(dt), dr=dr.to(dt), di=di.to(dt), dlam=(total(w) * (_sigmoid(lam) / sp)).float(),
             dr_bias=total(dr).float(), di_bias=total(di).float())
    return _ordered(g)


def _ordered(g):
    return {k: g[k] for k in ("dx", "dr", "di", "dz", "dlam", "dr_bias", "di_bias", "dh0") if g.get(k) is not None}


def _plain_step(s):
    _, i, _, a, beta, x = _gates(s)
    h = s["state"]
    h.copy_(a * h + beta * i * x)
    out = h
    if s["z"] is not None:
        z = s["z"].float()
        out = h * z * _sigmoid(z)
    return {"out": out.to(s["x"].dtype), "state": h}


def _plain_w4(s):
    case = s["case"]
    k, group = case["k"], case["group"]
    codes = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).flatten(1)[:, :k].float()
    scale = s["scales"].float().repeat_interleave(group, 1)[:, :k]
    zero = 8.0 if s["zeros"] is None else s["zeros"].float().repeat_interleave(group, 1)[:, :k]
    y = s["x"].float() @ ((codes - zero) * scale).T
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["x"].dtype)


def run(state):
    op = state["case"]["op"]
    if own:
        out = _run_own(state)
        return _ordered(out) if op == "bwd" else out
    return {"scan": _plain_scan, "bwd": _plain_bwd, "step": _plain_step, "w4": _plain_w4}[op](state)


# ---------------------------------------------------------------- 64 bits, from the definition

def _exact_terms(d):
    """a_t, the input gain, the gates and x in 64 bits, steps first: [L, rows of (batch, channel)]."""
    def flat(v):
        v = v.double()
        return v.permute(2, 0, 1).reshape(v.shape[2], -1) if v.dim() == 3 else v.reshape(1, -1)

    reps = d["x"].shape[0]
    lam = d["lam"].double().repeat(reps)
    r = torch.sigmoid(flat(d["r"]) + d["r_bias"].double().repeat(reps))
    i = torch.sigmoid(flat(d["i"]) + d["i_bias"].double().repeat(reps))
    # softplus as a logarithm of a sum of exponentials
    rate = C * torch.logaddexp(lam, torch.zeros_like(lam))
    return r, i, rate, lam, flat(d["x"]), flat


def _exact_w4(case, d):
    k, group = case["k"], case["group"]
    col = torch.arange(k, device="cuda")
    byte = d["codes"].long()[:, col // 2]
    code = torch.where(col % 2 == 0, byte % 16, byte // 16).double()
    zero = 8.0 if d["zeros"] is None else d["zeros"].double()[:, col // group]
    w = d["scales"].double()[:, col // group] * (code - zero)
    y = torch.einsum("mk,nk->mn", d["x"].double(), w)
    return y if d["bias"] is None else y + d["bias"].double()


def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "w4":
        return _exact_w4(case, d)
    r, i, rate, lam, x, flat = _exact_terms(d)
    steps, rows = x.shape
    batch, dim = d["x"].shape[:2]
    a = torch.exp(-rate * r)
    gain = torch.sqrt(-torch.expm1(-2 * rate * r))
    inp = gain * i * x
    if case["op"] == "step":
        h = a * d["state"].double().reshape(1, -1) + inp
        out = h if d["z"] is None else h * torch.nn.functional.silu(flat(d["z"]))
        return {"out": out.reshape(batch, dim), "state": h.reshape(batch, dim)}

    def unflat(v):
        return v.reshape(steps, batch, dim).permute(1, 2, 0)

    cu = None if d["cu"] is None else d["cu"].tolist()
    starts = {0: None} if cu is None else {cu[q]: q for q in range(len(cu) - 1) if cu[q + 1] > cu[q]}
    ends = {steps - 1: None} if cu is None else {cu[q + 1] - 1: q for q in range(len(cu) - 1) if cu[q + 1] > cu[q]}
    zero = torch.zeros(rows, device="cuda", dtype=torch.float64)

    def given(v, q):
        return zero if v is None else v.double().reshape(-1) if q is None else v[q].double()

    # the recurrence, step by step
    hs = torch.empty_like(x)
    before = torch.empty_like(x) if case["op"] == "bwd" else None
    h = zero
    for t in range(steps):
        if t in starts:
            h = given(d["h0"], starts[t])
        if before is not None:
            before[t] = h
        h = torch.addcmul(inp[t], a[t], h, out=hs[t])
    if case["op"] == "scan":
        last = hs[-1].reshape(batch, dim) if cu is None else torch.stack(
            [hs[cu[q + 1] - 1] if cu[q + 1] > cu[q] else given(d["h0"], q) for q in range(len(cu) - 1)])
        out = unflat(hs)
        return {"out": out if d["z"] is None else out * torch.nn.functional.silu(d["z"].double()),
                "last_state": last}
    del inp
    q = flat(d["dout"])
    g = {}
    if d["z"] is not None:
        z = flat(d["z"])
        sz = torch.sigmoid(z)
        g["dz"] = unflat(q * hs * (sz + z * sz * (1 - sz)))
        q = q * z * sz
        del z, sz
    del hs
    # the adjoint, step by step from the end
    adj = torch.empty_like(x)
    carry = zero
    dh0 = None if d["h0"] is None else d["dlast"].double().clone()
    for t in range(steps - 1, -1, -1):
        if t in ends:
            carry = given(d["dlast"], ends[t])
        torch.add(q[t], carry, out=adj[t])
        carry = a[t] * adj[t]
        if t in starts and dh0 is not None:
            if cu is None:
                dh0 = carry.reshape(batch, dim)
            else:
                dh0[starts[t]] = carry
    del q
    g["dx"] = unflat(adj * gain * i)
    di = adj * gain * x * i * (1 - i)
    g["di"] = unflat(di)
    g["di_bias"] = di.reshape(steps, batch, dim).sum((0, 1))
    del di
    # d h_t / d log a_t = a h_(t-1) + i x d gain / d log a, and log a = -rate r
    slope = -torch.exp(-2 * rate * r) / gain
    dla = adj * (a * before + i * x * torch.where(gain > 0, slope, torch.zeros_like(slope)))
    del slope, before, adj
    g["dlam"] = (dla * -r * C * torch.sigmoid(lam)).reshape(steps, batch, dim).sum((0, 1))
    dr = dla * -rate * r * (1 - r)
    g["dr"] = unflat(dr)
    g["dr_bias"] = dr.reshape(steps, batch, dim).sum((0, 1))
    g["dh0"] = dh0
    return _ordered(g)
