"""Cases of the gated delta rule and of the root-mean-square norm, with the operators' plain forms.

A case is a dict of plain values; ``prepare`` makes its inputs from a seed, ``run`` does one pass (in
elementary torch operations, or through the framework's entry points where ``own`` is true), ``exact``
gives the same outputs in 64 bits from the definition, and ``work`` counts bytes and operations.
"""
import math

import torch

own = False

D = 128   # key and value width of a head
C = 64    # tokens of a chunk in the plain form
QMAX = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # a short prompt in front of a served model: latency counts
        dict(name="gdn_prefill_short", op="gdn_prefill", dtype="bf16", total=77, seqs=1, hk=16, hv=32, start=False),
        # one prompt of 8k tokens, 32 heads
        dict(name="gdn_prefill_8k", op="gdn_prefill", dtype="bf16", total=8192, seqs=1, hk=32, hv=32, start=False),
        # a packed batch of prompts of different lengths (one empty), each continuing a cached prefix
        dict(name="gdn_prefill_varlen", op="gdn_prefill", dtype="bf16", total=24571, seqs=8, hk=16, hv=32, start=True),
        # the gradient over a few short, packed sequences
        dict(name="gdn_backward_short", op="gdn_backward", dtype="bf16", total=333, seqs=3, hk=4, hv=8, start=True),
        # the gradient of one training sequence of 8k tokens, 32 heads
        dict(name="gdn_backward_8k", op="gdn_backward", dtype="bf16", total=8192, seqs=1, hk=16, hv=32, start=False),
        # a single user's next token
        dict(name="gdn_decode_1", op="gdn_decode", dtype="bf16", total=1, slots=1, hk=16, hv=32),
        # a full serving batch, its states scattered over a larger pool
        dict(name="gdn_decode_256", op="gdn_decode", dtype="bf16", total=256, slots=300, hk=32, hv=32),
        # the norm of one decoded token, with the residual stream's addition
        dict(name="norm_token", op="norm", dtype="bf16", rows=1, dim=4096, residual=True, quant="", group=0),
        # the norm before a layer's projections over an 8k prompt, into 8-bit floats with a scale for 128 columns
        dict(name="norm_8k_e4m3", op="norm", dtype="bf16", rows=8192, dim=4096, residual=True, quant="e4m3", group=128),
        # an odd width and row count without a residual, into 8-bit floats with a scale for each token
        dict(name="norm_odd_e4m3", op="norm", dtype="bf16", rows=1003, dim=2310, residual=False, quant="e4m3", group=0),
        # the norm's gradient over an 8k sequence, the residual stream's own gradient added
        dict(name="norm_backward_8k", op="norm_backward", dtype="bf16", rows=8192, dim=4096, residual=True),
        # the norm's gradient in fp32 at an odd width
        dict(name="norm_backward_odd", op="norm_backward", dtype="f32", rows=777, dim=1001, residual=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gdn_prefill", "gdn_prefill", "gdn_backward", "gdn_decode", "norm", "norm_backward"])
    if op in ("gdn_prefill", "gdn_backward"):
        hk = rng.choice([1, 2, 4, 8, 16])
        hv = hk * rng.choice([1, 2, 4])
        dtype = "f32" if op == "gdn_prefill" and rng.random() < 0.2 else "bf16"
        most = 24571 * 32 if op == "gdn_prefill" and dtype == "bf16" else 4096 * 32
        return dict(op=op, dtype=dtype, total=_log_int(rng, 1, min(16384 if op == "gdn_prefill" else 8192, most // hv)),
                    seqs=_log_int(rng, 1, 12), hk=hk, hv=hv, start=rng.random() < 0.5)
    if op == "gdn_decode":
        hk = rng.choice([2, 4, 8, 16, 32])
        hv = hk * rng.choice([1, 2, 4]) if hk <= 8 else 32
        n = _log_int(rng, 1, 256 * 32 // hv if hv > 32 else 256)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), total=n, slots=n + rng.randrange(0, 40), hk=hk, hv=hv)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    rows, dim = _log_int(rng, 1, 8192), _log_int(rng, 64, 8192)
    if rows * dim > 4096 * 4096:
        rows = max(1, 4096 * 4096 // dim)
    if op == "norm_backward":
        return dict(op=op, dtype=dtype, rows=rows, dim=dim, residual=rng.random() < 0.5)
    quant = rng.choice(["", "e4m3", "int8"])
    group = rng.choice([0, 128]) if quant else 0
    return dict(op=op, dtype=dtype, rows=rows, dim=max(128, dim // 128 * 128) if group else dim,
                residual=rng.random() < 0.5, quant=quant, group=group)


def _lengths(case):
    """Packed lengths of a case: one sequence, or different ones whose second is empty from three on."""
    n, total = case["seqs"], case["total"]
    weight = [0 if n >= 3 and i == 1 else 1 + (3 * i) % 5 for i in range(n)]
    lengths = [total * w // sum(weight) for w in weight]
    lengths[0] += total - sum(lengths)
    return lengths


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        n = case["rows"] * case["dim"]
        out = n * (1 if case["quant"] else es)
        if case["quant"]:
            out += 4 * case["rows"] * (case["dim"] // case["group"] if case["group"] else 1)
        return dict(bytes=n * es * (3 if case["residual"] else 1) + out + 4 * case["dim"], flops=6 * n)
    if case["op"] == "norm_backward":
        n = case["rows"] * case["dim"]
        return dict(bytes=n * es * (4 if case["residual"] else 3) + 8 * case["dim"], flops=12 * n)
    t, hk, hv, state = case["total"], case["hk"], case["hv"], 4 * D * D
    if case["op"] == "gdn_decode":
        return dict(bytes=t * (2 * hk + 2 * hv) * D * es + t * hv * (8 + 2 * state), flops=t * hv * 6 * D * D)
    n = case["seqs"] * hv * state
    if case["op"] == "gdn_prefill":
        return dict(bytes=t * (2 * hk + 2 * hv) * D * es + 8 * t * hv + n * (2 if case["start"] else 1),
                    flops=t * hv * 6 * D * D)
    return dict(bytes=t * (4 * hk + 3 * hv) * D * es + 16 * t * hv + n * (3 if case["start"] else 1),
                flops=t * hv * 16 * D * D)


# ----------------------------------------------------------------- inputs ----
def _keys(shape, g, dtype):
    """Rows as they leave a projection: SiLU of N(0, 1), L2-normalised per (token, head)."""
    x = torch.nn.functional.silu(torch.randn(shape, generator=g, device="cuda"))
    return (x / x.norm(dim=-1, keepdim=True)).to(dtype)


def _gates(tokens, hv, g):
    """beta = sigmoid(N(0, 1)); log decay = -a softplus(N(0, 1)), a in [0.01, 4] for each head."""
    beta = torch.sigmoid(torch.randn(tokens, hv, generator=g, device="cuda"))
    a = torch.exp(torch.rand(hv, generator=g, device="cuda") * math.log(400.0) + math.log(0.01))
    decay = -a * torch.nn.functional.softplus(torch.randn(tokens, hv, generator=g, device="cuda"))
    return decay, beta


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype, op = _dtype(case), case["op"]
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = dict(case=case)
    if op in ("norm", "norm_backward"):
        rows, dim = case["rows"], case["dim"]
        s["x"] = (normal(rows, dim) * torch.exp(0.5 * normal(1, dim))).to(dtype)  # channels of different size
        s["weight"] = 1.0 + 0.2 * normal(dim)
        s["residual"] = (2.0 * normal(rows, dim)).to(dtype) if case["residual"] else None
        if op == "norm_backward":  # x is the normed row; the residual's slot is its other gradient
            s["grad_y"] = normal(rows, dim).to(dtype)
            s["grad_h"] = s.pop("residual")
        return s
    t, hk, hv = case["total"], case["hk"], case["hv"]
    s["q"], s["k"], s["v"] = _keys((t, hk, D), g, dtype), _keys((t, hk, D), g, dtype), normal(t, hv, D).to(dtype)
    s["log_decay"], s["beta"] = _gates(t, hv, g)
    if op == "gdn_decode":
        s["S"] = 0.1 * normal(case["slots"], hv, D, D)
        s["slots"] = torch.randperm(case["slots"], generator=g, device="cuda")[:t].to(torch.int32)
        return s
    s["lengths"] = _lengths(case)
    cu = [0]
    for n in s["lengths"]:
        cu.append(cu[-1] + n)
    s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["S0"] = 0.1 * normal(case["seqs"], hv, D, D) if case["start"] else None
    if op == "gdn_backward":
        s["grad_o"] = normal(t, hv, D).to(dtype)
        s["grad_S"] = 0.1 * normal(case["seqs"], hv, D, D) if case["start"] else None
    return s


# ------------------------------------------------------------- plain forms ----
def _padded(lengths):
    """Row of every place of the packed tokens padded to [sequences, chunks, C], or the row after the last."""
    n = torch.tensor(lengths, device="cuda")
    first = torch.cumsum(n, 0) - n
    at = torch.arange(max(1, -(-max(lengths) // C)) * C, device="cuda")
    idx = torch.where(at[None] < n[:, None], first[:, None] + at[None], sum(lengths))
    return idx.view(len(lengths), -1, C)


def _gather(x, idx, heads):
    """[T, h, ...] -> fp32 [sequences, heads, chunks, C, ...], zero behind a sequence's end, heads of a group alike."""
    x = torch.cat([x.float(), x.new_zeros((1,) + tuple(x.shape[1:]), dtype=torch.float32)])[idx]
    return x.repeat_interleave(heads // x.shape[3], 3).movedim(3, 1)


def _scatter(x, idx, tokens):
    """The reverse: fp32 [sequences, heads, chunks, C, ...] -> [T, heads, ...]."""
    x = x.movedim(1, 3)
    out = x.new_zeros((tokens + 1,) + tuple(x.shape[3:]))
    out[idx.reshape(-1)] = x.reshape((-1,) + tuple(x.shape[3:]))
    return out[:tokens]


def _chunk_terms(s):
    """What the chunks need besides the state: inputs in chunks, decays, T = (I + A)^-1 and P."""
    hv, idx = s["v"].shape[1], _padded(s["lengths"])
    q, k, v, beta = (_gather(s[n], idx, hv) for n in ("q", "k", "v", "beta"))
    g = torch.cumsum(_gather(s["log_decay"], idx, hv).double(), -1)
    low = torch.ones(C, C, device="cuda", dtype=torch.bool).tril()
    gam = torch.where(low, g[..., :, None] - g[..., None, :], -torch.inf).exp().float()
    kk, qk = k @ k.transpose(-1, -2), q @ k.transpose(-1, -2)
    A = (beta[..., None] * gam * kk).tril(-1)
    T = torch.eye(C, device="cuda").expand(A.shape).clone()
    for i in range(1, C):  # forward substitution, a row at a time
        T[..., i, :i] = -(A[..., i, None, :i] @ T[..., :i, :i]).squeeze(-2)
    return dict(idx=idx, q=q, k=k, v=v, beta=beta, gam=gam, kk=kk, qk=qk, A=A, T=T, P=gam * qk,
                eg=g.exp().float()[..., None], eo=(g[..., -1:] - g).exp().float()[..., None],
                ec=g[..., -1].exp().float()[..., None, None])


def _scan(s, c, keep):
    """The state over the chunks: outputs, the last state and, if `keep`, the start states and U."""
    shape = c["q"].shape
    S = torch.zeros(shape[0], shape[1], D, D, device="cuda") if s["S0"] is None else s["S0"].clone()
    o, starts, us = torch.empty_like(c["v"]), [], []
    for n in range(shape[2]):
        k, q, eg = c["k"][:, :, n], c["q"][:, :, n], c["eg"][:, :, n]
        U = c["T"][:, :, n] @ (c["beta"][:, :, n, :, None] * (c["v"][:, :, n] - eg * (k @ S)))
        o[:, :, n] = eg * (q @ S) + c["P"][:, :, n] @ U
        if keep:
            starts.append(S)
            us.append(U)
        S = c["ec"][:, :, n] * S + (c["eo"][:, :, n] * k).transpose(-1, -2) @ U
    return o, S, (torch.stack(starts, 2), torch.stack(us, 2)) if keep else None


def _prefill_plain(s):
    c = _chunk_terms(s)
    o, S, _ = _scan(s, c, False)
    return _scatter(o, c["idx"], s["v"].shape[0]).to(s["v"].dtype), S


def _backward_plain(s):
    c = _chunk_terms(s)
    _, _, (S, U) = _scan(s, c, True)
    t, hk, hv = s["v"].shape[0], s["q"].shape[1], s["v"].shape[1]
    dO = _gather(s["grad_o"], c["idx"], hv)
    tr = lambda x: x.transpose(-1, -2)  # noqa: E731
    dU, dS1, dR = tr(c["P"]) @ dO, torch.empty_like(S), torch.empty_like(U)
    qdo = tr(c["q"]) @ (c["eg"] * dO)
    dS = torch.zeros_like(S[:, :, 0]) if s["grad_S"] is None else s["grad_S"]
    for n in reversed(range(S.shape[2])):
        dS1[:, :, n] = dS
        dR[:, :, n] = tr(c["T"][:, :, n]) @ (dU[:, :, n] + c["eo"][:, :, n] * (c["k"][:, :, n] @ dS))
        x = -(c["beta"][:, :, n, :, None] * c["eg"][:, :, n]) * dR[:, :, n]
        dS = c["ec"][:, :, n] * dS + tr(c["k"][:, :, n]) @ x + qdo[:, :, n]
    beta = c["beta"][..., None]
    X = -(beta * c["eg"]) * dR
    KS, QS = c["k"] @ S, c["q"] @ S
    dA, dP = -(dR @ tr(U)).tril(-1), (dO @ tr(U)).tril()
    dqk, dkk = c["gam"] * dP, beta * c["gam"] * dA
    UdS = U @ tr(dS1)
    dq = c["eg"] * (dO @ tr(S)) + dqk @ c["k"]
    dk = X @ tr(S) + c["eo"] * UdS + tr(dqk) @ c["q"] + (dkk + tr(dkk)) @ c["k"]
    dbeta = (dR * (c["v"] - c["eg"] * KS)).double().sum(-1) + (dA * c["gam"] * c["kk"]).double().sum(-1)
    M = (dP * c["P"] + dA * c["A"]).double()
    e = (c["eo"] * c["k"] * UdS).double().sum(-1)  # through exp(gC - g)
    dg = M.sum(-1) - M.sum(-2) + (X * KS + c["eg"] * dO * QS).double().sum(-1) - e
    dg[..., -1] += e.sum(-1) + (c["ec"] * dS1 * S).double().sum((-1, -2))
    ddecay = dg.flip(-1).cumsum(-1).flip(-1)
    out = lambda x: _scatter(x, c["idx"], t)  # noqa: E731
    shared = lambda x: out(x).view(t, hk, hv // hk, D).sum(2).to(s["q"].dtype)  # noqa: E731
    return (shared(dq), shared(dk), out(beta * dR).to(s["v"].dtype), out(ddecay).float(), out(dbeta).float(), dS)


def _decode_plain(s):
    at, hv = s["slots"].long(), s["v"].shape[1]
    q, k = (s[n].float().repeat_interleave(hv // s[n].shape[1], 1)[..., None] for n in ("q", "k"))
    S = s["S"][at] * s["log_decay"].exp()[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (k * S).sum(-2))
    S = S + k * u[..., None, :]
    s["S"][at] = S
    return (q * S).sum(-2).to(s["v"].dtype), s["S"]


def _quantised(y, case):
    """y in 8 bits and its scales: e4m3 as it is, int8 (whose ties a last bit decides) as the values it stands for."""
    rows, dim = y.shape
    y = y.view(rows, -1, case["group"] or dim)
    qmax = QMAX[case["quant"]]
    scale = (y.abs().amax(-1, keepdim=True) / qmax).clamp_min(2.0 ** -126)
    z = (y / scale).clamp(-qmax, qmax)
    z = (z.round() * scale).to(torch.bfloat16) if case["quant"] == "int8" else z.float().to(torch.float8_e4m3fn)
    return z.view(rows, dim), scale.squeeze(-1)


def _norm_plain(s, eps=1e-6):
    x, case = s["x"], s["case"]
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    f = h.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + eps) * s["weight"]
    if not case["quant"]:
        return y.to(x.dtype), None, None if s["residual"] is None else h
    z, scale = _quantised(y, case)
    return z, scale, None if s["residual"] is None else h


def _norm_backward_plain(s, eps=1e-6):
    h, dy, w = s["x"].float(), s["grad_y"].float(), s["weight"]
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + eps)
    dx = r * w * dy - h * r ** 3 * (h * w * dy).mean(-1, keepdim=True)
    if s["grad_h"] is not None:
        dx = dx + s["grad_h"].float()
    return dx.to(s["x"].dtype), (dy * h * r).double().sum(0).float()


# ------------------------------------------------------------------- passes ----
def run(s):
    op = s["case"]["op"]
    if own:
        import linear_attention_chunkwise_gb300 as kda

        if op == "gdn_prefill":
            return kda.kda_gdn_prefill(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["cu_seqlens"], s["S0"])
        if op == "gdn_backward":
            return kda.kda_gdn_prefill_backward(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["cu_seqlens"],
                                                s["grad_o"], s["S0"], s["grad_S"])
        if op == "gdn_decode":
            return kda.kda_gdn_decode_step(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["S"], s["slots"]), s["S"]
        if op == "norm_backward":
            return kda.kda_rms_norm_backward(s["grad_y"], s["x"], s["weight"], grad_h=s["grad_h"], eps=1e-6)
        case = s["case"]
        if not case["quant"]:
            return kda.kda_rms_norm(s["x"], s["weight"], s["residual"], eps=1e-6)
        y, scale, h = kda.kda_rms_norm(s["x"], s["weight"], s["residual"], eps=1e-6, quant=case["quant"], group=case["group"])
        if case["quant"] == "int8":
            z = torch.empty(y.shape, dtype=torch.bfloat16, device=y.device)
            torch.mul(y.view(y.shape[0], scale.shape[1], -1), scale[..., None], out=z.view(y.shape[0], scale.shape[1], -1))
            y = z
        return y, scale, h
    return {"gdn_prefill": _prefill_plain, "gdn_backward": _backward_plain, "gdn_decode": _decode_plain,
            "norm": _norm_plain, "norm_backward": _norm_backward_plain}[op](s)


# ------------------------------------------------------------------ 64 bits ----
def _walk(s):
    """Token by token in 64 bits: yields (active sequences, rows, q, k, v, beta, decay) for every position."""
    hv = s["v"].shape[1]
    wide = lambda x: x.double().repeat_interleave(hv // x.shape[1], 1)  # noqa: E731
    q, k, v, beta, dec = wide(s["q"]), wide(s["k"]), s["v"].double(), s["beta"].double(), s["log_decay"].double().exp()
    first = [sum(s["lengths"][:i]) for i in range(len(s["lengths"]))]
    steps = []
    for t in range(max(s["lengths"])):
        live = [i for i, n in enumerate(s["lengths"]) if t < n]
        steps.append((live, [first[i] + t for i in live]))
    return q, k, v, beta, dec, steps


def _pick(ids):
    """An index for a list of places: a slice for one place, which makes views instead of copies."""
    return slice(ids[0], ids[0] + 1) if len(ids) == 1 else torch.tensor(ids, device="cuda")


def _exact_prefill(s):
    q, k, v, beta, dec, steps = _walk(s)
    n, hv = len(s["lengths"]), v.shape[1]
    S = torch.zeros(n, hv, D, D, device="cuda", dtype=torch.float64) if s["S0"] is None else s["S0"].double()
    o = torch.zeros_like(v)
    for live, rows in steps:
        b, r = _pick(live), _pick(rows)
        x = S[b] * dec[r][..., None, None]
        u = beta[r][..., None] * (v[r] - (k[r][..., None, :] @ x).squeeze(-2))
        x = x + k[r][..., :, None] * u[..., None, :]
        S[b] = x
        o[r] = (q[r][..., None, :] @ x).squeeze(-2)
    return o, S


def _exact_backward(s):
    q, k, v, beta, dec, steps = _walk(s)
    n, hv, t, hk = len(s["lengths"]), v.shape[1], v.shape[0], s["q"].shape[1]
    f64 = dict(device="cuda", dtype=torch.float64)
    S = torch.zeros(n, hv, D, D, **f64) if s["S0"] is None else s["S0"].double()
    before = torch.empty(t, hv, D, D, **f64)  # every token's state before it
    for live, rows in steps:
        b, r = _pick(live), _pick(rows)
        before[r] = S[b]
        x = S[b] * dec[r][..., None, None]
        u = beta[r][..., None] * (v[r] - (k[r][..., None, :] @ x).squeeze(-2))
        S[b] = x + k[r][..., :, None] * u[..., None, :]
    G = torch.zeros_like(S) if s["grad_S"] is None else s["grad_S"].double()
    dO = s["grad_o"].double()
    dq, dk, dv, dla, db = (torch.zeros_like(x) for x in (v, v, v, beta, beta))
    row = lambda x, m: (x[..., None, :] @ m).squeeze(-2)   # m^T x  # noqa: E731
    col = lambda m, x: (m @ x[..., :, None]).squeeze(-1)   # m x  # noqa: E731
    for live, rows in reversed(steps):
        b, r = _pick(live), _pick(rows)
        kr, br = k[r], beta[r][..., None]
        x = before[r] * dec[r][..., None, None]
        e = v[r] - row(kr, x)                                  # o = S^T q, S = x + k (b e)^T, e = v - x^T k
        Gb = G[b] + q[r][..., :, None] * dO[r][..., None, :]
        dq[r] = col(x + kr[..., :, None] * (br * e)[..., None, :], dO[r])
        gk = row(kr, Gb)
        db[r] = (gk * e).sum(-1)
        dv[r] = br * gk
        dk[r] = col(Gb, br * e) - col(x, br * gk)
        Gx = Gb - kr[..., :, None] * (br * gk)[..., None, :]
        dla[r] = (Gx * x).sum((-1, -2))
        G[b] = Gx * dec[r][..., None, None]
    shared = lambda x: x.view(t, hk, hv // hk, D).sum(2)  # noqa: E731
    return shared(dq), shared(dk), dv, dla, db, G


def _exact_decode(s):
    hv = s["v"].shape[1]
    q, k = (s[n].double().repeat_interleave(hv // s[n].shape[1], 1) for n in ("q", "k"))
    out, o = s["S"].double(), []
    for i, slot in enumerate(s["slots"].tolist()):
        S = out[slot] * s["log_decay"][i].double().exp()[:, None, None]
        e = s["v"][i].double() - torch.einsum("hi,hij->hj", k[i], S)
        S = S + torch.einsum("h,hi,hj->hij", s["beta"][i].double(), k[i], e)
        out[slot] = S
        o.append(torch.einsum("hi,hij->hj", q[i], S))
    return torch.stack(o), out


def _exact_norm(s, eps=1e-6):
    x, case = s["x"].double(), s["case"]
    h = x if s["residual"] is None else x + s["residual"].double()
    f = h.to(s["x"].dtype).double()  # the norm is that of the stored row
    y = f / (f.square().sum(-1, keepdim=True) / case["dim"] + eps).sqrt() * s["weight"].double()
    scale = None
    if case["quant"]:
        y, scale = _quantised(y, case)
        y = y.double()
    return y, scale, None if s["residual"] is None else h


def _exact_norm_backward(s, eps=1e-6):
    h, w = s["x"].double().requires_grad_(), s["weight"].double().requires_grad_()
    y = h / (h.square().sum(-1, keepdim=True) / h.shape[1] + eps).sqrt() * w
    loss = (y * s["grad_y"].double()).sum()
    if s["grad_h"] is not None:
        loss = loss + (h * s["grad_h"].double()).sum()
    return torch.autograd.grad(loss, (h, w))


def exact(case, seed):
    s = prepare(case, seed)
    return {"gdn_prefill": _exact_prefill, "gdn_backward": _exact_backward, "gdn_decode": _exact_decode,
            "norm": _exact_norm, "norm_backward": _exact_norm_backward}[case["op"]](s)
