"""Cases of the linear attention with a decay for each head, and of the head norms with the rotation before it.

`listed()` and `draw()` give cases, `prepare()` the inputs that a program has in hand, `run()` one pass through an
operator: in its plain form (elementary torch operations in fp32), or, where `own` is true, through the package's calls.
`exact()` gives the same outputs from the definition in float64, `work()` what a pass cannot do without.

Operators (per batch row or packed sequence; head h of v shares the q and k of head h // (H // Hk)):

    linattn      S_t = exp(log_decay_h) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t     (forward, backward, one token)
    qk_norm_rope y = R(position) (x / sqrt(mean(x^2) + eps) * weight), for every head of q and k (forward, backward);
                 "l2" takes the sum of squares in the place of their mean
"""

import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------------------------------------------------ cases
def _lin(name, op, dtype, B, T, Hk, H, Dk, Dv, **more):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "T": T, "Hk": Hk, "H": H, "Dk": Dk, "Dv": Dv, **more}


def _norm(name, op, dtype, B, T, Hk, H, D, rot, **more):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "T": T, "Hk": Hk, "H": H, "D": D, "rot": rot, **more}


def listed():
    return [
        # q and k of one generated token for each of 256 requests, cut from the fused projection's rows
        _norm("qk norm rope, 256 tokens", "norm_fwd", "bf16", 256, 1, 16, 16, 128, 128, l2=False, pairs=False),
        # the same layer in training: 8 sequences of 4096 tokens
        _norm("qk norm rope, 8 x 4096", "norm_fwd", "bf16", 8, 4096, 16, 16, 128, 128, l2=False, pairs=False),
        # its gradients, written into the fused projection's gradient rows
        _norm("qk norm rope backward, 8 x 4096", "norm_bwd", "bf16", 8, 4096, 16, 16, 128, 128, l2=False, pairs=False),
        # fp32, fewer key heads, half of each head rotated in neighbouring pairs, L2 norm, odd length
        _norm("qk norm rope backward, fp32 3 x 1237", "norm_bwd", "fp32", 3, 1237, 4, 12, 64, 32, l2=True, pairs=True),
        # prefill of 8 prompts that keeps the final states for decoding
        _lin("prefill 8 x 4096", "fwd", "bf16", 8, 4096, 16, 16, 128, 128, s0=False, sfin=True, decay="slopes"),
        # one long prompt: few heads to fill the card with
        _lin("prefill 1 x 65536", "fwd", "bf16", 1, 65536, 16, 16, 128, 128, s0=False, sfin=True, decay="near1"),
        # packed prompts of different lengths that go on from kept states, q and k shared by pairs of value heads
        _lin("packed prefill, 11 prompts", "fwd", "bf16", 11, 14029, 8, 16, 128, 64, s0=True, sfin=True, decay="slopes",
             packed=True),
        # fp32, odd length, small heads
        _lin("prefill fp32 2 x 1001", "fwd", "fp32", 2, 1001, 8, 8, 64, 64, s0=True, sfin=True, decay="slopes"),
        # the training backward at the benchmark's sizes
        _lin("backward 8 x 4096", "bwd", "bf16", 8, 4096, 16, 16, 128, 128, s0=False, sfin=False, decay="slopes"),
        # backward of an odd length with shared q and k heads, initial states and their gradients
        _lin("backward 2 x 2055, shared heads", "bwd", "bf16", 2, 2055, 4, 12, 64, 128, s0=True, sfin=True, decay="near1"),
        # one decode step of 256 requests whose states lie in a pool
        _lin("decode 256 requests", "decode", "bf16", 256, 1, 16, 16, 128, 128, decay="slopes", pool=300),
        # one decode step of one request: latency
        _lin("decode 1 request", "decode", "bf16", 1, 1, 16, 16, 128, 128, decay="slopes", pool=0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm_fwd", "norm_bwd", "fwd", "fwd", "bwd", "bwd", "decode"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    Hk = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    H = Hk * rng.choice([1, 1, 2, 3] if Hk < 8 else [1, 2])
    if kind.startswith("norm"):
        D = rng.choice([32, 64, 128])
        rot = rng.choice([r for r in (16, 32, 64, 128) if r <= D])
        tokens = _log_int(rng, 1, min(32768, 32 * 32768 // (H + Hk)))
        B = min(tokens, _log_int(rng, 1, 64))
        return {"op": kind, "dtype": dtype, "B": B, "T": max(1, tokens // B), "Hk": Hk, "H": H, "D": D, "rot": rot,
                "l2": rng.random() < 0.3, "pairs": rng.random() < 0.4}
    Dk, Dv = rng.choice([32, 64, 128]), rng.choice([32, 64, 128])
    decay = rng.choice(["slopes", "near1"])
    if kind == "decode":
        B = _log_int(rng, 1, min(256, 4096 // H))
        return {"op": kind, "dtype": dtype, "B": B, "T": 1, "Hk": Hk, "H": H, "Dk": Dk, "Dv": Dv, "decay": decay,
                "pool": rng.choice([0, B + rng.randrange(1, 50)])}
    tokens = _log_int(rng, 1, min(32768, 16 * (40000 if kind == "fwd" else 24576) // H))
    case = {"op": kind, "dtype": dtype, "Hk": Hk, "H": H, "Dk": Dk, "Dv": Dv, "decay": decay,
            "s0": rng.random() < 0.5, "sfin": rng.random() < 0.6}
    if rng.random() < 0.35:
        return {**case, "B": rng.randrange(2, 14), "T": max(64, tokens), "packed": True}
    B = min(tokens, _log_int(rng, 1, 16))
    return {**case, "B": B, "T": max(1, tokens // B)}


# ----------------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32).to(dtype)


def _offsets(case, seed):
    """Offsets of the packed sequences: uneven, one of them empty and one of a single token where there is room."""
    N, T = case["B"], case["T"]
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(N, generator=g, dtype=torch.float64).pow(2) + 0.02
    lens = (w / w.sum() * T).long()
    if N > 3:
        lens[1], lens[2] = 0, 1
    lens[N - 1] += T - int(lens.sum())
    return [0] + torch.cumsum(lens, 0).tolist()


def _log_decay(case):
    h = torch.arange(case["H"], dtype=torch.float64)
    if case["decay"] == "slopes":  # geometric slopes, 0.7 to 2^-8
        return -(2.0 ** (-8.0 * (h + 1) / case["H"]))
    return torch.log1p(-(2.0 ** (-5.0 - 10.0 * h / case["H"])))  # 1 - 2^-5 to 1 - 2^-15


def prepare(case, seed):
    g = _gen(seed)
    B, T, Hk, H, dt = case["B"], case["T"], case["Hk"], case["H"], DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"].startswith("norm"):
        D = case["D"]
        s["qkv"] = _randn(g, B, T, (H + 2 * Hk) * D, dtype=dt)  # the projection's rows: H heads of q, Hk of k, Hk of v
        s["q"] = s["qkv"][..., : H * D].unflatten(-1, (H, D))
        s["k"] = s["qkv"][..., H * D : (H + Hk) * D].unflatten(-1, (Hk, D))
        first = torch.randint(0, 120000, (B, 1), generator=g, device=DEVICE)
        s["positions"] = first + torch.arange(T, device=DEVICE)
        half = case["rot"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(DEVICE)
        s["q_weight"] = None if case["l2"] else 1 + 0.2 * _randn(g, D)
        s["k_weight"] = None if case["l2"] else 1 + 0.2 * _randn(g, D)
        if case["op"] == "norm_bwd":
            s["dq_out"], s["dk_out"] = _randn(g, B, T, H, D, dtype=dt), _randn(g, B, T, Hk, D, dtype=dt)
            s["dqkv"] = torch.zeros_like(s["qkv"])
        return s
    Dk, Dv = case["Dk"], case["Dv"]
    s["log_decay"] = _log_decay(case).float().to(DEVICE)
    s["scale"] = Dk ** -0.5
    if case["op"] == "decode":
        s["q"], s["k"], s["v"] = (_randn(g, B, n, d, dtype=dt) for n, d in ((Hk, Dk), (Hk, Dk), (H, Dv)))
        s["S"] = _randn(g, case["pool"] or B, H, Dk, Dv)
        if case["pool"]:
            s["slots"] = torch.randperm(case["pool"], generator=g, device=DEVICE)[:B].to(torch.int32)
        s["o"] = torch.empty(B, H, Dv, dtype=dt, device=DEVICE)
        return s
    rows, N = (1, B) if case.get("packed") else (B, B)
    s["q"], s["k"], s["v"] = (_randn(g, rows, T, n, d, dtype=dt) for n, d in ((Hk, Dk), (Hk, Dk), (H, Dv)))
    s["S0"] = _randn(g, N, H, Dk, Dv) if case["s0"] else None
    if case.get("packed"):
        cu = _offsets(case, seed)
        s["cu"] = torch.tensor(cu, dtype=torch.int64, device=DEVICE)
        s["longest"] = max(b - a for a, b in zip(cu, cu[1:]))
    if case["op"] == "bwd":
        s["dO"] = _randn(g, rows, T, H, Dv, dtype=dt)
        s["dS_final"] = _randn(g, N, H, Dk, Dv) if case["sfin"] else None
    return s


# -------------------------------------------------------------------------------------------------- the plain forms
def _rotated(x, cos, sin, half, pairs):
    a, b, rest = (x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2], x[..., 2 * half :]) if pairs else (
        x[..., :half], x[..., half : 2 * half], x[..., 2 * half :])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if pairs else torch.cat((a, b), -1)
    return torch.cat((turned, rest), -1)


def _cos_sin(s, dtype):
    angle = s["positions"].double()[..., None, None] * s["inv_freq"].double()
    return torch.cos(angle).to(dtype), torch.sin(angle).to(dtype)


def _inverse_norm(x, l2):
    x2 = x * x
    return torch.rsqrt((x2.sum(-1, keepdim=True) if l2 else x2.mean(-1, keepdim=True)) + EPS)


def _plain_norm(s):
    c = s["case"]
    cos, sin = _cos_sin(s, torch.float32)
    half, dt = c["rot"] // 2, s["q"].dtype
    H, D, Hk = c["H"], c["D"], c["Hk"]

    def forward(x, w):
        x = x.float()
        y = x * _inverse_norm(x, c["l2"])
        return _rotated(y if w is None else y * w, cos, sin, half, c["pairs"]).to(dt)

    def backward(x, w, dy):
        x, g = x.float(), _rotated(dy.float(), cos, -sin, half, c["pairs"])
        r = _inverse_norm(x, c["l2"])
        h = g if w is None else g * w
        share = (h * x).sum(-1, keepdim=True) * r * r * (1.0 if c["l2"] else 1.0 / D)
        return (r * (h - x * share)).flatten(-2).to(dt), (g * x * r).sum((0, 1, 2))

    if c["op"] == "norm_fwd":
        return {"q_out": forward(s["q"], s["q_weight"]), "k_out": forward(s["k"], s["k_weight"])}
    (dq, dqw), (dk, dkw) = (backward(s[n], s[n + "_weight"], s["d" + n + "_out"]) for n in "qk")
    s["dqkv"][..., : H * D], s["dqkv"][..., H * D : (H + Hk) * D] = dq, dk
    out = {"dqkv": s["dqkv"]}
    return out if c["l2"] else {**out, "dq_weight": dqw, "dk_weight": dkw}


def _power(log_decay, n):
    """exp(n log_decay) for a tensor of exponents n whose first dimension (or any size-1 one) is the head."""
    return torch.exp(log_decay.double().view(-1, *[1] * (n.dim() - 1)) * n.double()).float()


def _attend(q, k, v, log_decay, lens, S0, first):
    """sum over j <= t of decay^(t-j) (q_t . k_j) v_j + decay^(t+first) q_t S0, and the sum of decay^(T-1-j) k_j v_j^T (without S0).

    q, k [N, H, T, Dk], v [N, H, T, Dv] in fp32, every row's tokens at its end (zeros before them); the sums run over
    pieces of C tokens, whose states are joined by one product with the matrix of the decays between pieces."""
    N, H, T, Dk = q.shape
    Dv, C = v.shape[-1], 64 if T <= 8192 else 256
    P = -(-T // C)
    q, k, v = (torch.nn.functional.pad(x, (0, 0, P * C - T, 0)).view(N, H, P, C, x.shape[-1]) for x in (q, k, v))
    i = torch.arange(C, device=q.device)
    past = i[:, None] - i[None, :]
    within = torch.where(past >= 0, _power(log_decay, past.clamp(min=0)[None]), 0.0)
    o = (torch.matmul(q, k.transpose(-1, -2).contiguous()) * within[:, None]).matmul(v)
    new = torch.matmul((k * _power(log_decay, (C - 1 - i)[None])[:, None, :, None]).transpose(-1, -2).contiguous(), v)
    p = torch.arange(P + 1, device=q.device)
    gap = p[:, None] - 1 - p[None, :P]
    between = torch.where(gap >= 0, _power(log_decay, gap.clamp(min=0)[None] * C), 0.0)
    S = torch.matmul(between, new.view(N, H, P, Dk * Dv)).view(N, H, P + 1, Dk, Dv)
    o = o + torch.matmul(q * _power(log_decay, (i + 1)[None])[:, None, :, None], S[:, :, :P])
    o, q = (x.view(N, H, P * C, -1)[:, :, P * C - T :] for x in (o, q))
    if S0 is not None:
        t = torch.arange(T, device=q.device)[None] - (T - lens)[:, None]  # [N, T], below zero before a row's tokens
        weight = torch.exp(log_decay.double()[None, :, None] * (t.clamp(min=0) + first).double()[:, None]).float()
        o = o + weight[..., None] * torch.matmul(q, S0)
    return o, S[:, :, P]


def _decayed(S0, log_decay, lens):
    """decay^T S0 for every sequence's length T; zero without a state."""
    if S0 is None:
        return 0.0
    return torch.exp(log_decay.double()[None] * lens.double()[:, None]).float()[..., None, None] * S0


def _rows(s, x, flip=False):
    """[rows, T, heads, D] of any type as [N, H, T, D] in fp32, every sequence at the end of its row."""
    c = s["case"]
    x = x.float()
    if "cu" in s:
        cu, T = s["cu"], max(1, s["longest"])
        at = (cu[1:, None] - T + torch.arange(T, device=x.device)[None]) if not flip else (
            cu[:-1, None] + T - 1 - torch.arange(T, device=x.device)[None])
        fine = (at >= cu[:-1, None]) & (at < cu[1:, None])
        x = torch.where(fine[..., None, None], x[0][at.clamp(0, c["T"] - 1)], 0.0)
    elif flip:
        x = x.flip(1)
    return x.repeat_interleave(c["H"] // x.shape[2], 2).transpose(1, 2).contiguous()


def _unrows(s, x, flip=False):
    """_rows' inverse: [N, H, T, D] to [rows, T, H, D]."""
    x = x.transpose(1, 2)
    if "cu" in s:
        cu, T = s["cu"], max(1, s["longest"])
        at = (cu[1:, None] - T + torch.arange(T, device=x.device)[None]) if not flip else (
            cu[:-1, None] + T - 1 - torch.arange(T, device=x.device)[None])
        fine = (at >= cu[:-1, None]) & (at < cu[1:, None])
        out = x.new_zeros(s["case"]["T"], *x.shape[2:])
        out[at[fine]] = x[fine]
        return out[None]
    return x.flip(1) if flip else x


def _lens(s):
    return s["cu"][1:] - s["cu"][:-1] if "cu" in s else torch.full((s["case"]["B"],), s["case"]["T"], device=DEVICE)


def _plain_linattn(s):
    c, lens, ld, dt = s["case"], _lens(s), s["log_decay"], s["q"].dtype
    if c["op"] == "fwd":
        o, new = _attend(*(_rows(s, s[n]) for n in "qkv"), ld, lens, s["S0"], 1)
        out = {"o": _unrows(s, s["scale"] * o).to(dt)}
        return {**out, "S_final": new + _decayed(s["S0"], ld, lens)} if c["sfin"] else out

    def shared(x):  # the sum over the heads of v that share one of q and k
        return x.unflatten(2, (c["Hk"], -1)).sum(3).to(dt)

    def turned(S):
        return None if S is None else S.transpose(-1, -2).contiguous()

    q, k, v, dO = (_rows(s, s[n]) for n in ("q", "k", "v", "dO"))
    dq, _ = _attend(dO, v, k, ld, lens, turned(s["S0"]), 1)
    out = {"dq": shared(_unrows(s, s["scale"] * dq))}
    # reversed in time, where the gradient of the final state enters undecayed
    q, k, v, dO = (_rows(s, s[n], True) for n in ("q", "k", "v", "dO"))
    q = q * s["scale"]
    dk, _ = _attend(v, dO, q, ld, lens, turned(s["dS_final"]), 0)
    dv, new = _attend(k, q, dO, ld, lens, s["dS_final"], 0)
    out = {**out, "dk": shared(_unrows(s, dk, True)), "dv": _unrows(s, dv, True).to(dt)}
    if c["s0"]:  # the sum of decay^(t+1) q_t dO_t^T, and decay^T dS_final
        out["dS0"] = torch.exp(ld)[None, :, None, None] * new + _decayed(s["dS_final"], ld, lens)
    return out


def _plain_decode(s):
    G = s["case"]["H"] // s["case"]["Hk"]
    q, k = (s[n].float().repeat_interleave(G, 1) for n in "qk")
    S = s["S"][s["slots"].long()] if "slots" in s else s["S"]
    S = torch.exp(s["log_decay"])[None, :, None, None] * S + k[..., None] * s["v"].float()[:, :, None, :]
    o = s["scale"] * (q[..., None] * S).sum(-2)
    if "slots" in s:
        s["S"][s["slots"].long()] = S
    else:
        s["S"].copy_(S)
    s["o"].copy_(o)
    return {"o": s["o"], "S": s["S"]}


# --------------------------------------------------------------------------------------------- the package's calls
def _own(s):
    import delta_rule_recurrent_gdn_amd as gdn

    c = s["case"]
    if c["op"].startswith("norm"):
        more = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, l2=c["l2"], interleaved=c["pairs"])
        if c["op"] == "norm_fwd":
            q, k = gdn.gdn2_qk_norm_rope_fwd(s["q"], s["k"], s["positions"], s["inv_freq"], **more)
            return {"q_out": q, "k_out": k}
        H, D, Hk = c["H"], c["D"], c["Hk"]
        g = gdn.gdn2_qk_norm_rope_bwd(
            s["dq_out"], s["dk_out"], s["q"], s["k"], s["positions"], s["inv_freq"],
            dq=s["dqkv"][..., : H * D].unflatten(-1, (H, D)),
            dk=s["dqkv"][..., H * D : (H + Hk) * D].unflatten(-1, (Hk, D)), **more)
        out = {"dqkv": s["dqkv"]}
        return out if c["l2"] else {**out, "dq_weight": g["dq_weight"], "dk_weight": g["dk_weight"]}
    if c["op"] == "decode":
        x = (s["q"], s["k"], s["v"], s["log_decay"], s["S"])
        if "slots" in s:
            gdn.gdn2_linattn_decode_step_slots(*x, s["slots"], scale=s["scale"], o=s["o"])
        else:
            gdn.gdn2_linattn_decode_step(*x, scale=s["scale"], o=s["o"])
        return {"o": s["o"], "S": s["S"]}
    x = (s["q"], s["k"], s["v"], s["log_decay"])
    if c["op"] == "fwd":
        more = dict(S0=s["S0"], scale=s["scale"], want_final_state=c["sfin"])
        if "cu" in s:
            o, last = gdn.gdn2_linattn_fwd_varlen(*x, s["cu"], **more)
        else:
            o, last = gdn.gdn2_linattn_fwd_chunked(*x, **more)
        return {"o": o, "S_final": last} if c["sfin"] else {"o": o}
    more = dict(S0=s["S0"], dS_final=s["dS_final"], scale=s["scale"], want_dS0=c["s0"])
    if "cu" in s:
        g = gdn.gdn2_linattn_bwd_varlen(*x, s["dO"], s["cu"], **more)
    else:
        g = gdn.gdn2_linattn_bwd_chunked(*x, s["dO"], **more)
    return {n: g[n] for n in ("dq", "dk", "dv", "dS0") if g[n] is not None}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_norm(state) if op.startswith("norm") else _plain_decode(state) if op == "decode" else _plain_linattn(state)


# ------------------------------------------------------------------------------------------------------------- work
def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    B, T, Hk, H = case["B"], case["T"], case["Hk"], case["H"]
    if case["op"].startswith("norm"):
        n = B * T * (H + Hk) * case["D"]
        back = case["op"] == "norm_bwd"
        return {"bytes": n * b * (3 if back else 2) + 8 * B * T, "flops": n * (16 if back else 8)}
    Dk, Dv = case["Dk"], case["Dv"]
    if case["op"] == "decode":
        return {"bytes": 8 * B * H * Dk * Dv + b * B * (2 * Hk * Dk + 2 * H * Dv), "flops": 5 * B * H * Dk * Dv}
    rows, N = (T, B) if case.get("packed") else (B * T, B)
    token = b * (2 * Hk * Dk + H * Dv)
    state = 4 * N * H * Dk * Dv
    if case["op"] == "fwd":
        moved = rows * (token + b * H * Dv) + state * (case["s0"] + case["sfin"])
        return {"bytes": moved, "flops": 4 * rows * H * Dk * Dv}
    moved = rows * (2 * token + b * H * Dv) + state * (2 * case["s0"] + case["sfin"])
    return {"bytes": moved, "flops": 10 * rows * H * Dk * Dv}


# ---------------------------------------------------------------------------------------- the definition in 64 bits
def _exact_norm(s):
    c = s["case"]
    D, half = c["D"], c["rot"] // 2
    angle = s["positions"].double()[:, :, None] * s["inv_freq"].double()
    one = [2 * j if c["pairs"] else j for j in range(half)]
    two = [2 * j + 1 if c["pairs"] else j + half for j in range(half)]

    def rotate(x, sign):  # [B, T, heads, D]
        y = x.clone()
        cos, sin = torch.cos(angle)[:, :, None], sign * torch.sin(angle)[:, :, None]
        y[..., one] = x[..., one] * cos - x[..., two] * sin
        y[..., two] = x[..., one] * sin + x[..., two] * cos
        return y

    found = {}
    for n in "qk":
        x = s[n].double()
        w = torch.ones(D, dtype=torch.float64, device=DEVICE) if s[n + "_weight"] is None else s[n + "_weight"].double()
        m = (x ** 2).sum(-1, keepdim=True) / (1 if c["l2"] else D) + EPS
        if c["op"] == "norm_fwd":
            found[n + "_out"] = rotate(x / m.sqrt() * w, 1.0)
            continue
        g = rotate(s["d" + n + "_out"].double(), -1.0)
        found["d" + n + "_weight"] = (g * x / m.sqrt()).sum((0, 1, 2))
        dot = (g * w * x).sum(-1, keepdim=True) / (1 if c["l2"] else D)
        found["d" + n] = g * w / m.sqrt() - x * dot / m ** 1.5
    if c["op"] == "norm_fwd":
        return found
    d = torch.zeros(s["qkv"].shape, dtype=torch.float64, device=DEVICE)
    H, Hk = c["H"], c["Hk"]
    d[..., : H * D], d[..., H * D : (H + Hk) * D] = found["dq"].flatten(-2), found["dk"].flatten(-2)
    out = {"dqkv": d}
    return out if c["l2"] else {**out, "dq_weight": found["dq_weight"], "dk_weight": found["dk_weight"]}


def _steps(x, y, z, g, S, before):
    """Runs S <- decay S + y_t z_t^T over t in blocks, returning r_t = S^T x_t and the last S. `before`: S is decayed
    once before the first token (as the forward recurrence has it) or not (the reversed one). x, y [H, T, A], z [H, T, B]."""
    H, T = x.shape[:2]
    out = torch.empty(H, T, z.shape[-1], dtype=torch.float64, device=x.device)
    g = g[:, None, None]
    for a in range(0, T, 128):
        b = min(T, a + 128)
        n = torch.arange(b - a, dtype=torch.float64, device=x.device)
        lag = n[:, None] - n[None, :]
        score = torch.bmm(x[:, a:b], y[:, a:b].transpose(1, 2).contiguous()) * torch.exp(g * lag.clamp(min=0)) * (lag >= 0)
        out[:, a:b] = torch.bmm(score, z[:, a:b]) + torch.exp(g * (n[:, None] + before)) * torch.bmm(x[:, a:b], S)
        left = torch.exp(g * (b - a - before - n[:, None]))
        S = torch.exp(g * (b - a)) * S + torch.bmm((left * y[:, a:b]).transpose(1, 2).contiguous(), z[:, a:b])
    return out, S


def _exact_linattn(s):
    c, ld = s["case"], s["log_decay"].double()
    Hk, H, Dk, Dv = c["Hk"], c["H"], c["Dk"], c["Dv"]
    cu = s["cu"].tolist() if "cu" in s else [0] * (c["B"] + 1)
    back = c["op"] == "bwd"
    new = lambda n, d: torch.zeros(s["q"].shape[0], c["T"], n, d, dtype=torch.float64, device=DEVICE)  # noqa: E731
    out = {"dq": new(Hk, Dk), "dk": new(Hk, Dk), "dv": new(H, Dv)} if back else {"o": new(H, Dv)}
    states = torch.zeros(c["B"], H, Dk, Dv, dtype=torch.float64, device=DEVICE)
    for n in range(c["B"]):
        at = (0, slice(cu[n], cu[n + 1])) if "cu" in s else (n, slice(0, c["T"]))
        head = lambda x: x[at].double().repeat_interleave(H // x.shape[2], 1).transpose(0, 1).contiguous()  # noqa: E731,B023
        q, k, v = head(s["q"]) * s["scale"], head(s["k"]), head(s["v"])
        S0 = torch.zeros(H, Dk, Dv, dtype=torch.float64, device=DEVICE) if s["S0"] is None else s["S0"][n].double()
        if not back:
            o, states[n] = _steps(q, k, v, ld, S0, 1)
            out["o"][at] = o.transpose(0, 1)
            continue
        dO = head(s["dO"])
        dS = torch.zeros_like(S0) if s["dS_final"] is None else s["dS_final"][n].double()
        dq, _ = _steps(dO, v, k, ld, S0.transpose(1, 2).contiguous(), 1)
        q, k, v, dO = (x.flip(1).contiguous() for x in (q, k, v, dO))
        dk, _ = _steps(v, dO, q, ld, dS.transpose(1, 2).contiguous(), 0)
        dv, states[n] = _steps(k, q, dO, ld, dS, 0)
        out["dq"][at] = (dq * s["scale"]).transpose(0, 1).unflatten(1, (Hk, -1)).sum(2)
        out["dk"][at] = dk.flip(1).transpose(0, 1).unflatten(1, (Hk, -1)).sum(2)
        out["dv"][at] = dv.flip(1).transpose(0, 1)
    if back:
        return {**out, "dS0": states} if c["s0"] else out
    return {**out, "S_final": states} if c["sfin"] else out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    if case["op"] != "decode":
        return _exact_linattn(s)
    S, G = s["S"].double(), case["H"] // case["Hk"]
    at = s["slots"].long() if "slots" in s else torch.arange(case["B"], device=DEVICE)
    o = torch.empty(case["B"], case["H"], case["Dv"], dtype=torch.float64, device=DEVICE)
    for h in range(case["H"]):
        q, k, v = s["q"][:, h // G].double(), s["k"][:, h // G].double(), s["v"][:, h].double()
        S[at, h] = torch.exp(s["log_decay"][h].double()) * S[at, h] + k[:, :, None] * v[:, None, :]
        o[:, h] = s["scale"] * torch.bmm(q[:, None], S[at, h])[:, 0]
    return {"o": o, "S": S}
