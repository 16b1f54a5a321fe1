"""Linear attention with a decay for each head on the GPU, against the float64 oracle that steps it token by token.

Tolerances, element by element: with A the same recurrence over absolute values (the sum of the terms' magnitudes),
- bf16 outputs: one rounding of the result (2^-8 of it), and 2^-14 A: scores and states enter their products as two
  bf16 terms (what is left of them is at most 2^-16 and 2^-15 of the value), and the fp32 sums;
- fp32 outputs and states: 2^-24 A for each of the at most 4 (T + D) + 64 sums, products and powers in a row.
"""

import numpy as np
import pytest
import torch

import oracle.linattn as O

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make(seed, B, T, Hk, H, Dk, Dv, dt, decay=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = {"q": r(B, T, Hk, Dk).to(dt), "k": r(B, T, Hk, Dk).to(dt), "v": r(B, T, H, Dv).to(dt),
         "dO": r(B, T, H, Dv).to(dt), "S0": r(B, H, Dk, Dv), "dS": r(B, H, Dk, Dv)}
    x["ld"] = -torch.rand(H, generator=g) ** 3 if decay is None else torch.full((H,), decay)
    return x


def dev(x):
    return {n: t.cuda() for n, t in x.items()}


def check(name, got, ref, mag, T, D):
    got32, ref, mag = got.detach().cpu().double().numpy(), np.asarray(ref), np.asarray(mag)
    assert got32.shape == ref.shape
    if got.dtype == BF16:
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -14 * mag
    else:
        tol = (4 * (T + D) + 64) * 2.0 ** -24 * mag
    off = np.abs(got32 - ref) - tol
    assert np.isfinite(got32).all() and (off <= 1e-30).all(), (name, float(off.max()), float(np.abs(got32 - ref).max()))


def oracle_fwd(x, S0=True, scale=1.0):
    a = lambda f: O.linattn_forward(f(x["q"]), f(x["k"]), f(x["v"]), x["ld"], f(x["S0"]) if S0 else None, scale)  # noqa: E731
    return a(lambda t: t), a(lambda t: t.abs())


def oracle_bwd(x, S0=True, dS=True, scale=1.0):
    a = lambda f: O.linattn_backward(f(x["q"]), f(x["k"]), f(x["v"]), x["ld"], f(x["dO"]), f(x["S0"]) if S0 else None,  # noqa: E731
                                     f(x["dS"]) if dS else None, scale)
    return a(lambda t: t), a(lambda t: t.abs())


SIZES = [  # B, T, Hk, H, Dk, Dv: every head size, lengths around the tiles, shared heads
    (1, 1, 1, 1, 128, 128), (2, 3, 2, 2, 16, 16), (1, 31, 1, 2, 32, 16), (2, 32, 1, 1, 16, 128), (1, 33, 2, 2, 128, 16),
    (1, 63, 1, 3, 64, 64), (2, 64, 2, 4, 128, 64), (1, 65, 1, 1, 64, 128), (1, 127, 3, 3, 32, 32),
    (2, 130, 1, 2, 128, 128), (1, 257, 1, 1, 128, 32), (1, 200, 1, 2, 16, 64),
]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, dt):
    import delta_rule_recurrent_gdn_amd as gdn

    B, T, Hk, H, Dk, Dv = size
    x = make(sum(size), *size, dt)
    d = dev(x)
    (o, S), (mo, mS) = oracle_fwd(x, scale=0.5)
    go, gS = gdn.gdn2_linattn_fwd_chunked(d["q"], d["k"], d["v"], d["ld"], S0=d["S0"], scale=0.5)
    assert go.dtype == dt
    check("o", go, o, mo, T, Dk)
    check("S", gS, S, mS, T, Dk)
    (o, S), (mo, mS) = oracle_fwd(x, S0=False)
    go, gS = gdn.gdn2_linattn_fwd_chunked(d["q"], d["k"], d["v"], d["ld"])
    check("o without S0", go, o, mo, T, Dk)
    check("S without S0", gS, S, mS, T, Dk)
    go2, none = gdn.gdn2_linattn_fwd_chunked(d["q"], d["k"], d["v"], d["ld"], want_final_state=False)
    assert none is None and torch.equal(go, go2)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(size, dt):
    import delta_rule_recurrent_gdn_amd as gdn

    B, T, Hk, H, Dk, Dv = size
    x = make(sum(size) + 1, *size, dt)
    d = dev(x)
    g, m = oracle_bwd(x, scale=0.5)
    got = gdn.gdn2_linattn_bwd_chunked(d["q"], d["k"], d["v"], d["ld"], d["dO"], S0=d["S0"], dS_final=d["dS"], scale=0.5)
    for n in g:
        assert got[n].dtype == (F32 if n == "dS0" else dt)
        check(n, got[n], g[n], m[n], T, max(Dk, Dv))
    g, m = oracle_bwd(x, S0=False, dS=False)
    got = gdn.gdn2_linattn_bwd_chunked(d["q"], d["k"], d["v"], d["ld"], d["dO"], want_dS0=False)
    assert got["dS0"] is None
    for n in ("dq", "dk", "dv"):
        check(n + " without states", got[n], g[n], m[n], T, max(Dk, Dv))


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("decay", [0.0, -1e-4, -3.0, -90.0, -1e30, float("-inf"), 0.01])
def test_decays(decay, dt):
    """No decay, hardly any, strong ones, none of the past left, and growth."""
    import delta_rule_recurrent_gdn_amd as gdn

    x = make(5, 1, 150, 1, 1, 32, 64, dt, decay=decay)
    d = dev(x)
    (o, S), (mo, mS) = oracle_fwd(x)
    go, gS = gdn.gdn2_linattn_fwd_chunked(d["q"], d["k"], d["v"], d["ld"], S0=d["S0"])
    check("o", go, o, mo, 150, 64)
    check("S", gS, S, mS, 150, 64)
    g, m = oracle_bwd(x)
    got = gdn.gdn2_linattn_bwd_chunked(d["q"], d["k"], d["v"], d["ld"], d["dO"], S0=d["S0"], dS_final=d["dS"])
    for n in g:
        check(n, got[n], g[n], m[n], 150, 64)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
def test_pieces_of_a_long_sequence(dt):
    """One head and 1500 tokens: cut into pieces whose states are joined; S_final may be S0's memory."""
    import delta_rule_recurrent_gdn_amd as gdn
    from delta_rule_recurrent_gdn_amd import _lib

    x = make(6, 1, 1500, 1, 1, 32, 32, dt, decay=-2e-3)
    d = dev(x)
    assert gdn.gdn2_linattn_workspace_bytes(0, 1, 1500, 1, 1, 32, 32, dt) > 0
    (o, S), (mo, mS) = oracle_fwd(x)
    go, gS = gdn.gdn2_linattn_fwd_chunked(d["q"], d["k"], d["v"], d["ld"], S0=d["S0"])
    check("o", go, o, mo, 1500, 32)
    check("S", gS, S, mS, 1500, 32)
    g, m = oracle_bwd(x)
    got = gdn.gdn2_linattn_bwd_chunked(d["q"], d["k"], d["v"], d["ld"], d["dO"], S0=d["S0"], dS_final=d["dS"])
    for n in g:
        check(n, got[n], g[n], m[n], 1500, 32)
    lib, s, o2 = _lib.load(), d["S0"].clone(), torch.empty_like(go)
    ws = torch.empty(gdn.gdn2_linattn_workspace_bytes(0, 1, 1500, 1, 1, 32, 32, dt), dtype=torch.uint8, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    st = lib.gdn2_linattn_fwd_chunked(p(d["q"]), p(d["k"]), p(d["v"]), p(d["ld"]), p(s), p(o2), p(s), p(ws), ws.numel(),
                                      1, 1500, 1, 1, 32, 32, 1.0, 0 if dt == F32 else 1,
                                      torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(o2, go) and torch.equal(s, gS)


def test_large_batch_whole_sequences_equal_pieces():
    """The same sequences in a batch that fills the GPU (no pieces) and alone (pieces): the same to rounding."""
    import delta_rule_recurrent_gdn_amd as gdn

    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = (torch.randn(16, 1100, 8, 64, generator=g, device="cuda") for _ in range(3))
    ld = -torch.logspace(-4, 0, 8, device="cuda")
    assert gdn.gdn2_linattn_workspace_bytes(0, 16, 1100, 8, 8, 64, 64, F32) > 0
    big = [t.repeat(4, 1, 1, 1) for t in (q, k, v)]
    assert gdn.gdn2_linattn_workspace_bytes(0, 64, 1100, 8, 8, 64, 64, F32) == 0
    o, S = gdn.gdn2_linattn_fwd_chunked(q, k, v, ld)
    o4, S4 = gdn.gdn2_linattn_fwd_chunked(*big, ld)
    for i in range(4):
        torch.testing.assert_close(o4[16 * i:16 * i + 16], o, rtol=0, atol=2e-5 * float(o.abs().max()))
        torch.testing.assert_close(S4[16 * i:16 * i + 16], S, rtol=0, atol=2e-5 * float(S.abs().max()))
    assert torch.equal(o4[:16], o4[16:32]) and torch.equal(S4[:16], S4[48:])


CU = [[0, 0, 1, 70, 70, 199, 200], [5, 64, 64, 130], [0, 1000], [0, 17, 600, 1000]]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cu", CU, ids=str)
def test_packed(cu, dt):
    """Empty sequences, one token, offsets that start late and end early: rows outside are left as they were."""
    import delta_rule_recurrent_gdn_amd as gdn

    T, N, Hk, H, Dk, Dv = cu[-1] + 9, len(cu) - 1, 1, 2, 64, 32
    x = make(8, 1, T, Hk, H, Dk, Dv, dt)
    r = torch.Generator().manual_seed(9)
    x["S0"], x["dS"] = torch.randn(N, H, Dk, Dv, generator=r), torch.randn(N, H, Dk, Dv, generator=r)
    d = dev(x)
    c = torch.tensor(cu, dtype=torch.int64, device="cuda")
    keep = torch.full((1, T, H, Dv), 7.0, dtype=dt, device="cuda")
    go, gS = gdn.gdn2_linattn_fwd_varlen(d["q"], d["k"], d["v"], d["ld"], c, S0=d["S0"], scale=0.5, o=keep)
    assert go is keep
    gg = gdn.gdn2_linattn_bwd_varlen(d["q"], d["k"], d["v"], d["ld"], d["dO"], c, S0=d["S0"], dS_final=d["dS"], scale=0.5)
    inside = torch.zeros(T, dtype=torch.bool)
    for n in range(N):
        a, b = cu[n], cu[n + 1]
        inside[a:b] = True
        one = {m: x[m][:, a:b] for m in ("q", "k", "v", "dO")} | {m: x[m][n:n + 1] for m in ("S0", "dS")} | {"ld": x["ld"]}
        (o, S), (mo, mS) = oracle_fwd(one, scale=0.5)
        check("S", gS[n:n + 1], S, mS, b - a, Dk)
        g, m = oracle_bwd(one, scale=0.5)
        check("dS0", gg["dS0"][n:n + 1], g["dS0"], m["dS0"], b - a, Dk)
        if b > a:
            check("o", go[:, a:b], o, mo, b - a, Dk)
            for w in ("dq", "dk", "dv"):
                check(w, gg[w][:, a:b], g[w], m[w], b - a, Dk)
    assert (go[:, ~inside] == 7).all()
    for w in ("dq", "dk", "dv"):
        assert (gg[w][:, ~inside] == 0).all()


def test_packed_offsets_out_of_order_stay_inside():
    """Offsets that fall or leave [0, T] are made non-decreasing and clamped, as for the delta rule's packed calls."""
    import delta_rule_recurrent_gdn_amd as gdn

    x = dev(make(10, 1, 100, 1, 1, 32, 32, BF16))
    bad = torch.tensor([-5, 40, 20, 300], dtype=torch.int64, device="cuda")
    good = torch.tensor([0, 40, 40, 100], dtype=torch.int64, device="cuda")
    a = gdn.gdn2_linattn_fwd_varlen(x["q"], x["k"], x["v"], x["ld"], bad)
    b = gdn.gdn2_linattn_fwd_varlen(x["q"], x["k"], x["v"], x["ld"], good)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_many_packed_sequences():
    """150 sequences (more than the planner takes at a time), empty ones among them, against each sequence alone."""
    import delta_rule_recurrent_gdn_amd as gdn

    g = torch.Generator().manual_seed(31)
    lens = torch.randint(0, 40, (150,), generator=g)
    lens[::7] = 0
    lens[64], lens[128] = 400, 300
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    T = int(cu[-1]) + 3
    x = dev(make(32, 1, T, 1, 2, 32, 32, F32))
    S0 = torch.randn(150, 2, 32, 32, device="cuda")
    o, S = gdn.gdn2_linattn_fwd_varlen(x["q"], x["k"], x["v"], x["ld"], cu.cuda(), S0=S0)
    r = gdn.gdn2_linattn_bwd_varlen(x["q"], x["k"], x["v"], x["ld"], x["dO"], cu.cuda(), S0=S0)
    for n in range(150):
        a, b = int(cu[n]), int(cu[n + 1])
        part = [x[m][:, a:b].contiguous() for m in ("q", "k", "v")]
        o1, S1 = gdn.gdn2_linattn_fwd_chunked(*part, x["ld"], S0=S0[n:n + 1])
        r1 = gdn.gdn2_linattn_bwd_chunked(*part, x["ld"], x["dO"][:, a:b].contiguous(), S0=S0[n:n + 1])
        near = lambda s, t: torch.testing.assert_close(s, t, rtol=0, atol=1e-5 * (1 + float(t.abs().max()) if t.numel() else 1))  # noqa: E731
        near(o[:, a:b], o1)
        near(S[n:n + 1], S1)
        near(r["dS0"][n:n + 1], r1["dS0"])
        for m in ("dq", "dk", "dv"):
            near(r[m][:, a:b], r1[m])
    assert (o[:, T - 3:] == 0).all() and all((r[m][:, T - 3:] == 0).all() for m in ("dq", "dk", "dv"))


def test_gradient_of_the_first_state_in_place():
    """dS0 in the memory of S0 or of dS_final."""
    from delta_rule_recurrent_gdn_amd import _lib
    import delta_rule_recurrent_gdn_amd as gdn

    for T in (100, 1500):
        x = dev(make(33, 1, T, 1, 1, 32, 32, BF16))
        want = gdn.gdn2_linattn_bwd_chunked(x["q"], x["k"], x["v"], x["ld"], x["dO"], S0=x["S0"], dS_final=x["dS"])
        p = lambda t: t.data_ptr()  # noqa: E731
        need = gdn.gdn2_linattn_workspace_bytes(_lib.GDN2_OP_BWD, 1, T, 1, 1, 32, 32, BF16)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        for name in ("S0", "dS"):
            s = {n: x[n].clone() for n in ("S0", "dS")}
            d = [torch.empty_like(x[n]) for n in ("q", "k", "v")]
            st = _lib.load().gdn2_linattn_bwd_chunked(
                p(x["q"]), p(x["k"]), p(x["v"]), p(x["ld"]), p(s["S0"]), p(x["dO"]), p(s["dS"]), p(d[0]), p(d[1]), p(d[2]),
                p(s[name]), p(ws), ws.numel(), 1, T, 1, 1, 32, 32, 1.0, _lib.GDN2_BF16,
                torch.cuda.current_stream().cuda_stream)
            assert st == 0 and torch.equal(s[name], want["dS0"])
            for got, n in zip(d, ("dq", "dk", "dv")):
                assert torch.equal(got, want[n])


def test_empty_calls():
    import delta_rule_recurrent_gdn_amd as gdn

    e = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    S0 = torch.randn(2, 3, 16, 32, device="cuda")
    o, S = gdn.gdn2_linattn_fwd_chunked(e(2, 0, 3, 16), e(2, 0, 3, 16), e(2, 0, 3, 32), e(3), S0=S0)
    assert o.shape == (2, 0, 3, 32) and torch.equal(S, S0)
    g = gdn.gdn2_linattn_bwd_chunked(e(2, 0, 3, 16), e(2, 0, 3, 16), e(2, 0, 3, 32), e(3), e(2, 0, 3, 32), dS_final=S0)
    assert torch.equal(g["dS0"], S0)
    o, S = gdn.gdn2_linattn_fwd_chunked(e(0, 5, 3, 16), e(0, 5, 3, 16), e(0, 5, 3, 32), e(3))
    assert o.shape == (0, 5, 3, 32) and S.shape == (0, 3, 16, 32)
    cu = torch.zeros(3, dtype=torch.int64, device="cuda")
    o, S = gdn.gdn2_linattn_fwd_varlen(e(1, 0, 3, 16), e(1, 0, 3, 16), e(1, 0, 3, 32), e(3), cu, S0=S0)
    assert torch.equal(S, S0)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_tokens_stay_in_the_future(bad, dt):
    """Garbage in a token (a padded batch's tail, say) leaves every earlier output and gradient as it was."""
    import delta_rule_recurrent_gdn_amd as gdn

    x = make(11, 1, 100, 1, 1, 64, 64, dt)
    d = dev(x)
    args = lambda y: (y["q"], y["k"], y["v"], y["ld"])  # noqa: E731
    o, _ = gdn.gdn2_linattn_fwd_chunked(*args(d))
    g = gdn.gdn2_linattn_bwd_chunked(*args(d), d["dO"])
    at = 41
    for n in ("q", "k", "v", "dO"):
        y = {m: t.clone() for m, t in d.items()}
        y[n][:, at] = bad
        o2, S2 = gdn.gdn2_linattn_fwd_chunked(*args(y))
        assert torch.equal(o2[:, :at], o[:, :at]), n
        if n in ("k", "v"):
            assert not torch.isfinite(o2[:, at:]).any() and not torch.isfinite(S2).any()
        if n == "q":
            assert not torch.isfinite(o2[:, at]).any() and torch.equal(o2[:, at + 1:], o[:, at + 1:])
        g2 = gdn.gdn2_linattn_bwd_chunked(*args(y), y["dO"])
        assert torch.equal(g2["dq"][:, :at], g["dq"][:, :at]), n
        assert torch.equal(g2["dk"][:, at + 1:], g["dk"][:, at + 1:]), n
        assert torch.equal(g2["dv"][:, at + 1:], g["dv"][:, at + 1:]), n


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("size", [(1, 1, 1, 128, 128), (3, 2, 4, 16, 64), (5, 1, 3, 64, 16), (2, 2, 2, 128, 32)], ids=str)
def test_decode(size, dt):
    import delta_rule_recurrent_gdn_amd as gdn

    B, Hk, H, Dk, Dv = size
    x = make(12, B, 1, Hk, H, Dk, Dv, dt)
    d = dev(x)
    (o, S), (mo, mS) = oracle_fwd(x, scale=0.3)
    s = d["S0"].clone()
    go = gdn.gdn2_linattn_decode_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["ld"], s, scale=0.3)
    check("o", go, o[:, 0], mo[:, 0], 1, Dk)
    check("S", s, S, mS, 1, Dk)
    # a pool: one entry has no slot
    pool = torch.randn(B + 4, H, Dk, Dv, device="cuda")
    slots = torch.randperm(B + 4)[:B].to(torch.int32)
    for b in range(B):
        pool[slots[b]] = d["S0"][b]
    before, lost = pool.clone(), B - 1
    given = slots.clone()
    given[lost] = [-1, B + 4][B % 2]
    out = torch.full((B, H, Dv), 5.0, dtype=dt, device="cuda")
    gdn.gdn2_linattn_decode_step_slots(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["ld"], pool, given.cuda(), scale=0.3,
                                       o=out)
    for b in range(B):
        if b == lost:
            assert (out[b] == 0).all()
        else:
            assert torch.equal(out[b], go[b]) and torch.equal(pool[slots[b]], s[b])
    rest = [j for j in range(B + 4) if j not in [int(slots[b]) for b in range(B) if b != lost]]
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (128, 16)])
def test_decode_many_entries(Dk, Dv):
    """Every element of 4096 states of a full batch: fp32 states to 3 roundings, for each of several steps."""
    import delta_rule_recurrent_gdn_amd as gdn

    g = torch.Generator(device="cuda").manual_seed(30)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ld = -torch.rand(16, generator=g, device="cuda")
    S, S0 = r(256, 16, Dk, Dv), None
    for _ in range(3):
        q, k, v = (r(256, 16, d).bfloat16() for d in (Dk, Dk, Dv))
        S0 = S.double()
        gdn.gdn2_linattn_decode_step(q, k, v, ld, S)
        old, new = ld.double().exp()[None, :, None, None] * S0, k.double()[..., None] * v.double()[:, :, None, :]
        assert ((S - (old + new)).abs() <= 4 * 2.0 ** -24 * (old.abs() + new.abs())).all()


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
def test_state_over_a_long_slow_decay(dt):
    """The state of 8192 tokens walked by one workgroup, hardly decaying: a chunk's sum is added with one rounding (rms
    below 2^-24 / sqrt(3) of the value), so over n chunks the norm of the error stays below sqrt(n) 2^-24."""
    import delta_rule_recurrent_gdn_amd as gdn

    B, T, H, Dk, Dv = 64, 8192, 4, 32, 16
    assert gdn.gdn2_linattn_workspace_bytes(0, B, T, H, H, Dk, Dv, dt) == 0
    g = torch.Generator(device="cuda").manual_seed(40)
    k, v = (torch.randn(B, T, H, d, generator=g, device="cuda").to(dt) for d in (Dk, Dv))
    ld = torch.tensor([0.0, -2.0 ** -15, -2.0 ** -12, -2.0 ** -9], device="cuda")
    _, S = gdn.gdn2_linattn_fwd_chunked(k, k, v, ld)
    weight = torch.exp(ld.double() * torch.arange(T - 1, -1, -1, device="cuda", dtype=torch.float64)[:, None])
    kd, vd = (k.double() * weight[None, :, :, None]).permute(0, 2, 3, 1).contiguous(), v.double().transpose(1, 2).contiguous()
    want = torch.matmul(kd, vd)
    n = T // (64 if dt == BF16 else 32)
    for h in range(H):
        off = (S[:, h].double() - want[:, h]).norm() / want[:, h].norm()
        assert off <= n ** 0.5 * 2.0 ** -24, (h, float(off))


def test_deterministic_and_on_a_side_stream():
    import delta_rule_recurrent_gdn_amd as gdn

    x = dev(make(13, 2, 700, 2, 4, 128, 64, BF16))
    f = lambda: (*gdn.gdn2_linattn_fwd_chunked(x["q"], x["k"], x["v"], x["ld"], S0=x["S0"]),  # noqa: E731
                 *gdn.gdn2_linattn_bwd_chunked(x["q"], x["k"], x["v"], x["ld"], x["dO"], S0=x["S0"]).values())
    a = f()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = f()
    torch.cuda.current_stream().wait_stream(side)
    for s, t in zip(a, b):
        assert torch.equal(s, t)


def test_captured_and_replayed():
    """Forward, backward and a decode step in one graph, replayed with other eager work and new inputs in between."""
    import delta_rule_recurrent_gdn_amd as gdn

    x = dev(make(14, 1, 900, 1, 2, 64, 64, BF16))
    cu = torch.tensor([0, 300, 900], dtype=torch.int64, device="cuda")
    pool = torch.randn(2, 2, 64, 64, device="cuda")

    def step():
        o, S = gdn.gdn2_linattn_fwd_chunked(x["q"], x["k"], x["v"], x["ld"], S0=x["S0"])
        g = gdn.gdn2_linattn_bwd_chunked(x["q"], x["k"], x["v"], x["ld"], x["dO"], S0=x["S0"], dS_final=x["dS"])
        op, Sp = gdn.gdn2_linattn_fwd_varlen(x["q"], x["k"], x["v"], x["ld"], cu)
        d = gdn.gdn2_linattn_decode_step(x["q"][0, :1], x["k"][0, :1], x["v"][0, :1], x["ld"], S)
        return o, S, g["dq"], g["dk"], g["dv"], g["dS0"], op, Sp, d

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(4):
        new = dev(make(20 + seed, 1, 900, 1, 2, 64, 64, BF16))
        for n in x:
            x[n].copy_(new[n])
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        pool.mul_(1.5).sum()
        for s, t in zip(got, step()):
            assert torch.equal(s, t)


def test_states_and_rows_past_32_bits():
    """Rows whose offsets pass 2^31 elements: the last sequence of a large batch equals itself alone."""
    import delta_rule_recurrent_gdn_amd as gdn

    B, T, H, D = 9, 65536, 32, 128  # 2.4 G elements
    q = torch.zeros(B, T, H, D, dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(15)
    q[-1] = torch.randn(T, H, D, generator=g, device="cuda").to(BF16)
    ld = torch.full((H,), -0.05, device="cuda")
    o, S = gdn.gdn2_linattn_fwd_chunked(q, q, q, ld, scale=D ** -0.5)
    tail = q[-1:, -4096:].contiguous()  # decay^(61440) is nothing
    o1, S1 = gdn.gdn2_linattn_fwd_chunked(tail, tail, tail, ld, scale=D ** -0.5)
    assert (o[0, :100] == 0).all() and (o[-2, -100:] == 0).all()
    torch.testing.assert_close(S[-1:], S1, rtol=0, atol=1e-5 * float(S1.abs().max()))
    torch.testing.assert_close(o[-1:, -1000:].float(), o1[:, -1000:].float(), rtol=2 ** -7, atol=1e-2)


@pytest.mark.parametrize("T", [900, 1025])
def test_pieces_at_the_largest_heads(T):
    """bf16 at 128 x 128, cut into pieces: forward, backward and states against the oracle."""
    import delta_rule_recurrent_gdn_amd as gdn

    x = make(50 + T, 1, T, 1, 2, 128, 128, BF16, decay=-4e-3)
    d = dev(x)
    assert gdn.gdn2_linattn_workspace_bytes(0, 1, T, 1, 2, 128, 128, BF16) > 0
    (o, S), (mo, mS) = oracle_fwd(x, scale=0.1)
    go, gS = gdn.gdn2_linattn_fwd_chunked(d["q"], d["k"], d["v"], d["ld"], S0=d["S0"], scale=0.1)
    check("o", go, o, mo, T, 128)
    check("S", gS, S, mS, T, 128)
    g, m = oracle_bwd(x, scale=0.1)
    got = gdn.gdn2_linattn_bwd_chunked(d["q"], d["k"], d["v"], d["ld"], d["dO"], S0=d["S0"], dS_final=d["dS"], scale=0.1)
    for n in g:
        check(n, got[n], g[n], m[n], T, 128)
