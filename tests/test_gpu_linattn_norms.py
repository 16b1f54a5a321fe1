"""fp32 outputs of the linear attention, norm-wise: all of them with fp32 inputs, the states' with bf16 ones.

The bounds are linattn_bounds': what fp32 roundings come to in the norm, some 1e-6, where the element-wise ones of the
other tests count every rounding at its worst.
"""

import pytest
import torch

import linattn_bounds as L
import oracle.linattn as O

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
SIZES = [  # B, T, Hk, H, Dk, Dv, cut into pieces
    (1, 700, 2, 2, 64, 64, True), (1, 700, 1, 2, 64, 128, True), (1, 900, 1, 1, 128, 128, True),
    (16, 200, 16, 16, 32, 32, False), (32, 150, 4, 8, 64, 32, False), (16, 130, 16, 16, 128, 16, False),
]


def make(size, dt):
    B, T, Hk, H, Dk, Dv, pieces = size
    g = torch.Generator().manual_seed(sum(size))
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = {"q": r(B, T, Hk, Dk), "k": r(B, T, Hk, Dk), "v": r(B, T, H, Dv), "dO": r(B, T, H, Dv)}
    x = {n: t.to(dt) for n, t in x.items()}
    x.update(S0=r(B, H, Dk, Dv), dS=r(B, H, Dk, Dv), ld=-torch.rand(H, generator=g) ** 4)
    return x


def within(name, got, want, a2, n, axis):
    o = L.off(got.detach().cpu().double().numpy(), want, a2, axis)
    assert o <= L.bound(n), (name, o / L.bound(n))


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, dt):
    import delta_rule_recurrent_gdn_amd as gdn

    B, T, Hk, H, Dk, Dv, pieces = size
    C = 64 if dt == BF16 else 32
    assert (gdn.gdn2_linattn_workspace_bytes(0, B, T, Hk, H, Dk, Dv, dt) > 0) == pieces
    x = make(size, dt)
    a = [x[n] for n in ("q", "k", "v", "ld", "S0")]
    o, S = O.linattn_forward(*a)
    ao, aS = L.forward_a2(*a)
    go, gS = gdn.gdn2_linattn_fwd_chunked(*(t.cuda() for t in a[:4]), S0=x["S0"].cuda())
    within("S", gS, S, aS, L.roundings(0, T, C), 1)
    if dt == F32:
        within("o", go, o, ao, L.roundings(Dk, T, C), 2)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(size, dt):
    import delta_rule_recurrent_gdn_amd as gdn

    B, T, Hk, H, Dk, Dv, pieces = size
    C = 64 if dt == BF16 else 32
    x = make(size, dt)
    a = [x[n] for n in ("q", "k", "v", "ld", "dO", "S0", "dS")]
    want, a2 = O.linattn_backward(*a), L.backward_a2(*a)
    got = gdn.gdn2_linattn_bwd_chunked(*(t.cuda() for t in a[:5]), S0=x["S0"].cuda(), dS_final=x["dS"].cuda())
    within("dS0", got["dS0"], want["dS0"], a2["dS0"], L.roundings(0, T, C), 1)
    if dt == F32:
        for n, channels in (("dq", Dv), ("dk", Dv), ("dv", Dk)):
            within(n, got[n], want[n], a2[n], L.roundings(channels, T, C) + H // Hk, 2)


def test_packed():
    import delta_rule_recurrent_gdn_amd as gdn

    cu, H, Dk, Dv = [3, 3, 90, 700, 701, 1150], 2, 64, 32
    N, T = len(cu) - 1, 1160
    x = make((1, T, 1, H, Dk, Dv, True), F32)
    g = torch.Generator().manual_seed(3)
    S0, dS = torch.randn(N, H, Dk, Dv, generator=g), torch.randn(N, H, Dk, Dv, generator=g)
    d = [x[n].cuda() for n in ("q", "k", "v", "ld")]
    c = torch.tensor(cu, device="cuda")
    o, S = gdn.gdn2_linattn_fwd_varlen(*d, c, S0=S0.cuda())
    r = gdn.gdn2_linattn_bwd_varlen(*d, x["dO"].cuda(), c, S0=S0.cuda(), dS_final=dS.cuda())
    for n in range(N):
        at, len_ = slice(cu[n], cu[n + 1]), cu[n + 1] - cu[n]
        a = [x["q"][:, at], x["k"][:, at], x["v"][:, at], x["ld"]]
        more, s = x["dO"][:, at], S0[n:n + 1]
        (wo, wS), (ao, aS) = O.linattn_forward(*a, s), L.forward_a2(*a, s)
        want, a2 = O.linattn_backward(*a, more, s, dS[n:n + 1]), L.backward_a2(*a, more, s, dS[n:n + 1])
        within("S", S[n:n + 1], wS, aS, L.roundings(0, len_, 32), 1)
        within("dS0", r["dS0"][n:n + 1], want["dS0"], a2["dS0"], L.roundings(0, len_, 32), 1)
        if len_:
            within("o", o[:, at], wo, ao, L.roundings(Dk, len_, 32), 2)
            for m, channels in (("dq", Dv), ("dk", Dv), ("dv", Dk)):
                within(m, r[m][:, at], want[m], a2[m], L.roundings(channels, len_, 32) + H, 2)
