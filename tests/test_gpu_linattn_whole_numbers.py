"""Linear attention of whole numbers without decay: no rounding but the output's.

Every product and sum is a whole number below 2^24 in magnitude (asserted from the sums of the terms' magnitudes), so
fp32 work is exact in any order: a state is the exact one, and an output is the exact value rounded once, bit for bit.
Work that holds scores or states in fewer bits on the way misses the rounding of some outputs.
"""

import numpy as np
import pytest
import torch

import oracle.linattn as O

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def whole(g, top, *shape):
    return torch.randint(-top, top + 1, shape, generator=g).float()


def one_channel(g, *shape):
    """Rows of +1 or -1 in one channel."""
    x = torch.zeros(*shape)
    at = torch.randint(0, shape[-1], shape[:-1], generator=g)[..., None]
    return x.scatter_(-1, at, 2.0 * torch.randint(0, 2, at.shape, generator=g) - 1)


def few(g, *shape):
    """Tokens of -1, 0 and 1, one in 64 (of long sequences 256)."""
    return whole(g, 1, *shape) * (torch.rand(*shape[:2], 1, 1, generator=g) < (1 / 64 if shape[1] <= 256 else 1 / 256))


def equal(name, got, exact, mag):
    assert np.max(mag) < 2 ** 24, name
    want = torch.from_numpy(exact).float().to(got.dtype)
    off = (got.cpu() != want).sum()
    assert off == 0, (name, int(off), want.numel())


# which operand rows are read against the state (x), which build it (y, z), of the forward and of each gradient
ROLES = {"o": ("q", "k", "v"), "dq": ("dO", "v", "k"), "dk": ("v", "dO", "q"), "dv": ("k", "q", "dO")}
SIZES = [  # B, T, Hk, H, Dk, Dv
    (2, 200, 2, 2, 128, 128), (1, 90, 1, 2, 64, 64), (3, 65, 1, 1, 16, 128), (1, 130, 2, 4, 128, 32), (1, 40, 1, 1, 32, 16),
    (1, 700, 1, 1, 64, 128),  # few heads: cut into pieces
]


def make(seed, size, role, wide):
    """wide "state": states past 16 bits, read through one channel; "scores": scores past 16 bits, few of them used."""
    B, T, Hk, H, Dk, Dv = size
    g = torch.Generator().manual_seed(seed)
    shapes = {"q": (B, T, Hk, Dk), "k": (B, T, Hk, Dk), "v": (B, T, H, Dv), "dO": (B, T, H, Dv)}
    x, y, z = ROLES[role]
    d = {n: whole(g, 3, *s) for n, s in shapes.items()}
    if wide == "state":
        d[x], d[y], d[z] = one_channel(g, *shapes[x]), whole(g, 63, *shapes[y]), whole(g, 63, *shapes[z])
        S = whole(g, 2 ** 20, B, H, Dk, Dv)
    else:
        d[x], d[y], d[z] = whole(g, 255, *shapes[x]), whole(g, 255, *shapes[y]), few(g, *shapes[z])
        S = torch.zeros(B, H, Dk, Dv)
    if T > 256 and wide == "state":  # sums over more tokens
        d[y], d[z] = whole(g, 31, *shapes[y]), whole(g, 31, *shapes[z])
    return d, S


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("wide", ["state", "scores"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, wide, dt):
    import delta_rule_recurrent_gdn_amd as gdn

    d, S0 = make(sum(size), size, "o", wide)
    ld = torch.zeros(size[3])
    run = lambda f: O.linattn_forward(f(d["q"]), f(d["k"]), f(d["v"]), ld, f(S0))  # noqa: E731
    (o, S), (mo, mS) = run(lambda t: t), run(torch.abs)
    got, last = gdn.gdn2_linattn_fwd_chunked(*(d[n].to(dt).cuda() for n in "qkv"), ld.cuda(), S0=S0.cuda())
    equal("o", got, o, mo)
    equal("S", last, S, mS)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("wide", ["state", "scores"])
@pytest.mark.parametrize("role", ["dq", "dk", "dv"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(size, role, wide, dt):
    import delta_rule_recurrent_gdn_amd as gdn

    d, S = make(sum(size) + 1, size, role, wide)
    ld = torch.zeros(size[3])
    zero = torch.zeros_like(S)
    S0, dS = (S, zero) if role == "dq" else (zero, S)
    run = lambda f: O.linattn_backward(*(f(d[n]) for n in "qkv"), ld, f(d["dO"]), f(S0), f(dS))  # noqa: E731
    g, m = run(lambda t: t), run(torch.abs)
    for want_dS0 in (True, False):
        got = gdn.gdn2_linattn_bwd_chunked(*(d[n].to(dt).cuda() for n in "qkv"), ld.cuda(), d["dO"].to(dt).cuda(),
                                           S0=S0.cuda(), dS_final=dS.cuda(), want_dS0=want_dS0)
        equal(role, got[role], g[role], m[role])
        if want_dS0 and m["dS0"].max() < 2 ** 24:
            equal("dS0", got["dS0"], g["dS0"], m["dS0"])


@pytest.mark.parametrize("size", [(2, 300, 2, 4, 64, 64), (1, 700, 1, 1, 64, 128), (8, 130, 4, 4, 128, 128)], ids=str)
def test_gradients_do_not_depend_on_the_first_states(size):
    """dq, dk, dv are the same bits whether the gradient of the first state is asked for or not."""
    import delta_rule_recurrent_gdn_amd as gdn

    B, T, Hk, H, Dk, Dv = size
    g = torch.Generator().manual_seed(sum(size))
    q, k, v, dO = (torch.randn(B, T, n, d, generator=g).to(BF16).cuda() for n, d in ((Hk, Dk), (Hk, Dk), (H, Dv), (H, Dv)))
    dS = torch.randn(B, H, Dk, Dv, generator=g).cuda()
    ld = -torch.logspace(-4, 0, H).cuda()
    a = gdn.gdn2_linattn_bwd_chunked(q, k, v, ld, dO, dS_final=dS, want_dS0=True)
    b = gdn.gdn2_linattn_bwd_chunked(q, k, v, ld, dO, dS_final=dS, want_dS0=False)
    for n in ("dq", "dk", "dv"):
        assert torch.equal(a[n], b[n]), n
