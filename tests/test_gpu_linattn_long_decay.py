"""Linear attention: the decay over many steps does not drift away from exp(log_decay).

An fp32 factor is off by up to 2^-25 of the decay, the same way at every step. What a kernel multiplies a state with must
make up for that, so that what is left is the states' own roundings: these go either way, so n of them are worth
sqrt(n) 2^-24 in the norm at most, and next to nothing in the mean over many elements.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def badly_rounded(lo, hi, n, steps):
    """n log_decays (fp32) between lo and hi, those whose decay over `steps` tokens is the furthest from an fp32 value."""
    c = np.linspace(lo, hi, 64 * n).astype(np.float32).reshape(n, 64)
    g = np.exp(c.astype(np.float64) * steps)
    off = np.abs(g.astype(np.float32) - g) / g
    return torch.from_numpy(c[np.arange(n), off.argmax(1)].copy())


def test_decode_over_thousands_of_steps():
    import delta_rule_recurrent_gdn_amd as gdn

    B, H, Dk, Dv, steps = 4, 8, 64, 32, 2048
    ld = badly_rounded(-2.0 ** -15, -2.0 ** -9, H, 1)
    S0 = torch.randn(B, H, Dk, Dv, generator=torch.Generator().manual_seed(1))
    S, d = S0.cuda(), ld.cuda()
    zero = torch.zeros(B, H, Dk, device="cuda")
    q, v, o = zero.clone(), zero[..., :Dv].contiguous(), torch.empty(B, H, Dv, device="cuda")
    for _ in range(steps):
        gdn.gdn2_linattn_decode_step(q, zero, v, d, S, o=o)
    want = torch.exp(ld.double() * steps)[None, :, None, None] * S0.double()
    for h in range(H):
        off = (S[:, h].cpu().double() - want[:, h]).norm() / want[:, h].norm()
        assert off <= steps ** 0.5 * 2.0 ** -24, (h, float(off * 2 ** 24))


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("chunks,enters", [(7, 0), (8, 7), (8, 6), (15, 13), (16, 0)])
def test_forward_over_a_few_chunks(chunks, enters, dt):
    """One contribution alone: the first state (enters = 0), or the last token of chunk `enters` - 1, whose own factor is
    1; it decays over the chunks after it. The mean of the relative errors over all elements, where the n + 1 roundings of
    at most 2^-24 are worth 4 sqrt((n + 1) / elements) of that (their spread is at most 1 / sqrt(3) of it)."""
    import delta_rule_recurrent_gdn_amd as gdn

    B, H, Dk, Dv = 64, 4, 32, 16
    C = 64 if dt == BF16 else 32
    T = chunks * C
    assert gdn.gdn2_linattn_workspace_bytes(0, B, T, H, H, Dk, Dv, dt) == 0  # whole sequences
    ld = badly_rounded(np.log(0.1) / C, np.log(0.9) / C, H, C)
    g = torch.Generator().manual_seed(chunks + enters)
    q, k = torch.zeros(B, T, H, Dk), torch.zeros(B, T, H, Dk)
    v = torch.zeros(B, T, H, Dv)
    S0 = None
    if enters == 0:
        S0 = torch.randn(B, H, Dk, Dv, generator=g)
        want, n = S0.double(), chunks
    else:
        at = enters * C - 1
        k[:, at] = torch.randn(B, H, Dk, generator=g).to(dt).float()
        v[:, at] = torch.randn(B, H, Dv, generator=g).to(dt).float()
        want, n = k[:, at].double()[..., :, None] * v[:, at].double()[..., None, :], chunks - enters
    want = torch.exp(ld.double() * n * C)[None, :, None, None] * want
    _, S = gdn.gdn2_linattn_fwd_chunked(*(t.to(dt).cuda() for t in (q, k, v)), ld.cuda(),
                                        S0=None if S0 is None else S0.cuda())
    for h in range(H):
        rel = (S[:, h].cpu().double() / want[:, h] - 1).flatten()
        assert abs(rel.mean()) <= 4 * ((n + 1) / rel.numel()) ** 0.5 * 2.0 ** -24, (h, float(rel.mean() * 2 ** 24))
        assert rel.abs().max() <= (n + 1) * 2.0 ** -24, (h, float(rel.abs().max() * 2 ** 24))


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
def test_growth_after_padding(dt):
    """log_decay = 0.4 over 1500 tokens, of which all but the last 50 are zeros: nothing grows past e^20, though the
    growth over one of the pieces that the sequence is cut into is no fp32 number."""
    import delta_rule_recurrent_gdn_amd as gdn

    import oracle.linattn as O

    T, D = 1500, 32
    assert gdn.gdn2_linattn_workspace_bytes(0, 1, T, 1, 1, D, D, dt) > 0
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(1, T, 1, D, generator=g).to(dt) for _ in range(3))
    k[:, :T - 50] = 0
    ld = torch.tensor([0.4])
    (o, S), (mo, mS) = (O.linattn_forward(f(q), f(k), f(v), ld) for f in (lambda t: t, torch.abs))
    got, last = gdn.gdn2_linattn_fwd_chunked(q.cuda(), k.cuda(), v.cuda(), ld.cuda())
    for name, x, ref, mag in (("o", got, o, mo), ("S", last, S, mS)):
        x = x.cpu().double().numpy()
        tol = (2.0 ** -8 if name == "o" and dt == BF16 else 0) * np.abs(ref) + (4 * (50 + D) + 64) * 2.0 ** -24 * mag
        assert np.isfinite(x).all() and (np.abs(x - ref) <= tol).all(), name
    # the reversed recurrences: zeros at the end of dO
    dO = torch.randn(1, T, 1, D, generator=g).to(dt)
    dO[:, 50:] = 0
    want, mag = (O.linattn_backward(f(q), f(k), f(v), ld, f(dO)) for f in (lambda t: t, torch.abs))
    r = gdn.gdn2_linattn_bwd_chunked(q.cuda(), k.cuda(), v.cuda(), ld.cuda(), dO.cuda())
    for n in ("dk", "dv", "dS0"):
        x = r[n].cpu().double().numpy()
        tol = (2.0 ** -8 if n != "dS0" and dt == BF16 else 0) * np.abs(want[n]) + (4 * (50 + D) + 64) * 2.0 ** -24 * mag[n]
        assert np.isfinite(x).all() and (np.abs(x - want[n]) <= tol).all(), n
