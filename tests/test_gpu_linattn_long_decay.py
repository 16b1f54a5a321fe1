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
