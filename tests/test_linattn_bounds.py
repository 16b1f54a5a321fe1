"""The norm-wise bounds of the GPU tests tell fp32 work from work in fewer bits, on a CPU model of the chunked state."""

import numpy as np
import pytest
import torch

import linattn_bounds as L
import oracle.linattn as O

C = 64


def two_terms(x):
    """x as the sum of two bf16 values: its upper 8 bits, and the rest rounded to 8."""
    x = torch.from_numpy(x).float()
    hi = (x.view(torch.int32) & -65536).view(torch.float32)
    return (hi + (x - hi).bfloat16().float()).double().numpy()


def model(k, v, ld, held):
    """S_T of bf16 k, v [T, D]: each chunk's decayed v as `held` keeps it, the chunks' sums in fp32 (one rounding each)."""
    T, g = k.shape[0], np.exp(float(ld))
    S = np.zeros((k.shape[1], v.shape[1]))
    for t in range(0, T, C):
        kc, vc = k[t:t + C], v[t:t + C]
        n = len(kc)
        z = held(vc * g ** np.arange(n - 1, -1, -1.0)[:, None])
        s = (kc.T @ z).astype(np.float32).astype(np.float64)
        S = (S * g ** n + s).astype(np.float32).astype(np.float64)
    return S


@pytest.mark.parametrize("decay", [-1e-3, -0.02, -0.3])
@pytest.mark.parametrize("T,Dk,Dv", [(200, 32, 32), (700, 64, 128)])
def test_bounds_tell_two_bf16_terms_from_fp32(T, Dk, Dv, decay):
    g = torch.Generator().manual_seed(T + Dk)
    k, v = (torch.randn(1, T, 1, d, generator=g).bfloat16() for d in (Dk, Dv))
    ld = torch.tensor([decay])
    want = O.linattn_forward(k, k, v, ld)[1]
    a2 = L.forward_a2(k, k, v, ld)[1]
    run = lambda held: model(k[0, :, 0].double().numpy(), v[0, :, 0].double().numpy(), ld.double(), held)[None, None]  # noqa: E731
    limit = L.bound(L.roundings(0, T, C))
    assert L.off(run(np.float32), want, a2, 1) <= limit / 4
    assert L.off(run(two_terms), want, a2, 1) > limit
