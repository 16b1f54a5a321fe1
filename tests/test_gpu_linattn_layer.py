"""The operators as a layer uses them: norms and rotation from the fused projection, then the mixers."""

import numpy as np
import pytest
import torch

import oracle.linattn as O

pytestmark = pytest.mark.gpu


def _projection(seed, B, T, H, Hk, D):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, T, (H + Hk) * D + H * D, generator=g)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_prefill_then_decode_is_the_whole_forward(dt):
    """A prompt's prefill and then single tokens give what one forward over all tokens gives."""
    import delta_rule_recurrent_gdn_amd as gdn

    B, T, P, H, Hk, D = 2, 83, 75, 4, 2, 64
    x = _projection(1, B, T, H, Hk, D).to(dt).cuda()
    w = torch.linspace(0.5, 1.5, D, device="cuda")
    f = (10000.0 ** (-torch.arange(16) / 16)).cuda()
    ld = -torch.tensor([0.5, 0.1, 0.01, 0.001], device="cuda")

    def qkv(a, b):
        r = x[:, a:b]
        q, k = r[..., :H * D].unflatten(-1, (H, D)), r[..., H * D:(H + Hk) * D].unflatten(-1, (Hk, D))
        pos = torch.arange(a, b, device="cuda")
        if b - a < T:  # a slice of the batch's rows is not evenly spaced: a prompt's rows of its own
            q, k = q.contiguous(), k.contiguous()
        q, k = gdn.gdn2_qk_norm_rope_fwd(q, k, pos, f, q_weight=w, k_weight=w)
        q = q[:, :, :Hk].contiguous()  # as many query heads as key heads
        return q, k, r[..., (H + Hk) * D:].unflatten(-1, (H, D)).contiguous()

    whole, last = gdn.gdn2_linattn_fwd_chunked(*qkv(0, T), ld, scale=D ** -0.5)
    o, S = gdn.gdn2_linattn_fwd_chunked(*qkv(0, P), ld, scale=D ** -0.5)
    assert torch.equal(o, whole[:, :P])
    pool = torch.zeros(5, H, D, D, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pool[slots.long()] = S
    outs = [o]
    for t in range(P, T):
        q, k, v = (y[:, 0].contiguous() for y in qkv(t, t + 1))
        outs.append(gdn.gdn2_linattn_decode_step_slots(q, k, v, ld, pool, slots, scale=D ** -0.5)[:, None])
    got = torch.cat(outs, 1).double().cpu().numpy()
    q, k, v = (y.double().cpu().numpy() for y in qkv(0, T))
    ref, end = O.linattn_forward(q, k, v, ld, None, D ** -0.5)
    mag, _ = O.linattn_forward(abs(q), abs(k), abs(v), ld, None, D ** -0.5)
    unit = 2.0 ** -8 * np.abs(ref) + 2.0 ** -14 * mag if dt == torch.bfloat16 else 2.0 ** -14 * mag
    assert (np.abs(got - ref) <= unit).all()
    torch.testing.assert_close(pool[slots.long()], last, rtol=0, atol=1e-4 * float(last.abs().max()))
    assert (pool[[0, 2, 4]] == 0).all()


def test_gradients_through_the_layer_against_differences():
    """fp32: the chain of both backward calls against differences of the float64 oracles along random directions."""
    import delta_rule_recurrent_gdn_amd as gdn

    B, T, H, D = 1, 70, 2, 32
    x = _projection(2, B, T, H, H, D)
    w = torch.linspace(0.5, 1.5, D)
    f = 10000.0 ** (-torch.arange(8) / 8)
    ld = -torch.tensor([0.2, 0.01])
    pos = torch.arange(T)
    dO = torch.randn(B, T, H, D, generator=torch.Generator().manual_seed(3))

    def loss(x, w):
        q, k, v = (x[..., i * H * D:(i + 1) * H * D].reshape(B, T, H, D) for i in range(3))
        q = O.qk_norm_rope(q, pos[None].numpy(), f, w, eps=1e-6)
        k = O.qk_norm_rope(k, pos[None].numpy(), f, None, eps=1e-6, l2=False)
        return (O.linattn_forward(q, k, v, ld, None, 0.2)[0] * dO.double().numpy()).sum()

    d = x.cuda()
    q, k, v = (d[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3))
    yq, yk = gdn.gdn2_qk_norm_rope_fwd(q, k, pos.cuda(), f.cuda(), q_weight=w.cuda())
    g = gdn.gdn2_linattn_bwd_chunked(yq, yk, v.contiguous(), ld.cuda(), dO.cuda(), scale=0.2)
    dx = torch.empty_like(d)
    rows = [dx[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3)]
    n = gdn.gdn2_qk_norm_rope_bwd(g["dq"], g["dk"], q, k, pos.cuda(), f.cuda(), q_weight=w.cuda(), dq=rows[0], dk=rows[1])
    rows[2].copy_(g["dv"])
    r = np.random.default_rng(4)
    x64, w64 = x.double().numpy(), w.double().numpy()
    for _ in range(4):
        ex, ew = r.standard_normal(x64.shape), r.standard_normal(D)
        diff = (loss(x64 + 1e-5 * ex, w64 + 1e-5 * ew) - loss(x64 - 1e-5 * ex, w64 - 1e-5 * ew)) / 2e-5
        a, b = dx.double().cpu().numpy() * ex, n["dq_weight"].double().cpu().numpy() * ew
        # fp32 chains of some T + 3 D sums: 2^-15 of the terms' magnitude, which random signs keep far from
        assert abs(a.sum() + b.sum() - diff) <= 2.0 ** -15 * np.sqrt((a ** 2).sum() + (b ** 2).sum()) * 8 + 1e-6 * abs(diff)


def test_in_front_of_the_delta_rule():
    """L2 norms and rotation in front of the gated delta rule, and back through both."""
    import delta_rule_recurrent_gdn_amd as gdn
    import oracle

    B, T, H, D = 1, 40, 2, 32
    x = _projection(5, B, T, H, H, D)
    f = 10000.0 ** (-torch.arange(16) / 16)
    q, k, v = (x.cuda()[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3))
    yq, yk = gdn.gdn2_qk_norm_rope_fwd(q, k, None, f.cuda(), l2=True, q_scale=D ** -0.5)
    v = v.contiguous()
    g = torch.Generator().manual_seed(6)
    b, w = torch.rand(B, T, H, D, generator=g).cuda(), torch.rand(B, T, H, D, generator=g).cuda()
    la = -torch.rand(B, T, H, D, generator=g).cuda()
    dO = torch.randn(B, T, H, D, generator=g).cuda()
    o, S, _ = gdn.gdn2_fwd_chunked(yq, yk, v, la, b, w, chunk=32)
    h = gdn.gdn2_bwd_chunked(yq, yk, v, la, b, w, dO, chunk=32)
    n = gdn.gdn2_qk_norm_rope_bwd(h["dq"], h["dk"], q, k, None, f.cuda(), l2=True, q_scale=D ** -0.5)
    pos = np.arange(T)[None]
    x64 = [t.double().cpu().numpy() for t in (q, k, v, la, b, w)]
    rq = O.qk_norm_rope(x64[0], pos, f, l2=True, scale=D ** -0.5)
    rk = O.qk_norm_rope(x64[1], pos, f, l2=True)
    ref, _ = oracle.forward(rq, rk, *x64[2:], None)
    rms = lambda t: np.sqrt((np.asarray(t) ** 2).mean())  # noqa: E731
    assert np.abs(o.double().cpu().numpy() - ref).max() <= 1e-4 * rms(ref)
    back = oracle.backward(rq, rk, *x64[2:], None, dO.double().cpu().numpy())
    dq, _ = O.qk_norm_rope_backward(back["dq"], x64[0], pos, f, l2=True, scale=D ** -0.5)
    dk, _ = O.qk_norm_rope_backward(back["dk"], x64[1], pos, f, l2=True)
    for got, want in ((n["dq"], dq), (n["dk"], dk)):
        assert np.abs(got.double().cpu().numpy() - want).max() <= 1e-4 * rms(want)
