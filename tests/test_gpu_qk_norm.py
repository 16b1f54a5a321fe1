"""Head norms of q and k with the rotation on the GPU, against the float64 oracle.

Tolerances, element by element. fp32: 2^-24 for each of the at most D + 64 roundings in a row, of the pair's magnitude
(two channels mix); bf16 outputs one more rounding, 2^-8 of the result.
"""

import numpy as np
import pytest
import torch

import oracle.linattn as O

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make(seed, lead, Hq, Hk, D, rot, dt, far=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = {"qkv": r(*lead, (Hq + 2 * Hk) * D).to(dt), "dq": r(*lead, Hq, D).to(dt), "dk": r(*lead, Hk, D).to(dt),
         "wq": 1 + 0.3 * r(D), "wk": 1 + 0.3 * r(D), "f": 10000.0 ** (-torch.arange(rot // 2) / max(1, rot // 2)),
         "pos": torch.randint(0, 1000, lead, generator=g) + far}
    return x


def cut(x, Hq, Hk, D):
    return x["qkv"][..., :Hq * D].unflatten(-1, (Hq, D)), x["qkv"][..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))


def near(name, got, ref, mag, D):
    got64 = got.detach().cpu().double().numpy()
    assert got64.shape == ref.shape
    tol = (D + 64) * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(ref) if got.dtype == BF16 else 0)
    off = np.abs(got64 - ref) - tol
    assert np.isfinite(got64).all() and (off <= 1e-30).all(), (name, float(off.max()))


def magnitude(x, w, eps, l2):
    """The largest magnitude of a row's normed channels: what a rotation may mix in."""
    x = np.abs(x.double().numpy())
    m = (x * x).sum(-1, keepdims=True) / (1 if l2 else x.shape[-1])
    y = x / np.sqrt(m + eps) * (1 if w is None else np.abs(w.double().numpy()))
    return y.max(-1, keepdims=True)


CASES = [  # leading sizes, Hq, Hk, D, rot
    ((1, 1), 1, 1, 128, 128), ((2, 5), 4, 2, 128, 64), ((3, 7), 5, 3, 64, 64), ((1, 33), 16, 16, 128, 128),
    ((37,), 3, 1, 32, 16), ((2, 1), 7, 2, 16, 16), ((4, 3), 9, 9, 64, 0), ((1, 300), 2, 1, 128, 16), ((2, 9), 1, 17, 32, 32),
]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("l2", [False, True], ids=["rms", "l2"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward(case, l2, interleaved, dt):
    import delta_rule_recurrent_gdn_amd as gdn

    lead, Hq, Hk, D, rot = case
    x = make(D + rot + Hq, lead, Hq, Hk, D, rot, dt)
    d = {n: t.cuda() for n, t in x.items()}
    weights = not l2
    wq, wk = (x["wq"], x["wk"]) if weights else (None, None)
    kw = dict(eps=1e-3, l2=l2, interleaved=interleaved)
    gkw = dict(kw, q_weight=d["wq"] if weights else None, k_weight=d["wk"] if weights else None, q_scale=0.25)
    q, k = cut(x, Hq, Hk, D)
    gq, gk = cut(d, Hq, Hk, D)
    f = d["f"].float() if rot else None
    yq, yk = gdn.gdn2_qk_norm_rope_fwd(gq, gk, d["pos"], f, **gkw)
    assert yq.dtype == dt and yq.is_contiguous()
    pos, fr = x["pos"].numpy(), x["f"].float()
    for n, got, t, w, s in (("q", yq, q, wq, 0.25), ("k", yk, k, wk, 1.0)):
        ref = O.qk_norm_rope(t, pos, fr, w, scale=s, **kw)
        near(n, got, ref, s * magnitude(t, w, 1e-3, l2), D)
    g = gdn.gdn2_qk_norm_rope_bwd(d["dq"], d["dk"], gq, gk, d["pos"], f, **gkw)
    for n, t, dy, w, s in (("q", q, x["dq"], wq, 0.25), ("k", k, x["dk"], wk, 1.0)):
        dx, dw = O.qk_norm_rope_backward(dy, t, pos, fr, w, scale=s, **kw)
        t64, dy64 = np.abs(t.double().numpy()), np.abs(dy.double().numpy())
        m = (t64 ** 2).sum(-1, keepdims=True) / (1 if l2 else D) + 1e-3
        h = s * 2 * dy64.max(-1, keepdims=True) * (1 if w is None else np.abs(w.numpy()))
        mag = h / np.sqrt(m) + t64 * (h * t64).sum(-1, keepdims=True) / ((1 if l2 else D) * m ** 1.5)
        near("d" + n, g["d" + n], dx, mag, D)
        if w is None:
            assert g[f"d{n}_weight"] is None
        else:
            rows = t64.reshape(-1, D).shape[0]
            terms = (s * 2 * dy64.max(-1, keepdims=True) * t64 / np.sqrt(m)).reshape(-1, D).sum(0)
            got = g[f"d{n}_weight"].cpu().double().numpy()
            assert (np.abs(got - dw) <= (rows + D + 64) * 2.0 ** -24 * terms).all()


def test_far_positions():
    """Angles of positions near 2^31 and below zero: reduced in fp64, so as exact as the nearest ones'."""
    import delta_rule_recurrent_gdn_amd as gdn

    x = make(1, (2, 6), 2, 1, 64, 64, F32)
    x["pos"] = torch.tensor([[0, 1, 2 ** 20 + 1, 2 ** 31 + 7, 2 ** 30 + 3, -5], [10 ** 6, 10 ** 7, 10 ** 8, 10 ** 9, 3, -2 ** 31]])
    q, k = cut({"qkv": x["qkv"].cuda()}, 2, 1, 64)
    y, _ = gdn.gdn2_qk_norm_rope_fwd(q, k, x["pos"].cuda(), x["f"].float().cuda())
    t = cut(x, 2, 1, 64)[0]
    # the fp64 angles (here and in the oracle) are off by at most 2^-51 of 2^31: less than one fp32 rounding
    near("q", y, O.qk_norm_rope(t, x["pos"].numpy(), x["f"].float()), magnitude(t, None, 1e-6, False), 64)


def test_positions_shared_and_absent():
    import delta_rule_recurrent_gdn_amd as gdn

    x = {n: t.cuda() for n, t in make(2, (3, 11), 2, 2, 32, 32, BF16).items()}
    q, k = cut(x, 2, 2, 32)
    f = x["f"].float()
    t = torch.arange(11, device="cuda")
    a = gdn.gdn2_qk_norm_rope_fwd(q, k, t.expand(3, 11).contiguous(), f)
    for pos in (t, None):
        b = gdn.gdn2_qk_norm_rope_fwd(q, k, pos, f)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_q_alone_in_place_and_into_rows():
    import delta_rule_recurrent_gdn_amd as gdn

    x = {n: t.cuda() for n, t in make(3, (2, 40), 6, 2, 128, 128, BF16).items()}
    q, k = cut(x, 6, 2, 128)
    f = x["f"].float()
    yq, yk = gdn.gdn2_qk_norm_rope_fwd(q, k, x["pos"], f, q_weight=x["wq"])
    only, none = gdn.gdn2_qk_norm_rope_fwd(q, None, x["pos"], f, q_weight=x["wq"])
    assert none is None and torch.equal(only, yq)
    rows = x["qkv"].clone()
    rq, rk = cut({"qkv": rows}, 6, 2, 128)
    out = gdn.gdn2_qk_norm_rope_fwd(rq, rk, x["pos"], f, q_weight=x["wq"], q_out=rq, k_out=rk)
    assert out[0] is rq and torch.equal(rq, yq) and torch.equal(rk, yk)
    assert torch.equal(rows[..., 8 * 128:], x["qkv"][..., 8 * 128:])  # v's part of the rows is untouched
    g = gdn.gdn2_qk_norm_rope_bwd(x["dq"], x["dk"], q, k, x["pos"], f, q_weight=x["wq"])
    assert g["dk_weight"] is None
    drows = torch.full_like(x["qkv"], 3.0)
    dq, dk = cut({"qkv": drows}, 6, 2, 128)
    h = gdn.gdn2_qk_norm_rope_bwd(x["dq"], x["dk"], q, k, x["pos"], f, q_weight=x["wq"], dq=dq, dk=dk)
    assert torch.equal(dq, g["dq"]) and torch.equal(dk, g["dk"]) and torch.equal(h["dq_weight"], g["dq_weight"])
    assert (drows[..., 8 * 128:] == 3).all()
    one = gdn.gdn2_qk_norm_rope_bwd(x["dq"], None, q, None, x["pos"], f, q_weight=x["wq"])
    assert one["dk"] is None and torch.equal(one["dq"], g["dq"])


def test_fp32_gradients_of_bf16_inputs():
    """The delta rule's backward gives fp32 gradients of bf16 q and k: taken as they are."""
    import delta_rule_recurrent_gdn_amd as gdn

    x = make(4, (1, 50), 3, 3, 64, 32, BF16)
    dy = torch.randn(1, 50, 3, 64, generator=torch.Generator().manual_seed(5))
    q, k = cut({"qkv": x["qkv"].cuda()}, 3, 3, 64)
    g = gdn.gdn2_qk_norm_rope_bwd(dy.cuda(), dy.cuda(), q, k, x["pos"].cuda(), x["f"].float().cuda(), q_weight=x["wq"].cuda())
    t = cut(x, 3, 3, 64)[0]
    dx, dw = O.qk_norm_rope_backward(dy, t, x["pos"].numpy(), x["f"].float(), x["wq"])
    assert g["dq"].dtype == BF16
    r = 1 / np.sqrt((t.double().numpy() ** 2).mean(-1, keepdims=True) + 1e-6)
    mag = 2 * r * 2 * np.abs(dy.numpy()).max() * np.abs(x["wq"].numpy()).max() * (1 + np.abs(t.double().numpy()))
    near("dq", g["dq"], dx, mag, 64)


def test_no_tokens():
    import delta_rule_recurrent_gdn_amd as gdn

    e = torch.zeros(2, 0, 3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    q, k = gdn.gdn2_qk_norm_rope_fwd(e, e)
    assert q.shape == e.shape
    g = gdn.gdn2_qk_norm_rope_bwd(e, e, e, e, q_weight=w)
    assert (g["dq_weight"] == 0).all()


def test_refusals():
    import delta_rule_recurrent_gdn_amd as gdn

    x = torch.zeros(2, 5, 3, 64, device="cuda")
    f = torch.ones(16, device="cuda")
    bad = [
        (TypeError, lambda: gdn.gdn2_qk_norm_rope_fwd(x, x.bfloat16())),
        (ValueError, lambda: gdn.gdn2_qk_norm_rope_fwd(x, x[:, :4])),
        (ValueError, lambda: gdn.gdn2_qk_norm_rope_fwd(x[0, 0], None)),
        (ValueError, lambda: gdn.gdn2_qk_norm_rope_fwd(x, x, torch.zeros(5, 2, dtype=torch.int64, device="cuda"), f)),
        (TypeError, lambda: gdn.gdn2_qk_norm_rope_fwd(x, x, torch.zeros(2, 5, device="cuda"), f)),
        (TypeError, lambda: gdn.gdn2_qk_norm_rope_fwd(x, x, None, f.double())),
        (ValueError, lambda: gdn.gdn2_qk_norm_rope_fwd(x, x, None, f.cpu())),
        (ValueError, lambda: gdn.gdn2_qk_norm_rope_fwd(x, None, k_weight=torch.ones(64, device="cuda"))),
        (ValueError, lambda: gdn.gdn2_qk_norm_rope_fwd(x, x, q_weight=torch.ones(32, device="cuda"))),
        (ValueError, lambda: gdn.gdn2_qk_norm_rope_fwd(x, x, q_out=torch.zeros(2, 5, 4, 64, device="cuda"))),
        (RuntimeError, lambda: gdn.gdn2_qk_norm_rope_fwd(x, x, None, torch.ones(4, device="cuda"))),     # rot = 8
        (RuntimeError, lambda: gdn.gdn2_qk_norm_rope_fwd(x, x, None, torch.ones(48, device="cuda"))),    # rot > D
        (RuntimeError, lambda: gdn.gdn2_qk_norm_rope_fwd(x, x, eps=-1.0)),
        (ValueError, lambda: gdn.gdn2_qk_norm_rope_bwd(x, x[:, :4], x, x)),
        (ValueError, lambda: gdn.gdn2_qk_norm_rope_bwd(x.transpose(1, 2), x, x, x)),
        (RuntimeError, lambda: gdn.gdn2_qk_norm_rope_bwd(x, x, x, x, q_weight=torch.ones(64, device="cuda"),
                                                         workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("l2", [False, True], ids=["rms", "l2"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_fp32_gradients_of_bf16_inputs_row_by_row(case, l2, interleaved):
    """As the main test, with gradients in fp32: dq, dk and both weights' gradients (weights with the L2 norm too)."""
    import delta_rule_recurrent_gdn_amd as gdn

    lead, Hq, Hk, D, rot = case
    x = make(D + rot + Hq + 1, lead, Hq, Hk, D, rot, BF16)
    g = torch.Generator().manual_seed(rot + D)
    dy = {"q": torch.randn(*lead, Hq, D, generator=g), "k": torch.randn(*lead, Hk, D, generator=g)}
    d = {n: t.cuda() for n, t in x.items()}
    kw = dict(eps=1e-3, l2=l2, interleaved=interleaved)
    q, k = cut(x, Hq, Hk, D)
    gq, gk = cut(d, Hq, Hk, D)
    got = gdn.gdn2_qk_norm_rope_bwd(dy["q"].cuda(), dy["k"].cuda(), gq, gk, d["pos"], d["f"].float() if rot else None,
                                    q_weight=d["wq"], k_weight=d["wk"], q_scale=0.25, **kw)
    for n, t, w, s in (("q", q, x["wq"], 0.25), ("k", k, x["wk"], 1.0)):
        dx, dw = O.qk_norm_rope_backward(dy[n], t, x["pos"].numpy(), x["f"].float(), w, scale=s, **kw)
        t64, dy64 = np.abs(t.double().numpy()), np.abs(dy[n].double().numpy())
        m = (t64 ** 2).sum(-1, keepdims=True) / (1 if l2 else D) + 1e-3
        h = s * 2 * dy64.max(-1, keepdims=True) * np.abs(w.numpy())
        mag = h / np.sqrt(m) + t64 * (h * t64).sum(-1, keepdims=True) / ((1 if l2 else D) * m ** 1.5)
        assert got["d" + n].dtype == BF16
        near("d" + n, got["d" + n], dx, mag, D)
        rows = t64.reshape(-1, D).shape[0]
        terms = (s * 2 * dy64.max(-1, keepdims=True) * t64 / np.sqrt(m)).reshape(-1, D).sum(0)
        assert (np.abs(got[f"d{n}_weight"].cpu().double().numpy() - dw) <= (rows + D + 64) * 2.0 ** -24 * terms).all(), n
