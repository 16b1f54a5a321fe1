"""Refusals of the linear attention's and the head norms' entry points, before anything is launched (no GPU needed)."""

import pytest
import torch

import delta_rule_recurrent_gdn_amd as gdn
from delta_rule_recurrent_gdn_amd import _lib

A = 4096  # an aligned address that is never read: the checks fail first, or there is nothing to do
OK, NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3, -4, -5, -6


def fwd(**kw):
    a = dict(q=A, k=A, v=A, ld=A, S0=None, o=A, Sf=None, ws=None, wsb=0, B=1, T=64, Hk=2, H=4, Dk=64, Dv=64, dt=1)
    a.update(kw)
    return _lib.load().gdn2_linattn_fwd_chunked(a["q"], a["k"], a["v"], a["ld"], a["S0"], a["o"], a["Sf"], a["ws"],
                                                a["wsb"], a["B"], a["T"], a["Hk"], a["H"], a["Dk"], a["Dv"], 1.0,
                                                a["dt"], None)


def bwd(**kw):
    a = dict(q=A, dO=A, dq=A, dk=A, dv=A, dS0=None, ws=None, wsb=0, B=1, T=64, Hk=2, H=4, Dk=64, Dv=64, dt=1)
    a.update(kw)
    return _lib.load().gdn2_linattn_bwd_chunked(a["q"], A, A, A, None, a["dO"], None, a["dq"], a["dk"], a["dv"],
                                                a["dS0"], a["ws"], a["wsb"], a["B"], a["T"], a["Hk"], a["H"], a["Dk"],
                                                a["Dv"], 1.0, a["dt"], None)


def varlen(**kw):
    a = dict(cu=A, N=3, ws=None, wsb=0, T=64)
    a.update(kw)
    return _lib.load().gdn2_linattn_fwd_varlen(A, A, A, A, a["cu"], a["N"], None, A, None, a["ws"], a["wsb"], a["T"], 1,
                                               1, 64, 64, 1.0, 1, None)


def decode(**kw):
    a = dict(q=A, S=A, slots=A, num=4, B=2, Hk=2, H=4, Dk=64, dt=1)
    a.update(kw)
    return _lib.load().gdn2_linattn_decode_step_slots(a["q"], A, A, A, a["S"], a["slots"], a["num"], A, a["B"], a["Hk"],
                                                      a["H"], a["Dk"], 64, 1.0, a["dt"], None)


def norm(**kw):
    a = dict(q=A, k=A, pos=A, f=A, qo=A, ko=A, n=5, period=5, Hq=2, Hk=1, D=64, rot=32, sq=128, sk=64, so=128, sko=64,
             eps=1e-6, dt=1, flags=0)
    a.update(kw)
    return _lib.load().gdn2_qk_norm_rope_fwd(a["q"], a["k"], None, None, a["pos"], a["f"], a["qo"], a["ko"], a["n"],
                                             a["period"], a["Hq"], a["Hk"], a["D"], a["rot"], a["sq"], a["sk"],
                                             a["so"], a["sko"], a["eps"], 1.0, a["dt"], a["flags"], None)


def norm_bwd(**kw):
    a = dict(dq=A, dk=A, wq=None, ws=None, wsb=0, n=5, dt=1, dtg=1, sq=128)
    a.update(kw)
    return _lib.load().gdn2_qk_norm_rope_bwd(A, A, A, A, None, None, A, A, a["dq"], a["dk"], a["wq"], None, a["ws"],
                                             a["wsb"], a["n"], 5, 2, 1, 64, 32, a["sq"], 64, 128, 64, 1e-6, 1.0,
                                             a["dt"], a["dtg"], 0, None)


@pytest.mark.parametrize("call,kw,status", [
    (fwd, dict(q=None), NULL), (fwd, dict(ld=None), NULL), (fwd, dict(o=None), NULL),
    (fwd, dict(k=A + 8), ALIGN), (fwd, dict(S0=A + 4), ALIGN), (fwd, dict(ld=A + 2), ALIGN),
    (fwd, dict(dt=2), DTYPE), (fwd, dict(Dk=48), UNSUPPORTED), (fwd, dict(Dv=256), UNSUPPORTED),
    (fwd, dict(H=3), SHAPE), (fwd, dict(Hk=0), SHAPE), (fwd, dict(T=-1), SHAPE), (fwd, dict(T=(1 << 30) + 1), SHAPE),
    (fwd, dict(B=1 << 29, T=1), SHAPE), (fwd, dict(B=1 << 18, T=1), SHAPE),  # more threads than a grid holds
    (fwd, dict(T=65536), WORKSPACE), (fwd, dict(T=65536, ws=A, wsb=1), WORKSPACE),
    (fwd, dict(T=65536, ws=A + 16, wsb=1 << 40), ALIGN),
    (fwd, dict(B=0), OK), (fwd, dict(H=0), OK), (fwd, dict(T=0, q=None, o=None), OK),
    (bwd, dict(dO=None), NULL), (bwd, dict(dk=None), NULL), (bwd, dict(dv=A + 4), ALIGN), (bwd, dict(dS0=A + 4), ALIGN),
    (bwd, dict(), WORKSPACE),                                # shared heads: room for their gradients
    (bwd, dict(Dk=24), UNSUPPORTED), (bwd, dict(B=0), OK), (bwd, dict(T=0), OK),
    (varlen, dict(cu=None), NULL), (varlen, dict(cu=A + 4), ALIGN), (varlen, dict(), WORKSPACE), (varlen, dict(N=0), OK),
    (varlen, dict(N=-1), SHAPE),
    (decode, dict(S=None), NULL), (decode, dict(slots=None), NULL), (decode, dict(num=-1), SHAPE),
    (decode, dict(S=A + 8), ALIGN), (decode, dict(slots=A + 2), ALIGN), (decode, dict(H=5), SHAPE),
    (decode, dict(Dk=80), UNSUPPORTED), (decode, dict(dt=9), DTYPE), (decode, dict(B=0), OK),
    (decode, dict(B=1 << 22, Hk=4), SHAPE),
    (norm, dict(q=None), NULL), (norm, dict(k=None), NULL), (norm, dict(ko=None), NULL), (norm, dict(f=None), NULL),
    (norm, dict(q=A + 4), ALIGN), (norm, dict(pos=A + 4), ALIGN), (norm, dict(sq=132), ALIGN), (norm, dict(sq=64), SHAPE),
    (norm, dict(so=120), SHAPE), (norm, dict(rot=8), UNSUPPORTED), (norm, dict(rot=80), SHAPE),
    (norm, dict(rot=-16), SHAPE), (norm, dict(D=96), UNSUPPORTED), (norm, dict(flags=1), UNSUPPORTED),
    (norm, dict(eps=-1.0), SHAPE), (norm, dict(eps=float("nan")), SHAPE), (norm, dict(period=0), SHAPE),
    (norm, dict(Hq=0), SHAPE), (norm, dict(n=-1), SHAPE), (norm, dict(n=1 << 26), SHAPE), (norm, dict(dt=3), DTYPE), (norm, dict(n=0), OK),
    (norm_bwd, dict(dq=None), NULL), (norm_bwd, dict(wq=A), WORKSPACE), (norm_bwd, dict(wq=A + 4), ALIGN),
    (norm_bwd, dict(wq=A, ws=A + 64, wsb=1 << 30), ALIGN), (norm_bwd, dict(dt=0, dtg=1), DTYPE),
    (norm_bwd, dict(sq=100), SHAPE), (norm_bwd, dict(n=0), OK),
])
def test_refusals(call, kw, status):
    assert call(**kw) == status


@pytest.mark.parametrize("args,status", [
    ((None, A, 2, 8, 64), NULL), ((A, None, 2, 8, 64), NULL), ((A + 8, A, 2, 8, 64), ALIGN), ((A, A + 4, 2, 8, 64), ALIGN),
    ((A, A, 2, 8, 40), ALIGN), ((A, A, -1, 8, 64), SHAPE), ((A, A, 2, -8, 64), SHAPE), ((None, None, 0, 8, 64), OK),
    ((None, None, 2, 0, 64), OK),
])
def test_zero_outside_refusals(args, status):
    assert _lib.load().gdn2_varlen_zero_outside(*args, None) == status


def test_workspace_bytes():
    lib = _lib.load()
    size = lambda op, N, T, Hk, H, Dk, Dv, packed: lib.gdn2_linattn_workspace_bytes(op, N, T, Hk, H, Dk, Dv, packed, 1)  # noqa: E731
    assert size(0, 8, 4096, 16, 16, 128, 128, 0) == 0           # whole sequences fill the GPU
    pieces = size(0, 1, 65536, 16, 16, 128, 128, 0)             # a state a piece and head
    assert pieces > 0 and pieces % (16 * 128 * 128 * 4) == 0
    assert size(_lib.GDN2_OP_BWD, 8, 4096, 4, 16, 128, 128, 0) == 2 * 8 * 4096 * 16 * 128 * 4  # fp32 dq, dk of every head
    assert size(0, 3, 1000, 2, 2, 64, 64, 1) > 0
    assert size(0, 0, 64, 2, 2, 64, 64, 0) == size(0, 1, 64, 2, 3, 64, 64, 0) == 0
    assert size(_lib.GDN2_OP_DECODE, 1, 64, 2, 2, 64, 64, 0) == 0
    assert lib.gdn2_qk_norm_rope_workspace_bytes(32768, 16, 16, 128) == 1024 * 2 * 128 * 4
    assert lib.gdn2_qk_norm_rope_workspace_bytes(0, 16, 16, 128) == 0


def test_binding_refuses():
    q = torch.zeros(1, 8, 2, 64)
    ld = torch.zeros(2)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn2_linattn_fwd_chunked(q, q, q, ld)
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn2_linattn_decode_step(q[:, 0], q[:, 0], q[:, 0], ld, torch.zeros(1, 2, 64, 64))
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn2_qk_norm_rope_fwd(q, q)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        gdn.gdn2_linattn_fwd_chunked(q.half(), q.half(), q.half(), ld)
    with pytest.raises(TypeError):
        gdn.gdn2_linattn_fwd_chunked(None, q, q, ld)
    with pytest.raises(TypeError, match="dtype must be"):
        gdn.gdn2_linattn_workspace_bytes(0, 1, 64, 1, 1, 64, 64, torch.float16)


def test_rows_of_a_projection():
    from delta_rule_recurrent_gdn_amd.qk_norm import _rows

    x = torch.zeros(3, 5, 10 * 32)
    q = x[..., 64:192].unflatten(-1, (4, 32))
    assert _rows("q", q) == (15, 4, 32, 320)
    assert _rows("q", q[:, :1]) == (3, 4, 32, 1600)
    assert _rows("q", q[:1, 2:3]) == (1, 4, 32, 128)
    for bad in (q[:, :2], q.transpose(0, 1), q[..., :2], q[:, :, ::2], q.transpose(2, 3)):
        with pytest.raises(ValueError, match="side by side|evenly spaced"):
            _rows("q", bad)


@pytest.mark.parametrize("heads", [(1, 0), (16, 16)])
@pytest.mark.parametrize("D", [16, 128])
def test_norm_token_limit(heads, D):
    """Four tokens a workgroup of 256 threads, a grid of fewer than 2^32: 2^26 - 4 tokens are the most."""
    last = (1 << 26) - 4
    bytes_of = _lib.load().gdn2_qk_norm_rope_workspace_bytes
    assert bytes_of(last, *heads, D) > 0
    for n in (last + 1, last + 2, last + 3, last + 4):
        assert bytes_of(n, *heads, D) == 0
        assert norm(n=n, D=D, Hq=heads[0], Hk=heads[1], rot=16, sq=4096, sk=4096, so=4096, sko=4096) == SHAPE
        assert norm_bwd(n=n) == SHAPE
