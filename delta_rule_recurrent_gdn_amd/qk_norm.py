"""Torch binding of the q/k head norms with the position rotation (argument marshalling only).

    y = R(position) (x / sqrt(mean(x^2) + eps) * weight)      for every head of q (also times q_scale) and of k

as gdn2_qk_norm_rope_fwd / _bwd in include/gdn2.h. q [..., Hq, D] and k [..., Hk, D] may be cut from the rows of a
fused projection: their heads lie side by side, and the rows (all leading dimensions together) are evenly spaced.
"""

import torch

from . import _lib
from .linattn import _code, _like, _on, _ptr, _scratch, _stream


def _rows(name, t, like=None):
    """(rows, heads, D, row stride in elements) of a tensor [..., heads, D] whose rows are evenly spaced."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() < 3:
        raise ValueError(f"{name} must have the shape [..., heads, D], got {tuple(t.shape)}")
    if like is not None:
        if t.dtype != like.dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {like.dtype}")
        if t.device != like.device:
            raise ValueError(f"{name} is on {t.device}, expected {like.device}")
    shape, stride = t.shape, t.stride()
    heads, D = shape[-2:]
    if t.numel() == 0:
        return 0, heads, D, heads * D
    if (D > 1 and stride[-1] != 1) or (heads > 1 and stride[-2] != D):
        raise ValueError(f"{name}'s heads must lie side by side (strides {stride})")
    rows, step, want = 1, None, None
    for d in range(len(shape) - 3, -1, -1):
        n = shape[d]
        if n != 1:
            if step is None:
                step = stride[d]
                want = step * n
            elif stride[d] != want:
                raise ValueError(f"{name}'s rows must be evenly spaced (strides {stride})")
            else:
                want *= n
            rows *= n
    return rows, heads, D, heads * D if step is None else step


def _common(q, k, positions, inv_freq, q_weight, k_weight):
    """Checked sizes: (dtype code, device, rows, period, Hq, Hk, D, rot, strides of q and k)."""
    dt = _code(q, "q")
    rows, Hq, D, sq = _rows("q", q)
    Hk, sk = 0, 0
    if k is not None:
        krows, Hk, Dk, sk = _rows("k", k, q)
        if Dk != D or k.shape[:-2] != q.shape[:-2]:
            raise ValueError(f"k has shape {tuple(k.shape)}, expected {(*q.shape[:-2], Hk, D)}")
    elif k_weight is not None:
        raise ValueError("k_weight without k")
    dev = q.device
    period = q.shape[-3]
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or positions.shape not in (q.shape[:-2], q.shape[-3:-2]):
            raise ValueError(f"positions must be a tensor {tuple(q.shape[:-2])} or {tuple(q.shape[-3:-2])}")
        _like("positions", positions, positions.shape, torch.int64, dev)
        period = positions.numel()
    rot = 0
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be a tensor [rot / 2]")
        _like("inv_freq", inv_freq, inv_freq.shape, torch.float32, dev)
        rot = 2 * inv_freq.numel()
    for n, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _like(n, w, (D,), torch.float32, dev)
    return dt, dev, rows, period, Hq, Hk, D, rot, sq, sk


def _flags(l2, interleaved):
    return (_lib.GDN2_FLAG_L2_NORM if l2 else 0) | (_lib.GDN2_FLAG_INTERLEAVED if interleaved else 0)


def _output(name, t, x):
    """(tensor, row stride): the caller's output of x's shape, or a new contiguous one."""
    if x is None:
        return None, 0
    if t is None:
        return torch.empty(x.shape, dtype=x.dtype, device=x.device), x.shape[-2] * x.shape[-1]
    stride = _rows(name, t, x)[3]
    if t.shape != x.shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(x.shape)}")
    return t, stride


def gdn2_qk_norm_rope_fwd(q, k, positions=None, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6, l2=False,
                          interleaved=False, q_scale=1.0, q_out=None, k_out=None):
    """Norm of q [..., T, Hq, D] and k [..., T, Hk, D] (or None) for each head, then the rotation of the first
    2 * len(inv_freq) channels. positions int64 [..., T] or [T] (None: 0 .. T-1); inv_freq fp32 (None: no rotation);
    weights fp32 [D] (None: ones); l2: the L2 norm in the place of the RMS norm; interleaved: channels (2j, 2j+1)
    form a pair, not (j, j + rot/2). Returns (q_out, k_out): new contiguous tensors, or the given ones (q and k
    themselves among them)."""
    lib = _lib.load()
    dt, dev, rows, period, Hq, Hk, D, rot, sq, sk = _common(q, k, positions, inv_freq, q_weight, k_weight)
    q_out, so = _output("q_out", q_out, q)
    k_out, sko = _output("k_out", k_out, k)
    stream = _stream(dev)
    with _on(dev):
        st = lib.gdn2_qk_norm_rope_fwd(_ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(positions),
                                       _ptr(inv_freq), _ptr(q_out), _ptr(k_out), rows, period, Hq, Hk, D, rot, sq, sk,
                                       so, sko, eps, q_scale, dt, _flags(l2, interleaved), stream)
    _lib.check(st, "gdn2_qk_norm_rope_fwd")
    return q_out, k_out


def gdn2_qk_norm_rope_bwd(dq_out, dk_out, q, k, positions=None, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6,
                          l2=False, interleaved=False, q_scale=1.0, dq=None, dk=None, workspace=None):
    """Gradients of gdn2_qk_norm_rope_fwd from those of its outputs (contiguous, of q's type or fp32, as the mixers'
    backward gives them). dq, dk may be given, with evenly spaced rows (a fused projection's gradient). Returns a
    dict with dq, dk (q's type) and dq_weight, dk_weight (fp32 [D]; None without the weight)."""
    lib = _lib.load()
    dt, dev, rows, period, Hq, Hk, D, rot, sq, sk = _common(q, k, positions, inv_freq, q_weight, k_weight)
    dt_grad = _code(dq_out, "dq_out")
    _like("dq_out", dq_out, q.shape, dq_out.dtype, dev)
    if k is not None:
        _like("dk_out", dk_out, k.shape, dq_out.dtype, dev)
    elif dk_out is not None:
        raise ValueError("dk_out without k")
    dq, so = _output("dq", dq, q)
    dk, sko = _output("dk", dk, k)
    dqw, dkw = (None if w is None else torch.empty(D, dtype=torch.float32, device=dev) for w in (q_weight, k_weight))
    need = 0
    if dqw is not None or dkw is not None:
        need = lib.gdn2_qk_norm_rope_workspace_bytes(rows, Hq, Hk, D)
    ws, ws_bytes, keep = _scratch(workspace, need, dev)
    stream = _stream(dev)
    with _on(dev):
        st = lib.gdn2_qk_norm_rope_bwd(_ptr(dq_out), _ptr(dk_out), _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight),
                                       _ptr(positions), _ptr(inv_freq), _ptr(dq), _ptr(dk), _ptr(dqw), _ptr(dkw), ws,
                                       ws_bytes, rows, period, Hq, Hk, D, rot, sq, sk, so, sko, eps, q_scale, dt,
                                       dt_grad, _flags(l2, interleaved), stream)
    _lib.check(st, "gdn2_qk_norm_rope_bwd")
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
