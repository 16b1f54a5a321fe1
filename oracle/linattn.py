"""Float64 oracle of the linear attention with a decay for each head and of the q/k head norms with rotation.

Steps the definitions token by token with numpy on the CPU and shares no code with the GPU path:

    S_t = exp(log_decay_h) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
    y = R(p) (x r w),   r = (mean x^2 + eps)^(-1/2)   (l2: the sum of squares)
"""

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x.detach().cpu().double().numpy() if hasattr(x, "detach") else x, np.float64)


def linattn_forward(q, k, v, log_decay, S0=None, scale=1.0):
    """q, k [B,T,Hk,Dk], v [B,T,H,Dv] -> (o [B,T,H,Dv], S_T [B,H,Dk,Dv])."""
    q, k, v, ld, S0 = (_f64(x) for x in (q, k, v, log_decay, S0))
    B, T, Hk, Dk = q.shape
    H, Dv = v.shape[2:]
    g = np.exp(ld)
    S = np.zeros((B, H, Dk, Dv)) if S0 is None else S0.copy()
    o = np.zeros((B, T, H, Dv))
    head = np.arange(H) // (H // Hk)
    for t in range(T):
        S = g[None, :, None, None] * S + k[:, t][:, head][..., :, None] * v[:, t][..., None, :]
        o[:, t] = scale * (q[:, t][:, head][..., :, None] * S).sum(-2)
    return o, S


def linattn_backward(q, k, v, log_decay, dO, S0=None, dS_final=None, scale=1.0):
    """Gradients of <dO, o> + <dS_final, S_T>: dq, dk, dv, dS0, by the adjoint of the recurrence, token by token."""
    q, k, v, ld, dO, S0, dSf = (_f64(x) for x in (q, k, v, log_decay, dO, S0, dS_final))
    B, T, Hk, Dk = q.shape
    H, Dv = v.shape[2:]
    g = np.exp(ld)[None, :, None, None]
    head = np.arange(H) // (H // Hk)
    S = np.zeros((B, H, Dk, Dv)) if S0 is None else S0.copy()
    states = []
    for t in range(T):
        S = g * S + k[:, t][:, head][..., :, None] * v[:, t][..., None, :]
        states.append(S)
    dS = np.zeros((B, H, Dk, Dv)) if dSf is None else dSf.copy()
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for t in range(T - 1, -1, -1):
        for h in range(H):
            dq[:, t, head[h]] += scale * (states[t][:, h] * dO[:, t, h][:, None, :]).sum(-1)
        dS = dS + scale * q[:, t][:, head][..., :, None] * dO[:, t][..., None, :]
        for h in range(H):
            dk[:, t, head[h]] += (dS[:, h] * v[:, t, h][:, None, :]).sum(-1)
        dv[:, t] = (dS * k[:, t][:, head][..., :, None]).sum(-2)
        dS = g * dS
    return {"dq": dq, "dk": dk, "dv": dv, "dS0": dS}


def _pairs(rot, interleaved):
    j = np.arange(rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def rotate(x, positions, inv_freq, interleaved=False, back=False):
    """x [..., heads, D], positions [...]: the rotation of the first 2 len(inv_freq) channels, or its transpose."""
    y = x.copy()
    if inv_freq is None or len(inv_freq) == 0:
        return y
    one, two = _pairs(2 * len(inv_freq), interleaved)
    a = np.asarray(positions, np.float64)[..., None] * inv_freq
    c, s = np.cos(a)[..., None, :], np.sin(a)[..., None, :]
    if back:
        s = -s
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def qk_norm_rope(x, positions, inv_freq, weight=None, eps=1e-6, l2=False, interleaved=False, scale=1.0):
    """One of q and k: x [..., heads, D], positions [...]."""
    x, inv_freq, w = _f64(x), _f64(inv_freq), _f64(weight)
    m = (x * x).sum(-1, keepdims=True) / (1 if l2 else x.shape[-1])
    y = x / np.sqrt(m + eps)
    return scale * rotate(y if w is None else y * w, positions, inv_freq, interleaved)


def qk_norm_rope_backward(dy, x, positions, inv_freq, weight=None, eps=1e-6, l2=False, interleaved=False, scale=1.0):
    """(dx, dweight) of qk_norm_rope."""
    x, dy, inv_freq, w = _f64(x), _f64(dy), _f64(inv_freq), _f64(weight)
    w = np.ones(x.shape[-1]) if w is None else w
    n = 1 if l2 else x.shape[-1]
    m = (x * x).sum(-1, keepdims=True) / n + eps
    u = scale * rotate(dy, positions, inv_freq, interleaved, back=True)
    dw = (u * x / np.sqrt(m)).reshape(-1, x.shape[-1]).sum(0)
    h = u * w
    return h / np.sqrt(m) - x * (h * x).sum(-1, keepdims=True) / (n * m ** 1.5), dw
