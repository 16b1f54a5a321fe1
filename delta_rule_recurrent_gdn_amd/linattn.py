"""Torch binding of the linear attention with a decay for each head (argument marshalling only).

Each function has the name of the C entry point it calls (include/gdn2.h):

    S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t

    q, k : [B, T, Hk, Dk]    v, o, dO : [B, T, H, Dv]    (decode: without T; packed: B = 1)
    log_decay : [H] fp32     states : [B, H, Dk, Dv] fp32 (packed: [N, H, Dk, Dv])

H is a multiple of Hk: head h of v shares the q and k of head h // (H // Hk). q, k, v, dO are all bf16 or all fp32;
o, dq, dk, dv have their type. log_decay is a constant: no gradient with respect to it is formed.
"""

import contextlib

import torch

from . import _lib

_DT = {torch.float32: _lib.GDN2_F32, torch.bfloat16: _lib.GDN2_BF16}
_SAME = contextlib.nullcontext()


def _on(device):
    """The context that makes `device` current for a launch, where it is not."""
    return _SAME if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)


def _stream(device):
    """The handle of `device`'s current stream (without the Stream object, which costs some 3 us)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _code(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DT:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    return _DT[t.dtype]


def _like(name, t, shape, dtype, device):
    """Checks a contiguous tensor of the given shape, type and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _sizes(q, k, v, log_decay, ndim):
    """(dtype code, device, leading sizes, Hk, H, Dk, Dv) of checked inputs."""
    dt = _code(q, "q")
    if q.dim() != ndim:
        raise ValueError(f"q has {q.dim()} dimensions, expected {ndim}")
    if not isinstance(v, torch.Tensor) or v.dim() != ndim:
        raise ValueError(f"v must be a tensor of {ndim} dimensions")
    *lead, Hk, Dk = q.shape
    H, Dv = v.shape[-2:]
    _like("q", q, q.shape, q.dtype, q.device)
    _like("k", k, q.shape, q.dtype, q.device)
    _like("v", v, (*lead, H, Dv), q.dtype, q.device)
    _like("log_decay", log_decay, (H,), torch.float32, q.device)
    return dt, q.device, lead, Hk, H, Dk, Dv


def _state(name, t, shape, device):
    if t is not None:
        _like(name, t, shape, torch.float32, device)


def _scratch(workspace, need, device):
    """(pointer, bytes, keeper) of a workspace of at least `need` bytes: the caller's, or a new one."""
    if need == 0:
        return None, 0, None
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def gdn2_linattn_workspace_bytes(op, N, T, Hk, H, Dk, Dv, dtype, packed=False):
    """Bytes that a forward (op GDN2_OP_FWD) or backward (GDN2_OP_BWD) of these sizes needs as workspace."""
    if dtype not in _DT:
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    return _lib.load().gdn2_linattn_workspace_bytes(op, N, T, Hk, H, Dk, Dv, int(packed), _DT[dtype])


def _packed(q, cu_seqlens):
    if q.shape[0] != 1:
        raise ValueError(f"a packed batch has q of shape [1, T, Hk, Dk], got {tuple(q.shape)}")
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a tensor [N + 1]")
    _like("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int64, q.device)
    return cu_seqlens.numel() - 1


def _new(shape, dtype, device, cu, N):
    """An output: of a packed batch, with zeros in the rows outside every sequence, which the kernels do not write."""
    if cu is None or N == 0:
        return (torch.empty if cu is None else torch.zeros)(shape, dtype=dtype, device=device)
    t = torch.empty(shape, dtype=dtype, device=device)
    row = shape[2] * shape[3] * t.element_size()
    with _on(device):
        st = _lib.load().gdn2_varlen_zero_outside(t.data_ptr(), cu.data_ptr(), N, shape[1], row, _stream(device))
    _lib.check(st, "gdn2_varlen_zero_outside")
    return t


def _forward(q, k, v, log_decay, cu, S0, scale, want_final_state, o, workspace):
    lib = _lib.load()
    dt, dev, (B, T), Hk, H, Dk, Dv = _sizes(q, k, v, log_decay, 4)
    N = B if cu is None else _packed(q, cu)
    _state("S0", S0, (N, H, Dk, Dv), dev)
    if o is None:
        o = _new((B, T, H, Dv), q.dtype, dev, cu, N)
    else:
        _like("o", o, (B, T, H, Dv), q.dtype, dev)
    S_final = torch.empty((N, H, Dk, Dv), dtype=torch.float32, device=dev) if want_final_state else None
    need = lib.gdn2_linattn_workspace_bytes(_lib.GDN2_OP_FWD, N, T, Hk, H, Dk, Dv, int(cu is not None), dt)
    ws, ws_bytes, keep = _scratch(workspace, need, dev)
    stream = _stream(dev)
    with _on(dev):
        if cu is None:
            st = lib.gdn2_linattn_fwd_chunked(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(S0), _ptr(o),
                                              _ptr(S_final), ws, ws_bytes, B, T, Hk, H, Dk, Dv, scale, dt, stream)
        else:
            st = lib.gdn2_linattn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(cu), N, _ptr(S0),
                                             _ptr(o), _ptr(S_final), ws, ws_bytes, T, Hk, H, Dk, Dv, scale, dt, stream)
    _lib.check(st, "gdn2_linattn_fwd_chunked" if cu is None else "gdn2_linattn_fwd_varlen")
    return o, S_final


def gdn2_linattn_fwd_chunked(q, k, v, log_decay, S0=None, scale=1.0, want_final_state=True, o=None, workspace=None):
    """Chunked forward over T tokens. Returns (o [B,T,H,Dv], S_final [B,H,Dk,Dv] or None). `o` and `workspace` may
    supply the output and the scratch (gdn2_linattn_workspace_bytes(GDN2_OP_FWD, ...) bytes)."""
    return _forward(q, k, v, log_decay, None, S0, scale, want_final_state, o, workspace)


def gdn2_linattn_fwd_varlen(q, k, v, log_decay, cu_seqlens, S0=None, scale=1.0, want_final_state=True, o=None,
                            workspace=None):
    """Packed variable-length forward: q, k [1,T,Hk,Dk], v [1,T,H,Dv], cu_seqlens int64 [N+1] on the device. Returns
    (o [1,T,H,Dv], S_final [N,H,Dk,Dv] or None). Rows of a given `o` outside every sequence are left as they are;
    an `o` made here is zero there."""
    return _forward(q, k, v, log_decay, cu_seqlens, S0, scale, want_final_state, o, workspace)


def _backward(q, k, v, log_decay, dO, cu, S0, dS_final, scale, want_dS0, workspace):
    lib = _lib.load()
    dt, dev, (B, T), Hk, H, Dk, Dv = _sizes(q, k, v, log_decay, 4)
    N = B if cu is None else _packed(q, cu)
    _like("dO", dO, v.shape, q.dtype, dev)
    _state("S0", S0, (N, H, Dk, Dv), dev)
    _state("dS_final", dS_final, (N, H, Dk, Dv), dev)
    g = {n: _new(t.shape, q.dtype, dev, cu, N) for n, t in (("dq", q), ("dk", q), ("dv", v))}
    g["dS0"] = torch.empty((N, H, Dk, Dv), dtype=torch.float32, device=dev) if want_dS0 else None
    need = lib.gdn2_linattn_workspace_bytes(_lib.GDN2_OP_BWD, N, T, Hk, H, Dk, Dv, int(cu is not None), dt)
    ws, ws_bytes, keep = _scratch(workspace, need, dev)
    out = (_ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dS0"]), ws, ws_bytes)
    stream = _stream(dev)
    with _on(dev):
        if cu is None:
            st = lib.gdn2_linattn_bwd_chunked(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(S0), _ptr(dO),
                                              _ptr(dS_final), *out, B, T, Hk, H, Dk, Dv, scale, dt, stream)
        else:
            st = lib.gdn2_linattn_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(cu), N, _ptr(S0),
                                             _ptr(dO), _ptr(dS_final), *out, T, Hk, H, Dk, Dv, scale, dt, stream)
    _lib.check(st, "gdn2_linattn_bwd_chunked" if cu is None else "gdn2_linattn_bwd_varlen")
    return g


def gdn2_linattn_bwd_chunked(q, k, v, log_decay, dO, S0=None, dS_final=None, scale=1.0, want_dS0=True, workspace=None):
    """Gradients of <dO, o> + <dS_final, S_final>. Returns a dict with dq, dk, dv (the inputs' type) and dS0 (fp32,
    or None)."""
    return _backward(q, k, v, log_decay, dO, None, S0, dS_final, scale, want_dS0, workspace)


def gdn2_linattn_bwd_varlen(q, k, v, log_decay, dO, cu_seqlens, S0=None, dS_final=None, scale=1.0, want_dS0=True,
                            workspace=None):
    """Packed variable-length backward: the dict of gdn2_linattn_bwd_chunked, zero outside every sequence."""
    return _backward(q, k, v, log_decay, dO, cu_seqlens, S0, dS_final, scale, want_dS0, workspace)


def _decode(name, q, k, v, log_decay, S, slots, scale, o):
    lib = _lib.load()
    dt, dev, (B,), Hk, H, Dk, Dv = _sizes(q, k, v, log_decay, 3)
    if not isinstance(S, torch.Tensor) or S.dim() != 4:
        raise ValueError("the state must be a tensor of 4 dimensions")
    _state("S" if slots is None else "S_pool", S, (B if slots is None else S.shape[0], H, Dk, Dv), dev)
    if o is None:
        o = torch.empty((B, H, Dv), dtype=q.dtype, device=dev)
    else:
        _like("o", o, v.shape, q.dtype, dev)
    x = (_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(S))
    stream = _stream(dev)
    with _on(dev):
        if slots is None:
            st = lib.gdn2_linattn_decode_step(*x, _ptr(o), B, Hk, H, Dk, Dv, scale, dt, stream)
        else:
            _like("slots", slots, (B,), torch.int32, dev)
            st = lib.gdn2_linattn_decode_step_slots(*x, _ptr(slots), S.shape[0], _ptr(o), B, Hk, H, Dk, Dv, scale, dt,
                                                    stream)
    _lib.check(st, name)
    return o


def gdn2_linattn_decode_step(q, k, v, log_decay, S, scale=1.0, o=None):
    """One token: q, k [B,Hk,Dk], v [B,H,Dv]; S [B,H,Dk,Dv] fp32 is updated in place. Returns o [B,H,Dv]."""
    return _decode("gdn2_linattn_decode_step", q, k, v, log_decay, S, None, scale, o)


def gdn2_linattn_decode_step_slots(q, k, v, log_decay, S_pool, slots, scale=1.0, o=None):
    """One token for entries whose states are S_pool[slots[b]] ([num_slots,H,Dk,Dv] fp32, in place; distinct slots);
    slots int32 [B] on the device, an entry outside the pool gets o = 0. Returns o [B,H,Dv]."""
    if slots is None:
        raise TypeError("slots must be a torch.Tensor")
    return _decode("gdn2_linattn_decode_step_slots", q, k, v, log_decay, S_pool, slots, scale, o)
