"""Linear attention with a decay for each head (include/ssm_linattn.h)."""
from __future__ import annotations

import ctypes

from . import (_check, _ptr, _stream, library, ssm_linattn_dims)
from ._launch import apart, dense, dtype_code, launching


def _dims(dims):
    if isinstance(dims, ssm_linattn_dims):
        return dims
    return ssm_linattn_dims(*[int(d) for d in dims])


def ssm_linattn_workspace(device, dims, dtype, backward=False) -> int:
    """Bytes of workspace a forward (or backward) call needs."""
    n = ctypes.c_size_t(0)
    _check(library().ssm_linattn_workspace(int(device), _dims(dims),
                                           int(dtype), int(backward),
                                           ctypes.byref(n)),
           "ssm_linattn_workspace")
    return n.value


def ssm_linattn_fwd(device, q, k, v, log_decay, head_log_decay, scale, lengths,
                    h0, y, h_last, workspace, workspace_bytes, dims, dtype,
                    stream=None, check=True) -> int:
    """Call ssm_linattn_fwd with tensors (or raw addresses); dims is
    (batch, seqlen, heads, groups, dk, dv, q_stride, k_stride, v_stride).
    Returns the status; raises unless ``check`` is False."""
    rc = library().ssm_linattn_fwd(
        int(device), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay),
        _ptr(head_log_decay), scale, _ptr(lengths), _ptr(h0), _ptr(y),
        _ptr(h_last), _ptr(workspace), int(workspace_bytes), _dims(dims),
        int(dtype), _stream(stream))
    return _check(rc, "ssm_linattn_fwd") if check else rc


def ssm_linattn_step(device, q, k, v, log_decay, head_log_decay, scale, state,
                     y, dims, dtype, stream=None, check=True) -> int:
    """Call ssm_linattn_step (one token of every sequence)."""
    rc = library().ssm_linattn_step(
        int(device), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay),
        _ptr(head_log_decay), scale, _ptr(state), _ptr(y), _dims(dims),
        int(dtype), _stream(stream))
    return _check(rc, "ssm_linattn_step") if check else rc


def ssm_linattn_bwd(device, q, k, v, log_decay, head_log_decay, scale, lengths,
                    h0, dy, dh_last, dq, dk, dv, dlog_decay, dhead_log_decay,
                    dh0, workspace, workspace_bytes, dims, dtype, stream=None,
                    check=True) -> int:
    """Call ssm_linattn_bwd (gradients; see include/ssm_linattn.h)."""
    rc = library().ssm_linattn_bwd(
        int(device), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay),
        _ptr(head_log_decay), scale, _ptr(lengths), _ptr(h0), _ptr(dy),
        _ptr(dh_last), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlog_decay),
        _ptr(dhead_log_decay), _ptr(dh0), _ptr(workspace),
        int(workspace_bytes), _dims(dims), int(dtype), _stream(stream))
    return _check(rc, "ssm_linattn_bwd") if check else rc


class LinearAttention:
    """Linear attention with a decay for each head, on one device.

    S_t = exp(g_t) S_{t-1} + k_t (outer) v_t, y_t = scale q_t S_t, with
    g = log_decay + head_log_decay (either may be left out).

    q, k: [b, L, G, dk]; v: [b, L, H, dv], H a multiple of G; log_decay:
    [b, L, H], all of one type (float32 or bfloat16); head_log_decay: [H]
    float32; lengths: [b] int32; states: [b, H, dk, dv] float32. q, k and v may
    be slices of wider rows; everything else is contiguous. scale defaults to
    dk ** -0.5. The object keeps no device memory: calls may run at once on
    several streams and threads, and be captured into CUDA graphs.
    """

    def __init__(self, device: int = 0):
        import torch
        library()
        self.device = torch.device("cuda", int(device))
        self._bytes = {}

    def _rows(self, name, t, b, L, heads, d, dtype):
        """Elements from one token of `t` to the next."""
        s = t.stride() if t.dim() == 4 else None
        if (s is None or tuple(t.shape) != (b, L, heads, d)
                or t.dtype != dtype or t.device != self.device):
            raise ValueError("%s must be a %s tensor of shape %s on %s" % (
                name, dtype, (b, L, heads, d), self.device))
        step = s[1] if L > 1 else s[0] if b > 1 else heads * d
        if ((d > 1 and s[3] != 1) or (heads > 1 and s[2] != d)
                or step < heads * d or (L > 1 and b > 1 and s[0] != L * step)):
            raise ValueError(
                "%s must hold each token's heads in one piece, with one "
                "distance between all tokens" % name)
        return step

    def _inputs(self, q, k, v, log_decay, head_log_decay, lengths, scale):
        import torch
        if q.dim() != 4 or v.dim() != 4:
            raise ValueError("q, k and v must have the dimensions "
                             "[batch, tokens, heads, size]")
        code = dtype_code(q)
        b, L, G, dk = q.shape
        H, dv = v.shape[2:]
        if G == 0 or H % G:
            raise ValueError("v's heads must be a multiple of q's")
        dims = (b, L, H, G, dk, dv,
                self._rows("q", q, b, L, G, dk, q.dtype),
                self._rows("k", k, b, L, G, dk, q.dtype),
                self._rows("v", v, b, L, H, dv, q.dtype))
        dense("log_decay", log_decay, (b, L, H), q.dtype, self.device)
        dense("head_log_decay", head_log_decay, (H,), torch.float32,
              self.device)
        dense("lengths", lengths, (b,), torch.int32, self.device)
        return dims, code, dk ** -0.5 if scale is None else float(scale)

    def _workspace(self, dims, code, backward):
        """Allocated anew for each call, on its stream: nothing is shared."""
        import torch
        key = (dims[:6], code, backward)
        n = self._bytes.get(key)
        if n is None:
            n = self._bytes[key] = ssm_linattn_workspace(
                self.device.index, dims, code, backward)
        if n == 0:
            return None, 0
        return torch.empty(n, dtype=torch.uint8, device=self.device), n

    def __call__(self, q, k, v, log_decay=None, head_log_decay=None,
                 scale=None, lengths=None, h0=None, y=None, h_last=None,
                 return_last_state=True, stream=None):
        """A prompt: y [b, L, H, dv], and the last state with
        return_last_state. h_last may be h0 itself."""
        import torch
        dims, code, scale = self._inputs(q, k, v, log_decay, head_log_decay,
                                         lengths, scale)
        b, L, H, _, dk, dv = dims[:6]
        f32 = torch.float32
        dense("h0", h0, (b, H, dk, dv), f32, self.device)
        dense("h_last", h_last, (b, H, dk, dv), f32, self.device)
        dense("y", y, (b, L, H, dv), q.dtype, self.device)
        if h_last is not None and h0 is not None and \
                h_last.data_ptr() != h0.data_ptr():
            apart(h0=h0, h_last=h_last)
        with launching(self.device, stream) as s:
            if y is None:
                y = torch.empty((b, L, H, dv), dtype=q.dtype,
                                device=self.device)
            if h_last is None and return_last_state:
                h_last = torch.empty((b, H, dk, dv), dtype=f32,
                                     device=self.device)
            ws, n = self._workspace(dims, code, False)
            ssm_linattn_fwd(self.device.index, q, k, v, log_decay,
                            head_log_decay, scale, lengths, h0, y, h_last, ws,
                            n, dims, code, s)
        return (y, h_last) if return_last_state else y

    def step(self, q, k, v, state, log_decay=None, head_log_decay=None,
             scale=None, y=None, stream=None):
        """One token of every sequence: q, k [b, G, dk], v [b, H, dv],
        log_decay [b, H]. state is updated in place. Returns y [b, H, dv]."""
        import torch
        if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
            raise ValueError("q, k and v must have the dimensions "
                             "[batch, heads, size]")
        if log_decay is not None:
            log_decay = log_decay.unsqueeze(1)
        dims, code, scale = self._inputs(q.unsqueeze(1), k.unsqueeze(1),
                                         v.unsqueeze(1), log_decay,
                                         head_log_decay, None, scale)
        b, _, H, _, dk, dv = dims[:6]
        if state is None:
            raise ValueError("state is required")
        dense("state", state, (b, H, dk, dv), torch.float32, self.device)
        dense("y", y, (b, H, dv), q.dtype, self.device)
        with launching(self.device, stream) as s:
            if y is None:
                y = torch.empty((b, H, dv), dtype=q.dtype, device=self.device)
            ssm_linattn_step(self.device.index, q, k, v, log_decay,
                             head_log_decay, scale, state, y, dims, code, s)
        return y

    def backward(self, q, k, v, dy, log_decay=None, head_log_decay=None,
                 scale=None, lengths=None, h0=None, dh_last=None,
                 decay_gradient=True, stream=None):
        """Gradients of sum(dy * y) + sum(dh_last * h_last). Returns a dict:
        dq, dk [b, L, G, dk] (sums over each group's heads), dv, dlog_decay
        (activation dtype), dhead_log_decay, dh0 (float32). The decays'
        gradients are None without their inputs, or with decay_gradient=False
        (a fixed decay: fewer products)."""
        import torch
        dims, code, scale = self._inputs(q, k, v, log_decay, head_log_decay,
                                         lengths, scale)
        b, L, H, G, dk, dv = dims[:6]
        f32 = torch.float32
        if dy is None:
            raise ValueError("dy is required")
        dense("dy", dy, (b, L, H, dv), q.dtype, self.device)
        dense("h0", h0, (b, H, dk, dv), f32, self.device)
        dense("dh_last", dh_last, (b, H, dk, dv), f32, self.device)
        with launching(self.device, stream) as s:
            act = dict(dtype=q.dtype, device=self.device)
            f = dict(dtype=f32, device=self.device)
            g = dict(
                dq=torch.empty((b, L, G, dk), **act),
                dk=torch.empty((b, L, G, dk), **act),
                dv=torch.empty((b, L, H, dv), **act),
                dlog_decay=torch.empty((b, L, H), **act)
                if log_decay is not None and decay_gradient else None,
                dhead_log_decay=torch.empty((H,), **f)
                if head_log_decay is not None and decay_gradient else None,
                dh0=torch.empty((b, H, dk, dv), **f))
            ws, n = self._workspace(dims, code, True)
            ssm_linattn_bwd(self.device.index, q, k, v, log_decay,
                            head_log_decay, scale, lengths, h0, dy, dh_last,
                            g["dq"], g["dk"], g["dv"], g["dlog_decay"],
                            g["dhead_log_decay"], g["dh0"], ws, n, dims, code,
                            s)
        return g
