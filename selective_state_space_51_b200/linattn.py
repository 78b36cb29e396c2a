"""Linear attention with a decay for each head (include/ssm_linattn.h)."""
from __future__ import annotations

import ctypes

from . import (_check, _ptr, _stream, library, ssm_linattn_dims)
from ._launch import apart, dense, dtype_codes, dtype_error, launch, ptr


def _dims(dims):
    if isinstance(dims, ssm_linattn_dims):
        return dims
    return ssm_linattn_dims(*[int(d) for d in dims])


# of a backward call's workspace: what it does without
SSM_LINATTN_NO_HEAD_GRADIENT, SSM_LINATTN_NO_DECAY_GRADIENT = 2, 4


def ssm_linattn_workspace(device, dims, dtype, backward=False) -> int:
    """Bytes of workspace a forward (or backward) call needs; backward: True,
    or 1 plus what the call does without."""
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


def ssm_linattn_sync_status(device=0, stream=None) -> int:
    """Status code (not raised): SSM_OK, SSM_ERR_TIMEOUT or SSM_ERR_CUDA."""
    return library().ssm_linattn_sync_status(int(device), _stream(stream))


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

    stream: None for torch's current stream, a torch stream or a raw one. On
    another stream than the current one a call comes behind what the current
    stream has been given so far, and its tensors' memory is kept until it is
    done (with a raw stream the caller keeps it); its results belong to
    `stream`, and work on other streams that reads them waits for it.
    """

    def __init__(self, device: int = 0):
        import torch
        self._torch = torch
        self._lib = library()
        self._codes = dtype_codes()
        self.device = torch.device("cuda", int(device))
        self._bytes = {}

    def _rows(self, name, t, shape, heads, d, dtype):
        """Elements from one token of `t` to the next; shape: (b, L, heads,
        size), or (b, heads, size) for one token."""
        if t.shape != shape or t.dtype is not dtype or t.device != self.device:
            raise ValueError("%s must be a %s tensor of shape %s on %s" % (
                name, dtype, tuple(shape), self.device))
        dense_step = heads * d
        if t.is_contiguous():
            return dense_step
        s = t.stride()
        if len(shape) == 4 and shape[1] > 1:
            step = s[1]
            even = shape[0] == 1 or s[0] == shape[1] * step
        else:
            step, even = (s[0] if shape[0] > 1 else dense_step), True
        if not (even and step >= dense_step and (d == 1 or s[-1] == 1)
                and (heads == 1 or s[-2] == d)):
            raise ValueError(
                "%s must hold each token's heads in one piece, with one "
                "distance between all tokens" % name)
        return step

    def _inputs(self, q, k, v, log_decay, head_log_decay, lengths, scale,
                rank=4):
        sq, sv, ty = q.shape, v.shape, q.dtype
        if len(sq) != rank or len(sv) != rank:
            raise ValueError("q, k and v must have the dimensions [batch, "
                             "%sheads, size]" % ("tokens, " if rank == 4
                                                 else ""))
        code = self._codes.get(ty)
        if code is None:
            raise dtype_error()
        G, dk = sq[-2:]
        H, dv = sv[-2:]
        if 0 in sq or 0 in sv:
            raise ValueError("q, k and v must not be empty")
        if sv[:-2] != sq[:-2] or H % G:
            raise ValueError("v must have q's tokens, and a multiple of its "
                             "heads")
        rows = self._rows
        dims = (sq[0], sq[1] if rank == 4 else 1, H, G, dk, dv,
                rows("q", q, sq, G, dk, ty), rows("k", k, sq, G, dk, ty),
                rows("v", v, sv, H, dv, ty))
        if log_decay is not None:
            dense("log_decay", log_decay, sv[:-1], ty, self.device)
        if head_log_decay is not None:
            dense("head_log_decay", head_log_decay, (H,), self._torch.float32,
                  self.device)
        if lengths is not None:
            dense("lengths", lengths, (sq[0],), self._torch.int32, self.device)
        return dims, code, dk ** -0.5 if scale is None else scale

    def _workspace(self, dims, code, backward):
        """Allocated anew for each call, on its stream: nothing is shared."""
        torch = self._torch
        key = (dims[:6], code, backward)
        n = self._bytes.get(key)
        if n is None:
            n = self._bytes[key] = ssm_linattn_workspace(
                self.device.index, dims, code, backward)
        if n == 0:
            return None, 0
        return torch.empty(n, dtype=torch.uint8, device=self.device), n

    def sync_status(self, stream=None) -> int:
        """Waits for the stream; SSM_OK unless a kernel's bounded wait gave
        up or the device has an error."""
        torch = self._torch
        with torch.cuda.device(self.device):
            if stream is None:
                stream = torch.cuda.current_stream()
            return ssm_linattn_sync_status(self.device.index, stream)

    def __call__(self, q, k, v, log_decay=None, head_log_decay=None,
                 scale=None, lengths=None, h0=None, y=None, h_last=None,
                 return_last_state=True, stream=None):
        """A prompt: y [b, L, H, dv], and the last state with
        return_last_state. h_last may be h0 itself."""
        torch = self._torch
        dims, code, scale = self._inputs(q, k, v, log_decay, head_log_decay,
                                         lengths, scale)
        state = (dims[0], dims[2], dims[4], dims[5])
        dense("h0", h0, state, torch.float32, self.device)
        dense("h_last", h_last, state, torch.float32, self.device)
        dense("y", y, v.shape, q.dtype, self.device)
        if h_last is not None and h0 is not None and \
                h_last.data_ptr() != h0.data_ptr():
            apart(h0=h0, h_last=h_last)
        y, h_last = launch(self._torch, self.device, stream, self._prompt, q, k, v,
                           log_decay, head_log_decay, scale, lengths, h0, y,
                           h_last, return_last_state, dims, code)
        return (y, h_last) if return_last_state else y

    def _prompt(self, s, q, k, v, log_decay, head_log_decay, scale, lengths,
                h0, y, h_last, want_last, dims, code):
        torch = self._torch
        if y is None:
            y = torch.empty_like(v, memory_format=torch.contiguous_format)
        if h_last is None and want_last:
            h_last = torch.empty((dims[0], dims[2], dims[4], dims[5]),
                                 dtype=torch.float32, device=self.device)
        ws, n = self._workspace(dims, code, 0)
        _check(self._lib.ssm_linattn_fwd(
            self.device.index, q.data_ptr(), k.data_ptr(), v.data_ptr(),
            ptr(log_decay), ptr(head_log_decay), scale, ptr(lengths), ptr(h0),
            y.data_ptr(), ptr(h_last), ptr(ws), n, ssm_linattn_dims(*dims),
            code, s), "ssm_linattn_fwd")
        return y, h_last

    def step(self, q, k, v, state, log_decay=None, head_log_decay=None,
             scale=None, y=None, stream=None):
        """One token of every sequence: q, k [b, G, dk], v [b, H, dv],
        log_decay [b, H]. state is updated in place. Returns y [b, H, dv]."""
        torch = self._torch
        dims, code, scale = self._inputs(q, k, v, log_decay, head_log_decay,
                                         None, scale, rank=3)
        if state is None:
            raise ValueError("state is required")
        dense("state", state, (dims[0], dims[2], dims[4], dims[5]),
              torch.float32, self.device)
        dense("y", y, v.shape, q.dtype, self.device)
        return launch(self._torch, self.device, stream, self._step, q, k, v, state,
                      log_decay, head_log_decay, scale, y, dims, code)

    def _step(self, s, q, k, v, state, log_decay, head_log_decay, scale, y,
              dims, code):
        torch = self._torch
        if y is None:
            y = torch.empty_like(v, memory_format=torch.contiguous_format)
        _check(self._lib.ssm_linattn_step(
            self.device.index, q.data_ptr(), k.data_ptr(), v.data_ptr(),
            ptr(log_decay), ptr(head_log_decay), scale, state.data_ptr(),
            y.data_ptr(), ssm_linattn_dims(*dims), code, s),
            "ssm_linattn_step")
        return y

    def backward(self, q, k, v, dy, log_decay=None, head_log_decay=None,
                 scale=None, lengths=None, h0=None, dh_last=None,
                 decay_gradient=True, stream=None):
        """Gradients of sum(dy * y) + sum(dh_last * h_last). Returns a dict:
        dq, dk [b, L, G, dk] (sums over each group's heads), dv, dlog_decay
        (activation dtype), dhead_log_decay, dh0 (float32). The decays'
        gradients are None without their inputs, or with decay_gradient=False
        (a fixed decay: fewer products)."""
        torch = self._torch
        dims, code, scale = self._inputs(q, k, v, log_decay, head_log_decay,
                                         lengths, scale)
        if dy is None:
            raise ValueError("dy is required")
        state = (dims[0], dims[2], dims[4], dims[5])
        dense("dy", dy, v.shape, q.dtype, self.device)
        dense("h0", h0, state, torch.float32, self.device)
        dense("dh_last", dh_last, state, torch.float32, self.device)
        return launch(self._torch, self.device, stream, self._backward, q, k, v, dy,
                      log_decay, head_log_decay, scale, lengths, h0, dh_last,
                      decay_gradient, dims, code)

    def _backward(self, s, q, k, v, dy, log_decay, head_log_decay, scale,
                  lengths, h0, dh_last, decay_gradient, dims, code):
        torch = self._torch
        b, L, H, G, dk, dv = dims[:6]
        act = dict(dtype=q.dtype, device=self.device)
        f = dict(dtype=torch.float32, device=self.device)
        g = dict(
            dq=torch.empty((b, L, G, dk), **act),
            dk=torch.empty((b, L, G, dk), **act),
            dv=torch.empty((b, L, H, dv), **act),
            dlog_decay=torch.empty((b, L, H), **act)
            if log_decay is not None and decay_gradient else None,
            dhead_log_decay=torch.empty((H,), **f)
            if head_log_decay is not None and decay_gradient else None,
            dh0=torch.empty((b, H, dk, dv), **f))
        kind = 1
        if g["dhead_log_decay"] is None:
            kind += (SSM_LINATTN_NO_DECAY_GRADIENT if g["dlog_decay"] is None
                     else SSM_LINATTN_NO_HEAD_GRADIENT)
        ws, n = self._workspace(dims, code, kind)
        _check(self._lib.ssm_linattn_bwd(
            self.device.index, q.data_ptr(), k.data_ptr(), v.data_ptr(),
            ptr(log_decay), ptr(head_log_decay), scale, ptr(lengths), ptr(h0),
            dy.data_ptr(), ptr(dh_last), g["dq"].data_ptr(),
            g["dk"].data_ptr(), g["dv"].data_ptr(), ptr(g["dlog_decay"]),
            ptr(g["dhead_log_decay"]), g["dh0"].data_ptr(), ptr(ws), n,
            ssm_linattn_dims(*dims), code, s), "ssm_linattn_bwd")
        return g
