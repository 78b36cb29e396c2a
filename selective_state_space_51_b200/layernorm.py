"""Layer norm with the residual sum in front (include/ssm_layernorm.h)."""
from __future__ import annotations

import ctypes

from . import _check, _ptr, _stream, library
from ._launch import dense, dtype_codes, dtype_error, launch, ptr


def ssm_layernorm_workspace(device, rows, dim, dtype) -> int:
    """Bytes of workspace the backward call needs for its weight gradients."""
    n = ctypes.c_size_t(0)
    _check(library().ssm_layernorm_workspace(int(device), int(rows), int(dim),
                                             int(dtype), ctypes.byref(n)),
           "ssm_layernorm_workspace")
    return n.value


def ssm_layernorm_fwd(device, x, residual, weight, bias, eps, y, sum, mean,
                      rstd, rows, dim, dtype, stream=None, check=True) -> int:
    """Call ssm_layernorm_fwd with tensors (or raw addresses). Returns the
    status; raises unless ``check`` is False."""
    rc = library().ssm_layernorm_fwd(
        int(device), _ptr(x), _ptr(residual), _ptr(weight), _ptr(bias), eps,
        _ptr(y), _ptr(sum), _ptr(mean), _ptr(rstd), int(rows), int(dim),
        int(dtype), _stream(stream))
    return _check(rc, "ssm_layernorm_fwd") if check else rc


def ssm_layernorm_bwd(device, dy, x, mean, rstd, weight, dsum, dx, dweight,
                      dbias, workspace, workspace_bytes, rows, dim, dtype,
                      stream=None, check=True) -> int:
    """Call ssm_layernorm_bwd (gradients; see include/ssm_layernorm.h)."""
    rc = library().ssm_layernorm_bwd(
        int(device), _ptr(dy), _ptr(x), _ptr(mean), _ptr(rstd), _ptr(weight),
        _ptr(dsum), _ptr(dx), _ptr(dweight), _ptr(dbias), _ptr(workspace),
        int(workspace_bytes), int(rows), int(dim), int(dtype),
        _stream(stream))
    return _check(rc, "ssm_layernorm_bwd") if check else rc


class LayerNorm:
    """Layer norm over the last dimension, on one device.

    x, residual: contiguous [..., D], float32 or bfloat16; weight, bias: [D]
    float32 or None. The object keeps no device memory: calls may run at once
    on several streams and threads, and be captured into CUDA graphs. stream:
    as for LinearAttention.
    """

    def __init__(self, device: int = 0):
        import torch
        self._torch = torch
        self._lib = library()
        self._codes = dtype_codes()
        self.device = torch.device("cuda", int(device))
        self._bytes = {}

    def _rows(self, x):
        """x's type, rows and their width."""
        code, n = self._codes.get(x.dtype), x.numel()
        if code is None:
            raise dtype_error()
        if n == 0 or x.dim() < 1:
            raise ValueError("x must have at least one row")
        dim = x.shape[-1]
        return code, n // dim, dim

    def __call__(self, x, weight=None, bias=None, residual=None, eps=1e-5,
                 y=None, stream=None):
        """Norms s = x + residual (rounded to x's type). Returns a dict: y,
        sum (None without residual), mean and rstd [rows] float32, which the
        backward pass takes."""
        torch = self._torch
        code, rows, dim = self._rows(x)
        dense("x", x, x.shape, x.dtype, self.device)
        if residual is not None:
            dense("residual", residual, x.shape, x.dtype, self.device)
        if y is not None:
            dense("y", y, x.shape, x.dtype, self.device)
        if weight is not None:
            dense("weight", weight, (dim,), torch.float32, self.device)
        if bias is not None:
            dense("bias", bias, (dim,), torch.float32, self.device)
        return launch(torch, self.device, stream, self._forward, x, weight, bias,
                      residual, eps, y, rows, dim, code)

    def _forward(self, s, x, weight, bias, residual, eps, y, rows, dim, code):
        torch = self._torch
        if y is None:
            y = torch.empty_like(x)
        total = None if residual is None else torch.empty_like(x)
        mean = torch.empty(rows, dtype=torch.float32, device=self.device)
        rstd = torch.empty(rows, dtype=torch.float32, device=self.device)
        _check(self._lib.ssm_layernorm_fwd(
            self.device.index, x.data_ptr(), ptr(residual), ptr(weight),
            ptr(bias), eps, y.data_ptr(), ptr(total), mean.data_ptr(),
            rstd.data_ptr(), rows, dim, code, s), "ssm_layernorm_fwd")
        return dict(y=y, sum=total, mean=mean, rstd=rstd)

    def backward(self, dy, x, mean, rstd, weight=None, bias=None, dsum=None,
                 stream=None):
        """Gradients of sum(dy * y) + sum(dsum * s). x: what was normed (the
        forward's sum where there was a residual); mean, rstd: the forward's.
        Returns a dict: dx (of x, and of the residual), dweight, dbias
        (float32; None without weight / bias)."""
        torch = self._torch
        code, rows, dim = self._rows(x)
        if dy is None or mean is None or rstd is None:
            raise ValueError("dy, mean and rstd are required")
        f32 = torch.float32
        dense("x", x, x.shape, x.dtype, self.device)
        dense("dy", dy, x.shape, x.dtype, self.device)
        if dsum is not None:
            dense("dsum", dsum, x.shape, x.dtype, self.device)
        dense("mean", mean, (rows,), f32, self.device)
        dense("rstd", rstd, (rows,), f32, self.device)
        if weight is not None:
            dense("weight", weight, (dim,), f32, self.device)
        if bias is not None:
            dense("bias", bias, (dim,), f32, self.device)
        return launch(torch, self.device, stream, self._backward, dy, x, mean, rstd,
                      weight, bias, dsum, rows, dim, code)

    def _backward(self, s, dy, x, mean, rstd, weight, bias, dsum, rows, dim,
                  code):
        torch = self._torch
        f = dict(dtype=torch.float32, device=self.device)
        dx = torch.empty_like(x)
        dweight = None if weight is None else torch.empty(dim, **f)
        dbias = None if bias is None else torch.empty(dim, **f)
        ws, n = None, 0
        if weight is not None or bias is not None:
            key = (rows, dim, code)
            n = self._bytes.get(key)
            if n is None:
                n = self._bytes[key] = ssm_layernorm_workspace(
                    self.device.index, rows, dim, code)
            ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        _check(self._lib.ssm_layernorm_bwd(
            self.device.index, dy.data_ptr(), x.data_ptr(), mean.data_ptr(),
            rstd.data_ptr(), ptr(weight), ptr(dsum), dx.data_ptr(),
            ptr(dweight), ptr(dbias), ptr(ws), n, rows, dim, code, s),
            "ssm_layernorm_bwd")
        return dict(dx=dx, dweight=dweight, dbias=dbias)
