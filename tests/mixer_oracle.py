"""64-bit references of linear attention with a decay for each head and of
layer norm, token by token from the definitions, and the bounds their tests
hold the kernels to.

Every bound is arithmetic, not measurement. With u the half step of the output
type (2^-8 bfloat16, 2^-24 float32), a result r that is a sum of terms whose
absolute values add up to m (the same recurrence on |q|, |k|, |v|):
  - the last rounding is u |r|;
  - with bfloat16 and one plane, every term has one rounded factor (the score
    it is scaled by, or the state it is read from): 2^-8 m (1 + 2^-8);
  - float32 sums: a tensor-core instruction adds 16 products to its accumulator
    and may truncate, 2^-23 of the running sum; an output of one chunk goes
    through at most 6 (128 + 64 + 64) / 16 = 96 of them, and the state in front
    through 6 * 64 / 16 = 24 and one product more for each chunk: (100 + 25
    chunks) 2^-23 m. The exponentials add 2^-22 m for each chunk: 4 more. (A
    chunk here is 64 steps; one of 128 has 3 * 128 / 16 = 24 in its place.)
  - the decay's gradient beside bfloat16 may come of two planes: a scored or
    read term is then off by 2^-17 more, and its result is bfloat16.
"""
import numpy as np

CHUNK = 64
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def bf16(a):
    """Rounded to bfloat16 (to nearest even), as float64."""
    u = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32)
    u = (u + (((u >> 16) & 1) + 0x7FFF)) & np.uint32(0xFFFF0000)
    return u.view(np.float32).astype(np.float64)


def exponentials(g):
    with np.errstate(over="ignore"):
        a = np.exp(g)
    return np.where(g < -87.0, 0.0, a)


def forward(q, k, v, g, scale, h0=None, lengths=None):
    """y [b, L, H, dv] and the last state; q, k [b, L, G, dk], g [b, L, H]."""
    b, L, H, dv = v.shape
    G, dk = q.shape[2:]
    a = exponentials(g)
    y = np.zeros((b, L, H, dv))
    S = np.zeros((b, H, dk, dv)) if h0 is None else h0.astype(np.float64)
    S = S.copy()
    rep = H // G
    for i in range(b):
        n = L if lengths is None else int(np.clip(lengths[i], 0, L))
        for t in range(n):
            kk = np.repeat(k[i, t], rep, axis=0)
            qq = np.repeat(q[i, t], rep, axis=0)
            at = a[i, t][:, None, None]
            S[i] = np.where(at == 0, 0.0, at * S[i]) + \
                kk[:, :, None] * v[i, t][:, None, :]
            y[i, t] = scale * np.einsum("hk,hkv->hv", qq, S[i])
    return y, S


def backward(q, k, v, g, scale, dy, h0=None, dh_last=None, lengths=None,
             absolute=False):
    """Gradients, the adjoint recurrence token by token. With `absolute` (and
    inputs without signs) the decay's terms are added, not subtracted: what
    the bounds are proportional to."""
    b, L, H, dv = v.shape
    G, dk = q.shape[2:]
    rep = H // G
    a = exponentials(g)
    S = np.zeros((b, H, dk, dv)) if h0 is None else h0.astype(np.float64)
    dqh = np.zeros((b, L, H, dk))
    dkh = np.zeros((b, L, H, dk))
    out = dict(dv=np.zeros((b, L, H, dv)), dg=np.zeros((b, L, H)),
               dh0=np.zeros((b, H, dk, dv)))
    for i in range(b):
        n = L if lengths is None else int(np.clip(lengths[i], 0, L))
        states = [S[i].copy()]
        for t in range(n):
            kk = np.repeat(k[i, t], rep, axis=0)
            at = a[i, t][:, None, None]
            states.append(np.where(at == 0, 0.0, at * states[-1])
                          + kk[:, :, None] * v[i, t][:, None, :])
        M = (np.zeros((H, dk, dv)) if dh_last is None
             else dh_last[i].astype(np.float64))
        run = (states[n] * M).sum((1, 2))
        for t in reversed(range(n)):
            qq = np.repeat(q[i, t], rep, axis=0)
            kk = np.repeat(k[i, t], rep, axis=0)
            M = M + scale * qq[:, :, None] * dy[i, t][:, None, :]
            dqh[i, t] = scale * np.einsum("hkv,hv->hk", states[t + 1],
                                          dy[i, t])
            dkh[i, t] = np.einsum("hkv,hv->hk", M, v[i, t])
            out["dv"][i, t] = np.einsum("hk,hkv->hv", kk, M)
            at = a[i, t][:, None, None]
            if absolute:
                run = run + (qq * dqh[i, t]).sum(1) + (kk * dkh[i, t]).sum(1)
                out["dg"][i, t] = run
            else:
                # <a S_{t-1}, M>, the definition
                out["dg"][i, t] = (np.where(at == 0, 0.0, at * states[t])
                                   * M).sum((1, 2))
            M = np.where(at == 0, 0.0, at * M)
        out["dh0"][i] = M
    out["dq"] = dqh.reshape(b, L, G, rep, dk).sum(3)
    out["dk"] = dkh.reshape(b, L, G, rep, dk).sum(3)
    out["dhead"] = out["dg"].sum((0, 1))
    return out


def bound(ref, mag, dtype, L, planes_exact=False, out_dtype=None):
    """Elementwise bound of the module's docstring."""
    chunks = -(-L // CHUNK)
    tol = U[out_dtype or dtype] * np.abs(ref)
    tol = tol + (104 + 29 * chunks) * 2.0 ** -23 * mag
    if dtype == "bf16" and not planes_exact:
        tol = tol + 2.0 ** -8 * (1 + 2.0 ** -8) * mag
    return tol + 1e-30


def check(got, ref, tol, what):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), "%s has non-finite values" % what
    over = np.abs(got - ref) / tol
    assert over.size == 0 or over.max() <= 1.0, \
        "%s: %.2f times its bound (at %s)" % (
            what, over.max(), np.unravel_index(over.argmax(), over.shape))
    return float(over.max()) if over.size else 0.0


def norm_forward(x, residual, weight, bias, eps, rounded):
    s = x if residual is None else rounded(x + residual)
    mean = s.mean(1)
    rstd = 1.0 / np.sqrt(((s - mean[:, None]) ** 2).mean(1) + eps)
    y = (s - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return s, mean, rstd, y


def norm_backward(dy, s, mean, rstd, weight, dsum):
    xhat = (s - mean[:, None]) * rstd[:, None]
    u = dy if weight is None else dy * weight
    dx = rstd[:, None] * (u - u.mean(1, keepdims=True)
                          - xhat * (u * xhat).mean(1, keepdims=True))
    if dsum is not None:
        dx = dx + dsum
    return dx, (dy * xhat).sum(0), dy.sum(0)
