"""The operators as a model uses them: norm with the residual, projections,
linear attention, a norm over each head, and the way back, against the same
block in float64 with torch's differentiation; then the block's tokens one at
a time."""
import pytest
import torch

import selective_state_space_51_b200 as S

pytestmark = pytest.mark.gpu


def recurrence(q, k, v, g, scale):
    """float64, token by token, differentiable."""
    b, L, H, dv = v.shape
    rep = H // q.shape[2]
    q, k = (t.repeat_interleave(rep, dim=2) for t in (q, k))
    state = torch.zeros(b, H, q.shape[-1], dv, dtype=torch.float64,
                        device=q.device)
    ys = []
    for t in range(L):
        state = state * g[:, t].exp()[..., None, None] \
            + k[:, t][..., None] * v[:, t][..., None, :]
        ys.append((q[:, t][..., None, :] @ state)[..., 0, :] * scale)
    return torch.stack(ys, 1), state


def test_a_block_forward_backward_and_decode():
    attn, norm = S.LinearAttention(0), S.LayerNorm(0)
    b, L, D, H, G, dk, dv = 2, 90, 64, 4, 2, 16, 24
    gen = torch.Generator(device="cuda").manual_seed(3)

    def rand(*s, scale=1.0):
        return torch.randn(*s, generator=gen, device="cuda") * scale

    x, r = rand(b, L, D), rand(b, L, D)
    w1, b1, w2, b2 = (1 + rand(D, scale=.2), rand(D, scale=.2),
                      1 + rand(dv, scale=.2), rand(dv, scale=.2))
    width = 2 * G * dk + H * dv + H
    W = rand(D, width, scale=D ** -0.5)
    dout, ds = rand(b, L, H, dv), rand(b, L, D)
    cuts = [0, G * dk, 2 * G * dk, 2 * G * dk + H * dv, width]

    def split(p):
        q, k, v, g = (p[..., i:j] for i, j in zip(cuts, cuts[1:]))
        return (q.unflatten(-1, (G, dk)), k.unflatten(-1, (G, dk)),
                v.unflatten(-1, (H, dv)), g)

    # ---- the framework's calls
    o1 = norm(x, weight=w1, bias=b1, residual=r)
    p = o1["y"] @ W
    q, k, v, graw = split(p)              # q, k, v: slices of one projection
    g = torch.nn.functional.logsigmoid(graw).contiguous()
    y, last = attn(q, k, v, log_decay=g)
    o2 = norm(y, weight=w2, bias=b2)
    g2 = norm.backward(dout, y, o2["mean"], o2["rstd"], weight=w2, bias=b2)
    ga = attn.backward(q, k, v, g2["dx"], log_decay=g)
    dp = torch.cat([ga["dq"].flatten(-2), ga["dk"].flatten(-2),
                    ga["dv"].flatten(-2),
                    ga["dlog_decay"] * torch.sigmoid(-graw)], -1)
    g1 = norm.backward(dp @ W.t(), o1["sum"], o1["mean"], o1["rstd"],
                       weight=w1, bias=b1, dsum=ds)
    dW = o1["y"].flatten(0, 1).t() @ dp.flatten(0, 1)

    # ---- float64
    leaf = [t.double().requires_grad_() for t in (x, r, w1, b1, w2, b2, W)]
    X, R, A1, B1, A2, B2, WW = leaf
    s = X + R
    h = torch.nn.functional.layer_norm(s, (D,), A1, B1, 1e-5)
    q6, k6, v6, g6 = split(h @ WW)
    g6 = torch.nn.functional.logsigmoid(g6)
    y6, last6 = recurrence(q6, k6, v6, g6, dk ** -0.5)
    o6 = torch.nn.functional.layer_norm(y6, (dv,), A2, B2, 1e-5)
    grads = torch.autograd.grad((o6 * dout).sum() + (s * ds).sum(), leaf)

    def near(a, ref, what):
        # float32 through six operators in a row, each within about 1e-5 of
        # its terms: 1e-4 of the result's size leaves the norms' division by
        # small deviations room; a wrong or missing term is of order 1
        err = (a.double() - ref).norm() / ref.norm()
        assert err <= 1e-4, (what, float(err))

    near(o2["y"], o6, "out")
    near(last, last6, "state")
    for a, ref, what in ((g1["dx"], grads[0], "dx"),
                         (g1["dx"], grads[1], "dresidual"),
                         (g1["dweight"], grads[2], "dw1"),
                         (g1["dbias"], grads[3], "db1"),
                         (g2["dweight"], grads[4], "dw2"),
                         (g2["dbias"], grads[5], "db2"),
                         (dW, grads[6], "dW")):
        near(a, ref, what)

    # ---- one token at a time, from the middle of the sequence
    half = 45
    _, state = attn(q[:, :half].contiguous(), k[:, :half].contiguous(),
                    v[:, :half].contiguous(),
                    log_decay=g[:, :half].contiguous())
    for t in range(half, L):
        yt = attn.step(q[:, t], k[:, t], v[:, t], state,
                       log_decay=g[:, t].contiguous())
        near(norm(yt, weight=w2, bias=b2)["y"], o6[:, t].detach(),
             "token %d" % t)
    near(state, last6.detach(), "state after the tokens")
