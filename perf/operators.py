"""Measured cases of the operators beside the selective scan: linear attention
with a decay for each head (prompt, single token, backward) and layer norm with
the residual sum in front (forward, backward).

`own` selects what `run` does: False computes the plain form from elementary
torch operations, True makes the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"
CHUNK = 64          # steps per chunk of the plain chunked form
EPS = 1e-5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a prompt through a mixer of the 2.8B layer's width (40 heads of 128)
        dict(name="prompt_wide_bf16", op="prompt", dtype="bf16", batch=4,
             seqlen=8192, heads=40, groups=40, dk=128, dv=128, gate="token",
             ragged=False, state=False),
        # the 130M layer's width (24 heads of 64), q and k shared by all heads
        dict(name="prompt_shared_bf16", op="prompt", dtype="bf16", batch=8,
             seqlen=2048, heads=24, groups=1, dk=128, dv=64, gate="token",
             ragged=False, state=False),
        # the classifier's batch in float32, padded to the longest sequence
        dict(name="prompt_padded_f32", op="prompt", dtype="f32", batch=64,
             seqlen=512, heads=8, groups=8, dk=64, dv=64, gate="head",
             ragged=True, state=False),
        # one long document continued from an earlier state: few heads
        dict(name="prompt_long_bf16", op="prompt", dtype="bf16", batch=1,
             seqlen=65536, heads=8, groups=8, dk=128, dv=128, gate="both",
             ragged=False, state=True),
        # one sequence's next token: latency
        dict(name="step_one_bf16", op="step", dtype="bf16", batch=1,
             seqlen=1, heads=40, groups=40, dk=128, dv=128, gate="token",
             ragged=False, state=True),
        # a serving batch's next tokens: the states' bytes
        dict(name="step_batch_bf16", op="step", dtype="bf16", batch=256,
             seqlen=1, heads=40, groups=8, dk=128, dv=128, gate="token",
             ragged=False, state=True),
        # a training step's backward at the 130M layer's width
        dict(name="backward_bf16", op="backward", dtype="bf16", batch=8,
             seqlen=2048, heads=24, groups=24, dk=64, dv=64, gate="token",
             ragged=False, state=False),
        # float32, shared heads, odd sizes, padded, a learned decay per head
        dict(name="backward_odd_f32", op="backward", dtype="f32", batch=3,
             seqlen=1000, heads=6, groups=2, dk=48, dv=77, gate="both",
             ragged=True, state=True),
        # the norm in front of a mixer, 2.8B model width, with the residual
        dict(name="norm_wide_bf16", op="norm", dtype="bf16", rows=32768,
             dim=2560, residual=True, affine=True),
        # the norm of each head's output, as one decoding batch has it
        dict(name="norm_heads_f32", op="norm", dtype="f32", rows=4000, dim=77,
             residual=False, affine=True),
        # its backward pass in training
        dict(name="norm_back_wide_bf16", op="norm_back", dtype="bf16",
             rows=32768, dim=2560, residual=True, affine=True),
        # float32 at the classifier's tokens, odd width
        dict(name="norm_back_odd_f32", op="norm_back", dtype="f32",
             rows=32768, dim=511, residual=False, affine=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(
        rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "prompt", "step", "backward",
                     "backward", "norm", "norm_back"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op in ("norm", "norm_back"):
        dim = _log_int(rng, 16, 8192)
        return dict(op=op, dtype=dtype,
                    rows=_log_int(rng, 1, max(1, 50_000_000 // dim)), dim=dim,
                    residual=rng.random() < 0.5, affine=rng.random() < 0.8)
    groups = rng.choice((1, 1, 2, 3, 4, 8))
    heads = groups * rng.choice((1, 1, 2, 4, 5))
    size = lambda: (rng.choice((32, 64, 64, 128, 128))  # noqa: E731
                    if rng.random() < 0.6 else rng.randint(8, 128))
    case = dict(op=op, dtype=dtype, batch=0, seqlen=1, heads=heads,
                groups=groups, dk=size(), dv=size(),
                gate=rng.choice(("token", "head", "both")),
                ragged=op != "step" and rng.random() < 0.3,
                state=op == "step" or rng.random() < 0.5)
    if op == "step":
        case["batch"] = _log_int(rng, 1, 10000 // heads)
        return case
    most = 300_000 if op == "prompt" else 120_000   # tokens times heads
    case["seqlen"] = _log_int(rng, 1, most // heads)
    case["batch"] = _log_int(rng, 1, max(1, min(
        64, most // heads // case["seqlen"])))
    return case


# ---------------------------------------------------------------- inputs

def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    ty = _type(case)

    def normal(*shape, scale=1.0, dtype=ty):
        return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)

    f32 = torch.float32
    st = dict(case=dict(case))
    if case["op"] in ("norm", "norm_back"):
        r, d = case["rows"], case["dim"]
        # a residual stream: each channel with its own offset and size
        offset = normal(d, scale=0.5, dtype=f32)
        st["x"] = (normal(r, d, dtype=f32) + offset).to(ty)
        st["residual"] = normal(r, d) if case["residual"] else None
        st["weight"] = (1 + normal(d, scale=0.2, dtype=f32)
                        if case["affine"] else None)
        st["bias"] = normal(d, scale=0.2, dtype=f32) if case["affine"] else None
        if case["op"] == "norm_back":
            # what the forward pass kept: the sum (in x) and its statistics
            st["dsum"] = st.pop("residual")
            x = st["x"].double()
            st["mean"] = x.mean(1).float()
            st["rstd"] = (x.var(1, unbiased=False) + EPS).rsqrt().float()
            st["dy"] = normal(r, d)
        return st
    b, L, H, G = (case[k] for k in ("batch", "seqlen", "heads", "groups"))
    dk, dv = case["dk"], case["dv"]
    one = case["op"] == "step"
    tok = (b,) if one else (b, L)
    st["q"] = normal(*tok, G, dk)
    st["k"] = normal(*tok, G, dk, scale=dk ** -0.5)
    st["v"] = normal(*tok, H, dv)
    # log decay: a rate a head, log-uniform over memories of about 1 to 1000
    # steps; the token's part varies around it
    rate = torch.exp(torch.rand(H, generator=gen, device=DEV)
                     * math.log(1000.0) - math.log(1000.0))
    gate = case["gate"]
    st["head_log_decay"] = -rate if gate in ("head", "both") else None
    st["log_decay"] = None
    if gate in ("token", "both"):
        st["log_decay"] = (-rate * torch.nn.functional.softplus(
            torch.randn(*tok, H, generator=gen, device=DEV))).to(ty)
    st["scale"] = dk ** -0.5
    st["h0"] = (normal(b, H, dk, dv, scale=0.5, dtype=f32)
                if case["state"] else None)
    st["lengths"] = None
    if case["ragged"]:
        # short to full; the first sequence is empty, the last is full
        n = torch.randint(0, L + 1, (b,), generator=gen, device=DEV)
        n[0], n[-1] = 0, L
        st["lengths"] = n.to(torch.int32)
    if case["op"] == "backward":
        st["dy"] = normal(b, L, H, dv)
        st["dh_last"] = (normal(b, H, dk, dv, scale=0.5, dtype=f32)
                         if case["state"] else None)
    return st


# ---------------------------------------------------------------- the calls

_HANDLES = {}


def _handle(name):
    """The framework's object a program makes once and keeps."""
    if name not in _HANDLES:
        import selective_state_space_51_b200 as S
        _HANDLES[name] = getattr(S, name)(0)
    return _HANDLES[name]


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_prompt(s):
    return _handle("LinearAttention")(
        s["q"], s["k"], s["v"], log_decay=s["log_decay"],
        head_log_decay=s["head_log_decay"], scale=s["scale"],
        lengths=s["lengths"], h0=s["h0"])


def _own_step(s):
    y = _handle("LinearAttention").step(
        s["q"], s["k"], s["v"], s["h0"], log_decay=s["log_decay"],
        head_log_decay=s["head_log_decay"], scale=s["scale"])
    return y, s["h0"]


def _own_backward(s):
    return _handle("LinearAttention").backward(
        s["q"], s["k"], s["v"], s["dy"], log_decay=s["log_decay"],
        head_log_decay=s["head_log_decay"], scale=s["scale"],
        lengths=s["lengths"], h0=s["h0"], dh_last=s["dh_last"])


def _own_norm(s):
    return _handle("LayerNorm")(s["x"], weight=s["weight"], bias=s["bias"],
                                residual=s["residual"], eps=EPS)


def _own_norm_back(s):
    return _handle("LayerNorm").backward(
        s["dy"], s["x"], s["mean"], s["rstd"], weight=s["weight"],
        bias=s["bias"], dsum=s["dsum"])


_OWN = dict(prompt=_own_prompt, step=_own_step, backward=_own_backward,
            norm=_own_norm, norm_back=_own_norm_back)


# ---------------------------------------------------------------- plain forms

def _heads_first(x, heads, n):
    """[b, L, h, d] -> float32 [b, heads, n chunks, CHUNK, d], zero-padded."""
    x = x.float().transpose(1, 2)
    if x.shape[1] != heads:
        x = x.repeat_interleave(heads // x.shape[1], dim=1)
    pad = n * CHUNK - x.shape[2]
    if pad:
        x = torch.nn.functional.pad(x, (0, 0, 0, pad))
    return x.reshape(x.shape[0], heads, n, CHUNK, x.shape[-1])


def _tokens_first(x, L):
    """The reverse of _heads_first, without the sum over a group."""
    b, h, n, c, d = x.shape
    return x.reshape(b, h, n * c, d)[:, :, :L].transpose(1, 2)


def _chunked(s):
    """What the forward and the backward of the chunked form share."""
    c = s["case"]
    b, L, H = c["batch"], c["seqlen"], c["heads"]
    n = -(-L // CHUNK)
    keep = None
    q, k, v = s["q"], s["k"], s["v"]
    g = torch.zeros(b, L, H, device=DEV)
    if s["log_decay"] is not None:
        g = g + s["log_decay"].float()
    if s["head_log_decay"] is not None:
        g = g + s["head_log_decay"]
    if s["lengths"] is not None:
        keep = (torch.arange(L, device=DEV)[None] < s["lengths"][:, None]
                )[..., None, None]
        zero = torch.zeros((), device=DEV)
        q, k, v = (torch.where(keep, t.float(), zero) for t in (q, k, v))
        g = torch.where(keep[..., 0], g, zero)
    q, k, v = (_heads_first(t, H, n) for t in (q, k, v))
    g = _heads_first(g[..., None], H, n)[..., 0]
    cum = g.cumsum(-1)                                  # inside the chunk
    tot = cum[..., -1:]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(
        ~low, -math.inf))
    # over the chunks: sums of many terms, in 64 bits
    T = tot[..., 0].double().cumsum(-1)
    before = T - tot[..., 0].double()
    earlier = torch.ones(n, n, dtype=torch.bool, device=DEV).tril(-1)
    between = torch.exp((before[..., :, None] - T[..., None, :]).masked_fill(
        ~earlier, -math.inf)).float()
    return dict(b=b, L=L, H=H, n=n, keep=keep, q=q, k=k, v=v, cum=cum, tot=tot,
                decay=decay, T=T, before=before, between=between)


def _states(f, h0):
    """The state in front of each chunk and the last one."""
    dk, dv = f["k"].shape[-1], f["v"].shape[-1]
    write = (f["k"] * torch.exp(f["tot"] - f["cum"])[..., None]).transpose(
        -1, -2) @ f["v"]
    flat = write.reshape(f["b"], f["H"], f["n"], dk * dv)
    S = f["between"] @ flat
    if h0 is not None:
        S = S + torch.exp(f["before"]).float()[..., None] * h0.reshape(
            f["b"], f["H"], 1, dk * dv)
    last = S[:, :, -1] * torch.exp(f["tot"][:, :, -1]) + flat[:, :, -1]
    return (S.reshape(f["b"], f["H"], f["n"], dk, dv),
            last.reshape(f["b"], f["H"], dk, dv))


def _plain_prompt(s):
    f = _chunked(s)
    S, last = _states(f, s["h0"])
    y = ((f["q"] @ f["k"].transpose(-1, -2)) * f["decay"]) @ f["v"]
    y = y + (f["q"] * torch.exp(f["cum"])[..., None]) @ S
    y = _tokens_first(y, f["L"]) * s["scale"]
    if f["keep"] is not None:
        y = torch.where(f["keep"], y, torch.zeros((), device=DEV))
    return y.to(s["v"].dtype).contiguous(), last


def _plain_step(s):
    H, G = s["case"]["heads"], s["case"]["groups"]
    q, k = (t.float().repeat_interleave(H // G, dim=1)
            for t in (s["q"], s["k"]))
    g = torch.zeros(s["v"].shape[:2], device=DEV)
    if s["log_decay"] is not None:
        g = g + s["log_decay"].float()
    if s["head_log_decay"] is not None:
        g = g + s["head_log_decay"]
    S = s["h0"]
    S.mul_(torch.exp(g)[..., None, None])
    S.addcmul_(k[..., None], s["v"].float()[..., None, :])
    y = (q[..., None, :] @ S)[..., 0, :] * s["scale"]
    return y.to(s["v"].dtype), S


def _plain_backward(s):
    f = _chunked(s)
    ty, scale = s["v"].dtype, s["scale"]
    q, k, v = f["q"], f["k"], f["v"]
    dk, dv = k.shape[-1], v.shape[-1]
    dy = s["dy"]
    if f["keep"] is not None:
        dy = torch.where(f["keep"], dy.float(), torch.zeros((), device=DEV))
    dy = _heads_first(dy, f["H"], f["n"]) * scale
    S, last = _states(f, s["h0"])
    # the gradient of the state behind each chunk, and of the first state
    read = (q * torch.exp(f["cum"])[..., None]).transpose(-1, -2) @ dy
    flat = read.reshape(f["b"], f["H"], f["n"], dk * dv)
    G = f["between"].transpose(-1, -2) @ flat
    dh0 = (torch.exp(f["before"]).float()[..., None] * flat).sum(2)
    dlast = s["dh_last"]
    if dlast is not None:
        end = f["T"][..., -1:]
        G = G + torch.exp(end - f["T"]).float()[..., None] * dlast.reshape(
            f["b"], f["H"], 1, dk * dv)
        dh0 = dh0 + torch.exp(end).float() * dlast.reshape(
            f["b"], f["H"], dk * dv)
    G = G.reshape(f["b"], f["H"], f["n"], dk, dv)
    dh0 = dh0.reshape(f["b"], f["H"], dk, dv)
    dP = (dy @ v.transpose(-1, -2)) * f["decay"]
    P = (q @ k.transpose(-1, -2)) * f["decay"]
    into = torch.exp(f["cum"])[..., None]
    out = torch.exp(f["tot"] - f["cum"])[..., None]
    gq = dP @ k + into * (dy @ S.transpose(-1, -2))
    gk = dP.transpose(-1, -2) @ q + out * (v @ G.transpose(-1, -2))
    gv = P.transpose(-1, -2) @ dy + out * (k @ G)
    # the log decay's gradient: summed backwards from each chunk's end, where
    # it is the product of the state and the state's gradient
    r = (q * gq).sum(-1) - (k * gk).sum(-1)
    ends = torch.cat([S[:, :, 1:], last[:, :, None]], 2)
    gg = r.flip(-1).cumsum(-1).flip(-1) + (ends * G).sum((-1, -2))[..., None]
    gq, gk, gv, gg = (_tokens_first(t, f["L"])
                      for t in (gq, gk, gv, gg[..., None]))
    if f["keep"] is not None:
        gg = torch.where(f["keep"], gg, torch.zeros((), device=DEV))
    gg = gg[..., 0]
    b, L, n_groups = f["b"], f["L"], s["case"]["groups"]
    gq, gk = (t.reshape(b, L, n_groups, -1, dk).sum(3) for t in (gq, gk))
    return dict(
        dq=gq.to(ty).contiguous(), dk=gk.to(ty).contiguous(),
        dv=gv.to(ty).contiguous(),
        dlog_decay=None if s["log_decay"] is None else gg.to(ty).contiguous(),
        dhead_log_decay=None if s["head_log_decay"] is None
        else gg.double().sum((0, 1)).float(),
        dh0=dh0)


def _plain_norm(s):
    x = s["x"]
    if s["residual"] is not None:
        # the sum is the residual stream: held, and normed, in its type
        x = (x.float() + s["residual"].float()).to(x.dtype)
    f = x.float()
    mean = f.mean(1, keepdim=True)
    d = f - mean
    rstd = (d.square().mean(1, keepdim=True) + EPS).rsqrt()
    y = d * rstd
    if s["weight"] is not None:
        y = y * s["weight"] + s["bias"]
    return dict(y=y.to(x.dtype), mean=mean[:, 0], rstd=rstd[:, 0],
                sum=x if s["residual"] is not None else None)


def _plain_norm_back(s):
    dy = s["dy"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    w = dy if s["weight"] is None else dy * s["weight"]
    dx = (w - w.mean(1, keepdim=True)
          - xhat * (w * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    affine = s["weight"] is not None
    return dict(dx=dx.to(s["x"].dtype),
                dweight=(dy * xhat).sum(0) if affine else None,
                dbias=dy.sum(0) if affine else None)


_PLAIN = dict(prompt=_plain_prompt, step=_plain_step, backward=_plain_backward,
              norm=_plain_norm, norm_back=_plain_norm_back)


# ---------------------------------------------------------------- work

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_back"):
        n, d = case["rows"] * case["dim"], case["dim"]
        moved = 2 + 2 * case["residual"]                 # x, y; residual, sum
        if case["op"] == "norm_back":
            moved = 3 + case["residual"]                 # dy, x, dx; dsum
        params = (4 if case["op"] == "norm_back" else 2) * case["affine"]
        return {"bytes": n * e * moved + 8 * case["rows"] + 4 * d * params,
                "flops": n * (10 if case["op"] == "norm_back" else 8)}
    b, L, H, G = (case[k] for k in ("batch", "seqlen", "heads", "groups"))
    dk, dv = case["dk"], case["dv"]
    t = b * L
    gate = H * (case["gate"] != "head")
    state = 4 * b * H * dk * dv
    if case["op"] == "step":
        return {"bytes": t * e * (2 * G * dk + 2 * H * dv + gate) + 2 * state,
                "flops": 5 * t * H * dk * dv}
    if case["op"] == "prompt":
        return {"bytes": t * e * (2 * G * dk + 2 * H * dv + gate)
                + state * (1 + case["state"]),
                "flops": 4 * t * H * dk * dv}
    return {"bytes": t * e * (4 * G * dk + 3 * H * dv + 2 * gate)
            + state * (1 + 2 * case["state"]),
            "flops": 10 * t * H * dk * dv}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "norm_back":
        return _exact_norm_back(s)
    return _exact_recurrence(s)


def _exact_norm(s):
    x = s["x"].double()
    if s["residual"] is not None:
        x = (x + s["residual"].double()).to(s["x"].dtype).double()
    var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
    rstd = 1 / torch.sqrt(var + EPS)
    y = (x - mean) * rstd
    if s["weight"] is not None:
        y = y * s["weight"].double() + s["bias"].double()
    return dict(y=y, mean=mean[:, 0], rstd=rstd[:, 0],
                sum=x if s["residual"] is not None else None)


def _exact_norm_back(s):
    """Through the Jacobian's three terms, from the kept statistics."""
    n = s["x"].shape[1]
    dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
    hat = (s["x"].double() - s["mean"].double()[:, None]) * rstd
    up = dy if s["weight"] is None else torch.einsum(
        "rd,d->rd", dy, s["weight"].double())
    along = torch.einsum("rd,rd->r", up, hat)[:, None]
    dx = rstd * up - rstd * up.sum(1, keepdim=True) / n - rstd * hat * along / n
    if s["dsum"] is not None:
        dx += s["dsum"].double()
    affine = s["weight"] is not None
    return dict(dx=dx,
                dweight=torch.einsum("rd,rd->d", dy, hat) if affine else None,
                dbias=torch.einsum("rd->d", dy) if affine else None)


def _exact_recurrence(s):
    """Token by token: S = a S + k v^T, y = scale q S, and the adjoint."""
    c = s["case"]
    b, L, H, G = (c[k] for k in ("batch", "seqlen", "heads", "groups"))
    dk, dv, R = c["dk"], c["dv"], H // G
    one = c["op"] == "step"
    back = c["op"] == "backward"
    per = lambda x: x.double().reshape(b, L, x.shape[-2], -1)  # noqa: E731
    q, k, v = per(s["q"]), per(s["k"]), per(s["v"])
    g = torch.zeros(b, L, H, dtype=torch.float64, device=DEV)
    if s["log_decay"] is not None:
        g += s["log_decay"].double().reshape(b, L, H)
    if s["head_log_decay"] is not None:
        g += s["head_log_decay"].double()
    live = torch.ones(b, L, dtype=torch.bool, device=DEV)
    if s["lengths"] is not None:
        live = torch.arange(L, device=DEV)[None] < s["lengths"][:, None]
    a = torch.where(live[..., None], g, 0.0).exp()
    dead = ~live[..., None, None]
    q, k, v = (t.masked_fill(dead, 0.0) for t in (q, k, v))
    S = (torch.zeros(b, H, dk, dv, dtype=torch.float64, device=DEV)
         if s["h0"] is None else s["h0"].double().clone())
    heads = lambda x: (x[:, :, None].expand(b, G, R, dk)  # noqa: E731
                       .reshape(b, H, dk))
    if back:
        dy = (s["dy"].double() * s["scale"]).masked_fill(dead, 0.0)
    out = torch.empty(b, L, H, dk if back else dv, dtype=torch.float64,
                      device=DEV)
    for t in range(L):
        S.mul_(a[:, t, :, None, None])
        S.addcmul_(heads(k[:, t])[..., None], v[:, t][:, :, None])
        if back:      # the gradient of q reads the state, as y does
            out[:, t] = (S @ dy[:, t][..., None])[..., 0]
        else:
            out[:, t] = (heads(q[:, t])[:, :, None] @ S)[:, :, 0] * s["scale"]
    if not back:
        return (out[:, 0] if one else out), S
    gq, gk, gv = out, torch.empty_like(out), torch.empty_like(v)
    M = (torch.zeros_like(S) if s["dh_last"] is None
         else s["dh_last"].double().clone())
    gg = torch.empty_like(g)
    run = (S * M).sum((-1, -2))
    for t in reversed(range(L)):
        M.addcmul_(heads(q[:, t])[..., None], dy[:, t][:, :, None])
        gk[:, t] = (M @ v[:, t][..., None])[..., 0]
        gv[:, t] = (heads(k[:, t])[:, :, None] @ M)[:, :, 0]
        run = (run + (heads(q[:, t]) * gq[:, t]).sum(-1)
               - (heads(k[:, t]) * gk[:, t]).sum(-1))
        gg[:, t] = run
        M.mul_(a[:, t, :, None, None])
    gg = gg.masked_fill(~live[..., None], 0.0)
    gv, gq, gk = (t.masked_fill(dead, 0.0) for t in (gv, gq, gk))
    return dict(dq=gq.reshape(b, L, G, R, dk).sum(3),
                dk=gk.reshape(b, L, G, R, dk).sum(3), dv=gv,
                dlog_decay=None if s["log_decay"] is None else gg,
                dhead_log_decay=None if s["head_log_decay"] is None
                else gg.sum((0, 1)), dh0=M)
