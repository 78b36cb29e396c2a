"""A workspace that lies over a buffer of its own call is refused before
anything is launched (each buffer here is a view of one allocation that holds
the whole workspace)."""
import pytest
import torch

import selective_state_space_51_b200 as S

pytestmark = pytest.mark.gpu


def over(n, like):
    """A buffer of n bytes and a tensor like `like` inside it."""
    whole = torch.zeros(n + like.numel() * like.element_size() + 512,
                        dtype=torch.uint8, device="cuda")
    part = whole[256:256 + like.numel() * like.element_size()]
    return whole, part.view(like.dtype).view(like.shape)


def test_layer_norm():
    rows, dim = 500, 256
    n = S.ssm_layernorm_workspace(0, rows, dim, S.SSM_F32)
    a = {k: torch.zeros(rows, dim, device="cuda") for k in
         ("dy", "x", "dsum", "dx")}
    a.update({k: torch.zeros(rows, device="cuda") for k in ("mean", "rstd")})
    a.update({k: torch.zeros(dim, device="cuda") for k in
              ("weight", "dweight", "dbias")})
    apart = torch.zeros(n, dtype=torch.uint8, device="cuda")

    def call(ws, **kw):
        b = {**a, **kw}
        return S.ssm_layernorm_bwd(
            0, b["dy"], b["x"], b["mean"], b["rstd"], b["weight"], b["dsum"],
            b["dx"], b["dweight"], b["dbias"], ws, n, rows, dim, S.SSM_F32,
            check=False)

    assert call(apart) == S.SSM_OK
    for k in a:
        whole, part = over(n, a[k])
        assert call(whole, **{k: part}) == S.SSM_ERR_INVALID, k
    # none is needed: what is passed is not looked at
    assert call(a["x"], dweight=None, dbias=None) == S.SSM_OK
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [S.SSM_F32, S.SSM_BF16])
def test_linear_attention(dtype):
    ty = torch.float32 if dtype == S.SSM_F32 else torch.bfloat16
    b, L, H, G, dk, dv = 1, 1200, 4, 2, 64, 64
    dims = (b, L, H, G, dk, dv, 0, 0, 0)
    z = lambda *s, t=ty: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    f32 = torch.float32
    a = dict(q=z(b, L, G, dk), k=z(b, L, G, dk), v=z(b, L, H, dv),
             log_decay=z(b, L, H), head=z(H, t=f32),
             lengths=torch.full((b,), L, dtype=torch.int32, device="cuda"),
             h0=z(b, H, dk, dv, t=f32))
    fwd = dict(a, y=z(b, L, H, dv), h_last=z(b, H, dk, dv, t=f32))
    bwd = dict(a, dy=z(b, L, H, dv), dh_last=z(b, H, dk, dv, t=f32),
               dq=z(b, L, G, dk), dk=z(b, L, G, dk), dv=z(b, L, H, dv),
               dlog=z(b, L, H), dhead=z(H, t=f32), dh0=z(b, H, dk, dv, t=f32))

    def forward(ws, n, c):
        return S.ssm_linattn_fwd(
            0, c["q"], c["k"], c["v"], c["log_decay"], c["head"], 1.0,
            c["lengths"], c["h0"], c["y"], c["h_last"], ws, n, dims, dtype,
            check=False)

    def backward(ws, n, c):
        return S.ssm_linattn_bwd(
            0, c["q"], c["k"], c["v"], c["log_decay"], c["head"], 1.0,
            c["lengths"], c["h0"], c["dy"], c["dh_last"], c["dq"], c["dk"],
            c["dv"], c["dlog"], c["dhead"], c["dh0"], ws, n, dims, dtype,
            check=False)

    for call, args, back in ((forward, fwd, False), (backward, bwd, True)):
        n = S.ssm_linattn_workspace(0, dims, dtype, back)
        assert n > 0
        assert call(z(n, t=torch.uint8), n, args) == S.SSM_OK
        for k in args:
            whole, part = over(n, args[k])
            assert call(whole, n, {**args, k: part}) == S.SSM_ERR_INVALID, k
    torch.cuda.synchronize()
    assert S.ssm_linattn_sync_status(0) == S.SSM_OK


NONE = 1 + S.SSM_LINATTN_NO_DECAY_GRADIENT
TOKENS, HEADS = 1 + S.SSM_LINATTN_NO_HEAD_GRADIENT, 1


@pytest.mark.parametrize("dtype", [S.SSM_F32, S.SSM_BF16])
@pytest.mark.parametrize("d", [64, 128, 45])
@pytest.mark.parametrize("kind", [NONE, TOKENS, HEADS])
def test_what_is_asked_for_is_enough_and_no_more(dtype, d, kind):
    """A backward call runs in the workspace of its kind; the states that a
    float32 gradient of the decay is anchored to, one for 128 steps, are in the
    workspace of calls that have one only."""
    ty = torch.float32 if dtype == S.SSM_F32 else torch.bfloat16
    b, L, H = 1, 4096, 160
    dims = (b, L, H, H, d, d, 0, 0, 0)
    sizes = {k: S.ssm_linattn_workspace(0, dims, dtype, k)
             for k in (NONE, TOKENS, HEADS)}
    assert sizes[NONE] <= sizes[TOKENS] <= sizes[HEADS]
    assert S.ssm_linattn_workspace(0, dims, dtype, True) == sizes[HEADS]
    pad = 64 if d <= 64 else 128
    anchors = 2 * H * (L // 128) * pad * pad * 4
    # (and as many segments' states as there may be: three of each)
    segments = 3 * H * (L // 2048) * pad * pad * 4
    rows = 2 * H * L * 2 * (pad // 64) * 4
    exact = kind == HEADS or (dtype == S.SSM_F32 and kind == TOKENS)
    assert (sizes[kind] >= anchors) == exact
    assert sizes[kind] <= exact * anchors + 2 * segments + rows + (1 << 24)
    z = lambda *s, t=ty: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    q = z(b, L, H, d)
    out = [torch.empty_like(q) for _ in range(3)]
    log, head = z(b, L, H), z(H, t=torch.float32)
    n = sizes[kind]
    rc = S.ssm_linattn_bwd(
        0, q, q, q, log, head, 1.0, None, None, q, None, *out,
        None if kind == NONE else torch.empty_like(log),
        torch.empty_like(head) if kind == HEADS else None, None,
        z(max(n, 1), t=torch.uint8) if n else None, n, dims, dtype,
        check=False)
    torch.cuda.synchronize()
    assert rc == S.SSM_OK


def test_the_class_asks_for_what_it_needs():
    """128-wide bfloat16 heads with the tokens' decay gradient: no anchors."""
    attn = S.LinearAttention(0)
    b, L, H, d = 1, 4096, 160, 128
    q = torch.zeros(b, L, H, d, dtype=torch.bfloat16, device="cuda")
    log = q[..., 0].contiguous()
    attn.backward(q, q, q, q, log_decay=log)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    g = attn.backward(q, q, q, q, log_decay=log)
    torch.cuda.synchronize()
    kept = torch.cuda.memory_allocated() - before
    used = torch.cuda.max_memory_allocated() - before
    anchors = 2 * H * (L // 128) * d * d * 4
    assert used - kept < anchors / 2
    del g
