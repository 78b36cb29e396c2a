"""Keys and values of 128 with bfloat16, where the tensor-memory kernel has one
q in place of two and y in the place of k: padded batches, cut sequences,
restarts, shared heads, several calls at once, replays."""
import numpy as np
import pytest
import torch

import mixer_oracle as M
import selective_state_space_51_b200 as S
from test_gpu_linattn import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    return S.LinearAttention(0)


def case(b, L, H, G, dk=128, dv=128, **kw):
    return Case("bf16", b, L, H, G, dk, dv, gate="token", **kw)


@pytest.mark.parametrize("L", [1, 127, 128, 129, 255, 256, 257, 383, 384, 385,
                               511, 640])
@pytest.mark.parametrize("dk,dv", [(128, 128), (72, 128), (128, 72),
                                   (120, 104)])
def test_chunks(attn, L, dk, dv):
    c = case(1, L, 2, 2, dk, dv, rate=0.05)
    c.check_forward(*c.run(attn))
    c.check_backward(c.run_back(attn))
    assert attn.sync_status() == S.SSM_OK


@pytest.mark.parametrize("groups", [1, 2])
@pytest.mark.parametrize("lengths", [[400, 0, 1, 399, 256, 130],
                                     [128, 127, 129, 383]])
def test_padded_batches(attn, groups, lengths):
    """Neither the rows behind a sequence nor what they hold matter."""
    c = case(len(lengths), 400, 2, groups, lengths=lengths)
    y0, h0 = c.run(attn)
    c.check_forward(y0, h0)
    g0 = c.run_back(attn)
    c.check_backward(g0)
    for i, n in enumerate(lengths):
        for a in (c.q, c.k, c.v, c.log_decay, c.dy):
            a[i, n:] = np.nan
            a[i, n + 1:] = np.inf
    y1, h1 = c.run(attn)
    g1 = c.run_back(attn)
    assert torch.equal(y0, y1) and torch.equal(h0, h1)
    for k in g0:
        assert g0[k] is None or torch.equal(g0[k], g1[k]), k
    for i, n in enumerate(lengths):
        assert not y1[i, n:].any() and not g1["dv"][i, n:].any()
        assert not g1["dk"][i, n:].any() and not g1["dlog_decay"][i, n:].any()
    assert attn.sync_status() == S.SSM_OK


@pytest.mark.parametrize("L,lengths", [(3000, None), (2500, [2049]),
                                       (5000, [4111])])
def test_cut_sequences(attn, L, lengths):
    c = case(1, L, 1, 1, lengths=lengths, rate=0.02)
    c.check_forward(*c.run(attn))
    c.check_backward(c.run_back(attn))


def test_more_heads_than_multiprocessors(attn):
    heads = torch.cuda.get_device_properties(0).multi_processor_count + 3
    c = case(1, 1100, heads, heads, 72, 72, state=False)
    c.check_forward(*c.run(attn))


def test_restarts(attn):
    c = case(2, 700, 2, 2)
    for t in (0, 1, 10, 63, 64, 127, 128, 255, 256, 511, 699):
        c.log_decay[:, t] = -np.inf
    c.check_forward(*c.run(attn))
    c.check_backward(c.run_back(attn))
    c.h0 = c.h0 * np.inf
    y, h = c.run(attn)
    c.h0 = np.zeros_like(c.h0)
    c.check_forward(y, h)


def test_the_same_at_once_and_replayed(attn):
    c = case(1, 1300, 4, 2)
    y, h = c.run(attn)
    g = c.run_back(attn)
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(4)]:
        with torch.cuda.stream(s):
            got.append((c.run(attn), c.run_back(attn)))
    torch.cuda.synchronize()
    ins = {n: c.t(n) for n in ("q", "k", "v", "dy", "log_decay", "h0", "dh")}
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a = attn(ins["q"], ins["k"], ins["v"], log_decay=ins["log_decay"],
                 scale=c.scale, h0=ins["h0"])
        b = attn.backward(ins["q"], ins["k"], ins["v"], ins["dy"],
                          log_decay=ins["log_decay"], scale=c.scale,
                          h0=ins["h0"], dh_last=ins["dh"])
    for _ in range(3):
        for t in list(a) + [x for x in b.values() if x is not None]:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got.append(([t.clone() for t in a],
                    {k: x if x is None else x.clone() for k, x in b.items()}))
    for (y2, h2), g2 in got:
        assert torch.equal(y, y2) and torch.equal(h, h2)
        for k in g:
            assert g[k] is None or torch.equal(g[k], g2[k]), k


def test_a_slice_of_a_wider_row(attn):
    """q, k and v as columns of one projection, 16 bytes aligned."""
    c = case(2, 300, 2, 2)
    b, L, H, G, dk, dv = c.dims
    w = 2 * G * dk + H * dv + 16
    row = torch.full((b, L, w), float("nan"), dtype=c.ty, device="cuda")
    cuts = [8, 8 + G * dk, 8 + 2 * G * dk]
    q = row[..., cuts[0]:cuts[1]].unflatten(-1, (G, dk))
    k = row[..., cuts[1]:cuts[2]].unflatten(-1, (G, dk))
    v = row[..., cuts[2]:cuts[2] + H * dv].unflatten(-1, (H, dv))
    for dst, name in ((q, "q"), (k, "k"), (v, "v")):
        dst.copy_(c.t(name))
    y, h = c.run(attn, q=q, k=k, v=v)
    y1, h1 = c.run(attn)
    assert torch.equal(y, y1) and torch.equal(h, h1)
    c.check_forward(y, h)
