"""The log decay's gradient over long sums and across restarts, as a whole
(per head), within the bounds of decay_bound."""
import numpy as np
import pytest
import torch

import decay_bound as D
import mixer_oracle as M
import selective_state_space_51_b200 as S
from test_gpu_linattn import Case, host

pytestmark = pytest.mark.gpu

# activation type, decay: the pass's kernel and planes
PATHS = {"f32": ("f32", "both", "planes3"),
         "bf16_head": ("bf16", "both", "planes3"),
         "bf16_token": ("bf16", "token", "planes2")}


@pytest.fixture(scope="module")
def attn():
    return S.LinearAttention(0)


def reference(c):
    return M.backward(c.q, c.k, c.v, c.g, c.scale, c.dy, c.h0, c.dh,
                      c.lengths)


@pytest.mark.parametrize("path", sorted(PATHS))
@pytest.mark.parametrize("at", [1, 7, 700, 1000, 1023, 1024, 1499])
def test_nothing_crosses_a_restart(attn, path, at):
    """No gradient in front of a restart when all that is differentiated lies
    behind it: exactly 0, wherever it falls."""
    dtype, gate, _ = PATHS[path]
    c = Case(dtype, 2, 1500, 2, 2, 64, 64, gate=gate, state=False)
    c.log_decay[:, at] = -np.inf
    c.dy[:, :at] = 0.0
    c.dy *= 64.0
    g = c.run_back(attn)
    for n in ("dq", "dk", "dv", "dlog_decay"):
        assert not g[n][:, :at].any(), n
    assert not g["dlog_decay"][:, at].any()
    assert g["dlog_decay"][:, at + 1:].any() or at == 1499
    assert attn.sync_status() == S.SSM_OK


@pytest.mark.parametrize("path", sorted(PATHS))
def test_packed_documents_keep_their_own_scale(attn, path):
    """Documents of one sequence whose gradients differ by 2^20: each within
    the bound of its own size."""
    dtype, gate, planes = PATHS[path]
    c = Case(dtype, 1, 1700, 2, 2, 32, 32, gate=gate, state=False)
    starts = [0, 333, 900, 1500, 1700]
    size = [1.0, 2.0 ** 20, 1.0, 2.0 ** 20]
    for i, s in zip(starts[1:], size):
        c.log_decay[:, i % 1700] = -np.inf
    for i, j, s in zip(starts, starts[1:], size):
        c.dy[:, i:j] *= s
    ref = reference(c)
    got = host(c.run_back(attn)["dlog_decay"])
    m = np.sqrt(((c.q * ref["dq"]) ** 2).sum(-1)
                + ((c.k * ref["dk"]) ** 2).sum(-1))
    for i, j in zip(starts, starts[1:]):
        part = slice(i, j)
        off = D.rms(got[:, part] - ref["dg"][:, part])
        tol = 4 * D.DELTA[planes] * D.rms(m[:, part]) * np.sqrt(j - i) \
            + (4 * 2.0 ** -22 + M.U[dtype]) * D.rms(ref["dg"][:, part])
        assert np.all(tol < 0.05 * D.rms(ref["dg"][:, part]))
        assert np.all(off <= tol), (i, off / tol)


# steps from an anchor to the next: 128, or a segment (of 2048 at most) where
# the gradient is bfloat16 and comes of the tensor-memory kernel
LONG = {"f32": 128, "bf16_head": 128, "bf16_token": 2048}


@pytest.mark.parametrize("path", sorted(LONG))
@pytest.mark.parametrize("b,L,state", [(1, 8192, False), (2, 2049, True),
                                       (1, 4223, True), (3, 300, True)])
@pytest.mark.parametrize("rate", [0.1, 0.003])
def test_long_sums(attn, path, b, L, state, rate):
    dtype, gate, planes = PATHS[path]
    c = Case(dtype, b, L, 2, 2, 32, 32, gate=gate, state=state, rate=rate)
    ref = reference(c)
    each, total = D.tolerances(c, ref, LONG[path], D.DELTA[planes], dtype)
    size = D.sizes(c, ref)[1]
    assert np.all(each <= 0.02 * size)
    g = c.run_back(attn)
    off = D.rms(host(g["dlog_decay"]) - ref["dg"])
    print("each", off / each)
    assert np.all(off <= each), off / each
    if g["dhead_log_decay"] is not None:
        off = np.abs(host(g["dhead_log_decay"]) - ref["dhead"])
        print("total", off / total)
        assert np.all(off <= total), off / total


@pytest.mark.parametrize("path", sorted(LONG))
def test_long_sums_where_heads_fill_the_gpu(attn, path):
    """Sequences that are not cut for want of heads are not summed in longer
    pieces for it."""
    dtype, gate, planes = PATHS[path]
    c = Case(dtype, 1, 6144, 64, 64, 8, 8, gate=gate, state=False, rate=0.003)
    ref = reference(c)
    each, total = D.tolerances(c, ref, LONG[path], D.DELTA[planes], dtype)
    assert np.all(each <= 0.05 * D.sizes(c, ref)[1])
    g = c.run_back(attn)
    off = D.rms(host(g["dlog_decay"]) - ref["dg"]) / each
    print("each", off.max())
    assert np.all(off <= 1), off
    if g["dhead_log_decay"] is not None:
        off = np.abs(host(g["dhead_log_decay"]) - ref["dhead"]) / total
        print("total", off.max())
        assert np.all(off <= 1), off


@pytest.mark.parametrize("path", sorted(LONG))
def test_long_sums_of_padded_sequences(attn, path):
    """A padded batch gives, sequence by sequence, what the sequences alone
    are bound to."""
    dtype, gate, planes = PATHS[path]
    lengths = [2500, 0, 128, 1025]
    c = Case(dtype, 4, 2500, 2, 2, 32, 32, gate=gate, lengths=lengths)
    ref = reference(c)
    got = host(c.run_back(attn)["dlog_decay"])
    m = ((c.q * ref["dq"]) ** 2).sum(-1) + ((c.k * ref["dk"]) ** 2).sum(-1)
    for i, n in enumerate(lengths):
        assert not got[i, n:].any()
        if n == 0:
            continue
        dg = np.sqrt((ref["dg"][i, :n] ** 2).mean(0))
        tol = 4 * (D.DELTA[planes] * np.sqrt(m[i, :n].mean(0))
                   * np.sqrt(min(n, LONG[path])) + 2.0 ** -22 * dg) \
            + M.U[dtype] * dg
        assert np.all(tol <= 0.02 * dg)
        off = np.sqrt(((got[i, :n] - ref["dg"][i, :n]) ** 2).mean(0))
        assert np.all(off <= tol), (i, off / tol)


@pytest.mark.parametrize("L", [2048, 2049, 4223])
def test_long_sums_of_odd_bfloat16_rows(attn, L):
    """Rows that the tensor-memory kernel does not take, the gradient bfloat16:
    groups of 2048 steps, three planes."""
    c = Case("bf16", 1, L, 2, 2, 33, 31, gate="token", rate=0.003)
    ref = reference(c)
    each, _ = D.tolerances(c, ref, 2048, D.DELTA["planes3"], "bf16")
    assert np.all(each <= 0.02 * D.sizes(c, ref)[1])
    off = D.rms(host(c.run_back(attn)["dlog_decay"]) - ref["dg"])
    assert np.all(off <= each), off / each
