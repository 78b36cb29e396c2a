"""States that remember tens of thousands of steps: the kept part of a state
is multiplied hundreds of times, and what it is rounded by must not add up.

With u = 2^-24: a chunk's update rounds the state once or twice, to either side
(0.3 u, the root mean square of a rounding to nearest), so n chunks leave
0.6 u sqrt(n); the products in front of it are 8 u off whatever n is (truncated
sums of 16 products and the weights' exponentials). Twice that is allowed:
u (16 + 1.2 sqrt(n)). A kept part that were off by 0.3 u to the same side each
time would make 0.3 u n / 2."""
import numpy as np
import pytest
import torch

import mixer_oracle as M
import selective_state_space_51_b200 as S
from test_gpu_linattn import Case, host

pytestmark = pytest.mark.gpu
L = 40_000


@pytest.fixture(scope="module")
def attn():
    return S.LinearAttention(0)


def rel(got, ref):
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [4, 148])        # cut into segments, and not
@pytest.mark.parametrize("decay", [1e-5, 1e-4, -2e-5])
def test_long_memory(attn, dtype, heads, decay):
    c = Case(dtype, 1, L, heads, heads, 8, 8, gate="head", state=True)
    rng = np.random.default_rng(3)
    c.head = (-decay * (0.5 + rng.random(heads))).astype(
        np.float32).astype(np.float64)
    ref_y, ref_h = M.forward(c.q, c.k, c.v, c.g, c.scale, c.h0)
    y, h = c.run(attn)
    tol = 2.0 ** -24 * (16 + 1.2 * np.sqrt(L / 64))
    print("h %.2f of its bound" % (rel(host(h), ref_h) / tol))
    assert rel(host(h), ref_h) <= tol
    if dtype == "f32":
        assert rel(host(y), ref_y) <= tol


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [1e-5, 1e-4, -2e-5])
def test_many_single_tokens(attn, dtype, decay):
    """25,600 tokens one at a time: two roundings of the state each, to either
    side."""
    heads, T, times = 16, 256, 100
    c = Case(dtype, 1, T, heads, heads, 8, 8, gate="head", state=True)
    rng = np.random.default_rng(5)
    c.head = (-decay * (0.5 + rng.random(heads))).astype(
        np.float32).astype(np.float64)
    q, k, v, head, state = (c.t(n) for n in ("q", "k", "v", "head", "h0"))

    def tokens():
        for t in range(T):
            attn.step(q[:, t], k[:, t], v[:, t], state, head_log_decay=head)

    attn.step(q[:, 0], k[:, 0], v[:, 0], state.clone(), head_log_decay=head)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens()
    state.copy_(c.t("h0"))
    for _ in range(times):
        graph.replay()
    a = np.exp(c.head)[:, None, None]
    ref = c.h0[0].copy()
    kv = c.k[0][:, :, :, None] * c.v[0][:, :, None, :]
    for t in range(T * times):
        ref = a * ref + kv[t % T]
    tol = 2.0 ** -24 * (16 + 1.2 * np.sqrt(T * times))
    off = rel(host(state)[0], ref)
    print("state %.2f of its bound" % (off / tol))
    assert off <= tol
