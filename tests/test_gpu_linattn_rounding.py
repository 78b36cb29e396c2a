"""bfloat16 results are off by their own rounding and little else.

With r the root mean square of what rounding the exact result to bfloat16
takes (about 0.43 of half a step: 1.66e-3 of the result), a rounding of every
score, or of the state, to one bfloat16 plane would add as much again: sqrt(2)
r. Two planes leave 2^-17 of a term where one leaves 2^-9, so the terms'
absolute sum would have to be 80 times the result for 5% of r to come of them
(added as squares: 0.32 r), and float32 sums leave 2^-17 of r. 1.05 r is what
the results are held to."""
import numpy as np
import pytest

import mixer_oracle as M
import selective_state_space_51_b200 as S
from test_gpu_linattn import Case, host

pytestmark = pytest.mark.gpu
# the tensor-memory kernel's four sizes, sizes inside them, and what the other
# kernel takes
SIZES = [(128, 128), (128, 64), (64, 128), (64, 64), (24, 96), (16, 16),
         (45, 77), (33, 128), (128, 1)]


@pytest.fixture(scope="module")
def attn():
    return S.LinearAttention(0)


def close(got, ref, what):
    r = np.sqrt(((M.bf16(ref) - ref) ** 2).mean())
    off = np.sqrt(((host(got) - ref) ** 2).mean())
    print(what, "%.3f" % (off / r))
    assert off <= 1.05 * r, (what, off / r)


@pytest.mark.parametrize("dk,dv", SIZES + [(64, 200)])
@pytest.mark.parametrize("rate", [0.3, 0.01])
@pytest.mark.parametrize("L", [1, 40, 700])
def test_prompt(attn, dk, dv, rate, L):
    c = Case("bf16", 2, L, 4, 2, dk, dv, gate="both", rate=rate)
    ref, _ = M.forward(c.q, c.k, c.v, c.g, c.scale, c.h0)
    y, _ = c.run(attn)
    close(y, ref, "y")


@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("groups", [1, 2])
def test_backward(attn, dk, dv, gate, groups):
    c = Case("bf16", 2, 500, 2, groups, dk, dv, gate="token", rate=0.02)
    ref = M.backward(c.q, c.k, c.v, c.g, c.scale, c.dy, c.h0, c.dh)
    g = c.run_back(attn, decay_gradient=gate)
    for n in ("dq", "dk", "dv"):
        close(g[n], ref[n], n)
    if gate:
        close(g["dlog_decay"], ref["dg"], "dlog_decay")
