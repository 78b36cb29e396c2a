"""Where a step starts the state anew: below a log decay of -87, both decays
added, and not at it."""
import numpy as np
import pytest
import torch

import mixer_oracle as M
import selective_state_space_51_b200 as S
from test_gpu_linattn import TYPES, Case, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    return S.LinearAttention(0)


def case(dtype, size, below):
    """Restarts at tokens 0, 70 and 200 of 300: log decays of -87.2, or of -87
    where `below` is False, from the two decays together."""
    c = Case(dtype, 1, 300, 2, 2, size, size, gate="token", rate=0.01)
    c.log_decay[:] = 0.0
    c.head = np.full(2, np.float32(-0.2 if below else 0.0)).astype(float)
    c.log_decay[:, [0, 70, 200]] = -87.0
    return c


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("size", [16, 45])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_just_below_the_border(attn, dtype, size, value):
    c = case(dtype, size, True)
    h0 = c.h0
    c.h0 = np.full_like(h0, value)
    y, h = c.run(attn)
    g = c.run_back(attn)
    c.h0 = h0
    c.check_forward(y, h)
    for n in ("dlog_decay", "dk", "dv", "dq"):
        assert bool(g[n].isfinite().all()), n
    assert not g["dlog_decay"][:, [0, 70, 200]].any()
    assert not g["dh0"].any()
    assert attn.sync_status() == S.SSM_OK


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("size", [16, 45])
def test_the_border_itself_keeps_the_state(attn, dtype, size):
    c = case(dtype, size, False)
    c.h0 = np.full_like(c.h0, np.nan)
    y, h = c.run(attn)
    assert bool(y[:, 0].isnan().all())


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("head,anew", [(-0.2, True), (0.0, False)])
def test_step(attn, dtype, head, anew):
    ty = TYPES[dtype]
    state = torch.full((2, 2, 8, 8), float("nan"), device="cuda")
    q, k, v = (torch.ones(2, 2, 8, device="cuda", dtype=ty) for _ in range(3))
    y = attn.step(q, k, v, state, scale=1.0,
                  log_decay=torch.full((2, 2), -87.0, device="cuda", dtype=ty),
                  head_log_decay=torch.full((2,), head, device="cuda"))
    if anew:
        assert torch.equal(state, torch.ones_like(state))
        assert torch.equal(y, torch.full_like(y, 8.0))
    else:
        assert bool(state.isnan().all())


def test_the_reference_has_the_same_border():
    a = M.exponentials(np.array([-87.0, np.nextafter(-87.0, -88.0)]))
    assert a[0] > 0 and a[1] == 0
