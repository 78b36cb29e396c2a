"""The bounds of decay_bound see the mistakes they are there for: an anchor
left out, or taken one group off, and a sum that goes on over a restart (CPU,
planted in the 64-bit reference)."""
import types

import numpy as np
import pytest

import decay_bound as D
import mixer_oracle as M


def case(L, rate, seed=0):
    rng = np.random.default_rng(seed)
    H, d = 2, 16
    c = types.SimpleNamespace(
        q=rng.standard_normal((1, L, H, d)),
        k=rng.standard_normal((1, L, H, d)),
        v=rng.standard_normal((1, L, H, d)),
        dy=rng.standard_normal((1, L, H, d)),
        g=-rate * rng.exponential(size=(1, L, H)))
    return c, M.backward(c.q, c.k, c.v, c.g, 0.25, c.dy)


@pytest.mark.parametrize("rate", [0.1, 0.003])
@pytest.mark.parametrize("dtype,anchor,planes", [("f32", 128, "planes3"),
                                                 ("bf16", 128, "planes3"),
                                                 ("bf16", 512, "planes2")])
def test_a_wrong_anchor_is_seen(rate, dtype, anchor, planes):
    c, ref = case(1500, rate)
    each, total = D.tolerances(c, ref, anchor, D.DELTA[planes], dtype)
    dots = (c.q * ref["dq"]).sum(-1) - (c.k * ref["dk"]).sum(-1)
    dg = ref["dg"][0]
    for wrong in ("none", "left out", "one off"):
        got = np.zeros_like(dg)
        for t0 in range(0, 1500, anchor):
            t1 = min(t0 + anchor, 1500)
            end = np.zeros(2)
            if t1 < 1500 and wrong != "left out":
                end = dg[t1] if wrong == "none" else dg[min(t1 + 1, 1499)]
            run = dots[0, t0:t1][::-1].cumsum(0)[::-1]
            got[t0:t1] = end + run
        off = D.rms((got - dg)[None])
        sums = np.abs(got.sum(0) - ref["dhead"])
        if wrong == "none":
            assert np.all(off <= 1e-9 * each + 1e-9)
        elif wrong == "left out":
            assert np.all(off > each)
            assert dtype == "bf16" or np.any(sums > total)
        else:
            assert np.any(off > each)


def test_a_planes_error_is_within_its_bound():
    """Independent errors of delta a row dot stay inside, with the anchors
    exact; a hundred times that does not."""
    c, ref = case(1500, 0.003)
    each, total = D.tolerances(c, ref, 128, D.DELTA["planes3"], "f32")
    m = np.sqrt(((c.q * ref["dq"]) ** 2).sum(-1)
                + ((c.k * ref["dk"]) ** 2).sum(-1))
    rng = np.random.default_rng(1)
    for factor in (1.0, 100.0):
        e = factor * D.DELTA["planes3"] * m[0] * rng.standard_normal((1500, 2))
        off = np.zeros_like(e)
        for t0 in range(0, 1500, 128):
            off[t0:t0 + 128] = e[t0:t0 + 128][::-1].cumsum(0)[::-1]
        inside = np.all(D.rms(off[None]) <= each)
        assert inside == (factor == 1.0)
        assert np.all(np.abs(off.sum(0)) <= total) == (factor == 1.0)
