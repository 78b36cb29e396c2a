"""How far the log decay's gradient may be off as a whole, for sums that are
too long for elementwise worst cases to say anything.

The kernels sum dg_t = dg_{t+1} + q_t . dq_t - k_t . dk_t backwards from an
anchor <S, G>, at most A steps away. One element of dq or dk is a sum of some
16 truncating additions, each off by 2^-24 of it or so, which makes 2^-22 as
the root of their squares (two bfloat16 planes in place of three: 2^-18 at the
most of one term, taken as 2^-17 of all); the errors of different steps are
independent. With m_t the root of the sum of (q dq)^2 and (k dk)^2 over the
size, over the steps of one head:
  - a row dot is off by delta m_t, the anchor, a product of float32 states, by
    2^-22 of the gradient's size, and the sum behind a step takes A of the
    first and one of the second: root mean square delta m sqrt(A) + 2^-22 |dg|;
  - the sum over N steps: an error made d steps behind the anchor's other end
    is in d gradients, so A steps add sqrt(A^3 / 3) delta m, and N / A such
    groups delta m A sqrt(N / 3); the anchors 2^-22 |dg| A sqrt(N / A).
Both are taken four times (what a normal deviate passes once in 16,000), and
the output's own rounding is added.
"""
import numpy as np

import mixer_oracle as M

DELTA = {"planes3": 2.0 ** -22, "planes2": 2.0 ** -17}


def sizes(c, ref):
    """m and |dg| of each head, as root mean squares over all steps."""
    q, k = c.q, c.k
    m = ((q * ref["dq"]) ** 2).sum(-1) + ((k * ref["dk"]) ** 2).sum(-1)
    return (np.sqrt(m.mean((0, 1))), np.sqrt((ref["dg"] ** 2).mean((0, 1))))


def tolerances(c, ref, anchor, delta, out_dtype):
    """Of a head's gradients as root mean square, and of their sum. For cases
    with as many groups as heads."""
    m, g = sizes(c, ref)
    n = ref["dg"].shape[0] * ref["dg"].shape[1]
    a = min(anchor, ref["dg"].shape[1])
    each = 4 * (delta * m * np.sqrt(a) + 2.0 ** -22 * g) \
        + M.U[out_dtype] * g
    total = 4 * (delta * m * a * np.sqrt(n / 3)
                 + 2.0 ** -22 * g * np.sqrt(a * n))
    return each, total + 2.0 ** -23 * np.abs(ref["dhead"])


def rms(d):
    return np.sqrt((d ** 2).mean((0, 1)))
