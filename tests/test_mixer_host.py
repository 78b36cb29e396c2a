"""What the linear-attention and layer-norm entry points refuse, found on the
host before anything is launched (no GPU needed)."""
import ctypes

import pytest

import selective_state_space_51_b200 as S
from selective_state_space_51_b200 import build as B

P = 4096          # an aligned address that no call gets to read
DIMS = dict(batch=2, seqlen=8, heads=4, groups=2, dk=16, dv=16)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return S.library()


def dims(**kw):
    d = dict(DIMS, q_stride=0, k_stride=0, v_stride=0)
    d.update(kw)
    return S.ssm_linattn_dims(**d)


def fwd(lib, d=None, dtype=S.SSM_F32, **kw):
    a = dict(q=P, k=P, v=P, log_decay=P, head=P, lengths=P, h0=P, y=P,
             h_last=P, ws=P, n=1 << 40)
    a.update(kw)
    return lib.ssm_linattn_fwd(
        0, a["q"], a["k"], a["v"], a["log_decay"], a["head"], 1.0,
        a["lengths"], a["h0"], a["y"], a["h_last"], a["ws"], a["n"],
        d or dims(), dtype, None)


def bwd(lib, d=None, dtype=S.SSM_F32, **kw):
    names = ("q", "k", "v", "log_decay", "head")
    more = ("lengths", "h0", "dy", "dh_last", "dq", "dk", "dv", "dlog_decay",
            "dhead", "dh0", "ws")
    a = {n: P for n in names + more}
    a.update(kw)
    return lib.ssm_linattn_bwd(0, *[a[n] for n in names], 1.0,
                               *[a[n] for n in more], 1 << 40, d or dims(),
                               dtype, None)


def step(lib, d=None, dtype=S.SSM_F32, **kw):
    a = dict(q=P, k=P, v=P, log_decay=P, head=P, state=P, y=P)
    a.update(kw)
    return lib.ssm_linattn_step(0, a["q"], a["k"], a["v"], a["log_decay"],
                                a["head"], 1.0, a["state"], a["y"],
                                d or dims(seqlen=1), dtype, None)


@pytest.mark.parametrize("bad", [
    dict(batch=0), dict(seqlen=0), dict(heads=0), dict(groups=0), dict(dk=0),
    dict(dv=-1), dict(heads=5), dict(groups=3), dict(q_stride=31),
    dict(k_stride=1), dict(v_stride=63), dict(batch=1 << 40, seqlen=1 << 40),
    dict(batch=1 << 50), dict(seqlen=1 << 52)])
def test_bad_dims(lib, bad):
    assert fwd(lib, dims(**bad)) == S.SSM_ERR_INVALID
    assert bwd(lib, dims(**bad)) == S.SSM_ERR_INVALID
    n = ctypes.c_size_t(7)
    assert lib.ssm_linattn_workspace(0, dims(**bad), S.SSM_F32, 0,
                                     ctypes.byref(n)) == S.SSM_ERR_INVALID
    assert n.value == 0
    if "seqlen" not in bad:
        assert step(lib, dims(seqlen=1, **bad)) == S.SSM_ERR_INVALID


@pytest.mark.parametrize("bad", [dict(dk=129), dict(dv=257)])
def test_sizes_that_are_not_built(lib, bad):
    assert fwd(lib, dims(**bad)) == S.SSM_ERR_UNSUPPORTED
    assert bwd(lib, dims(**bad)) == S.SSM_ERR_UNSUPPORTED
    assert step(lib, dims(seqlen=1, **bad)) == S.SSM_ERR_UNSUPPORTED
    assert bwd(lib, dims(dv=129)) == S.SSM_ERR_UNSUPPORTED
    assert fwd(lib, dtype=2) == S.SSM_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["q", "k", "v", "y"])
def test_required_and_misaligned_forward(lib, name):
    assert fwd(lib, **{name: None}) == S.SSM_ERR_INVALID
    assert fwd(lib, **{name: P + 2}) == S.SSM_ERR_ALIGN
    assert fwd(lib, dtype=S.SSM_BF16, **{name: P + 1}) == S.SSM_ERR_ALIGN
    assert step(lib, **{name: None}) == S.SSM_ERR_INVALID
    assert step(lib, **{name: P + 2}) == S.SSM_ERR_ALIGN


def test_pairs_need_their_alignment(lib):
    assert fwd(lib, y=P + 4) == S.SSM_ERR_ALIGN
    assert fwd(lib, dtype=S.SSM_BF16, y=P + 2) == S.SSM_ERR_ALIGN
    assert bwd(lib, dq=P + 4) == S.SSM_ERR_ALIGN
    assert bwd(lib, dv=P + 4) == S.SSM_ERR_ALIGN


@pytest.mark.parametrize("name", ["head", "lengths", "h0", "h_last"])
def test_misaligned_floats(lib, name):
    assert fwd(lib, **{name: P + 1}) == S.SSM_ERR_ALIGN


@pytest.mark.parametrize("name", ["q", "k", "v", "dy", "dq", "dk", "dv"])
def test_required_backward(lib, name):
    assert bwd(lib, **{name: None}) == S.SSM_ERR_INVALID


def test_a_decay_gradient_needs_its_decay(lib):
    assert bwd(lib, log_decay=None) == S.SSM_ERR_INVALID
    assert bwd(lib, head=None) == S.SSM_ERR_INVALID


def test_step_takes_one_token(lib):
    assert step(lib, dims(seqlen=2)) == S.SSM_ERR_INVALID
    assert step(lib, state=None) == S.SSM_ERR_INVALID


def test_bad_device(lib):
    n = ctypes.c_size_t()
    for device in (-1, 64):
        assert lib.ssm_linattn_workspace(device, dims(), S.SSM_F32, 0,
                                         ctypes.byref(n)) == S.SSM_ERR_INVALID
        assert lib.ssm_layernorm_workspace(
            device, 4, 4, S.SSM_F32, ctypes.byref(n)) == S.SSM_ERR_INVALID
    assert lib.ssm_linattn_workspace(0, dims(), S.SSM_F32, 0,
                                     None) == S.SSM_ERR_INVALID


def norm(lib, rows=4, dim=8, dtype=S.SSM_F32, **kw):
    a = dict(x=P, residual=P, weight=P, bias=P, y=P, sum=P, mean=P, rstd=P)
    a.update(kw)
    return lib.ssm_layernorm_fwd(0, a["x"], a["residual"], a["weight"],
                                 a["bias"], 1e-5, a["y"], a["sum"], a["mean"],
                                 a["rstd"], rows, dim, dtype, None)


def norm_back(lib, rows=4, dim=8, dtype=S.SSM_F32, **kw):
    names = ("dy", "x", "mean", "rstd", "weight", "dsum", "dx", "dweight",
             "dbias", "ws")
    a = {n: P for n in names}
    a.update(kw)
    return lib.ssm_layernorm_bwd(0, *[a[n] for n in names], 1 << 40, rows,
                                 dim, dtype, None)


def test_norm_refusals(lib):
    for kw in (dict(rows=0), dict(dim=0), dict(x=None), dict(y=None),
               dict(residual=None)):          # a sum without its residual
        assert norm(lib, **kw) == S.SSM_ERR_INVALID
    for kw in (dict(rows=0), dict(dim=-1), dict(dy=None), dict(x=None),
               dict(mean=None), dict(rstd=None), dict(dx=None)):
        assert norm_back(lib, **kw) == S.SSM_ERR_INVALID
    for call in (norm, norm_back):
        assert call(lib, dim=8193) == S.SSM_ERR_UNSUPPORTED
        assert call(lib, dtype=5) == S.SSM_ERR_UNSUPPORTED
        assert call(lib, x=P + 2) == S.SSM_ERR_ALIGN
        assert call(lib, weight=P + 2) == S.SSM_ERR_ALIGN


def far(names, first=1 << 30, step=1 << 24):
    """Addresses of buffers that lie apart."""
    return {n: first + i * step for i, n in enumerate(names)}


FWD = ("q", "k", "v", "log_decay", "head", "lengths", "h0", "y", "h_last",
       "ws")
BWD = ("q", "k", "v", "log_decay", "head", "lengths", "h0", "dy", "dh_last",
       "dq", "dk", "dv", "dlog_decay", "dhead", "dh0", "ws")
NORM = ("x", "residual", "weight", "bias", "y", "sum", "mean", "rstd")
NORM_BACK = ("dy", "x", "mean", "rstd", "weight", "dsum", "dx", "dweight",
             "dbias", "ws")


def passes(rc):
    """A call whose arguments are accepted gets as far as the device."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: these addresses are not its own")
    assert rc in (S.SSM_ERR_CUDA, S.SSM_ERR_ARCH)


@pytest.mark.parametrize("out", ["y", "h_last"])
@pytest.mark.parametrize("other", ["q", "k", "v", "log_decay", "head",
                                   "lengths", "h0", "y"])
def test_forward_outputs_lie_apart(lib, out, other):
    a = far(FWD)
    if (out, other) == ("y", "y"):
        return passes(fwd(lib, **a))
    if (out, other) == ("h_last", "h0"):
        passes(fwd(lib, **{**a, out: a[other]}))     # in place
        assert fwd(lib, **{**a, out: a[other] + 8}) == S.SSM_ERR_INVALID
    else:
        assert fwd(lib, **{**a, out: a[other]}) == S.SSM_ERR_INVALID


def test_strided_rows_count_to_their_last_element(lib):
    a, d = far(FWD), dims(q_stride=100)   # 2 x 8 tokens
    end = a["q"] + (15 * 100 + 32) * 4
    assert fwd(lib, d, **{**a, "y": end - 8}) == S.SSM_ERR_INVALID
    passes(fwd(lib, d, **{**a, "y": end}))


@pytest.mark.parametrize("out", BWD[9:15])
@pytest.mark.parametrize("other", BWD[:15])
def test_backward_outputs_lie_apart(lib, out, other):
    a = far(BWD)
    if out == other:
        return passes(bwd(lib, **a))
    assert bwd(lib, **{**a, out: a[other]}) == S.SSM_ERR_INVALID


@pytest.mark.parametrize("other", ["q", "k", "v", "log_decay", "head", "y"])
def test_step_outputs_lie_apart(lib, other):
    a = far(("q", "k", "v", "log_decay", "head", "state", "y"))
    assert step(lib, **{**a, "state": a[other]}) == S.SSM_ERR_INVALID
    if other != "y":
        assert step(lib, **{**a, "y": a[other]}) == S.SSM_ERR_INVALID
    passes(step(lib, **a))


def test_norm_in_place_or_apart(lib):
    a = far(NORM)
    for out in ("y", "sum"):
        for other in ("x", "residual"):
            assert norm(lib, **{**a, out: a[other] + 16}) == S.SSM_ERR_INVALID
        for other in ("weight", "mean"):
            assert norm(lib, **{**a, out: a[other]}) == S.SSM_ERR_INVALID
    assert norm(lib, **{**a, "sum": a["y"]}) == S.SSM_ERR_INVALID
    assert norm(lib, **{**a, "mean": a["x"]}) == S.SSM_ERR_INVALID
    b = far(NORM_BACK)
    for other in ("x", "dy", "dsum"):
        assert norm_back(lib, **{**b, "dx": b[other] + 16}) == \
            S.SSM_ERR_INVALID
        assert norm_back(lib, **{**b, "dbias": b[other]}) == S.SSM_ERR_INVALID
    assert norm_back(lib, **{**b, "dweight": b["dbias"]}) == S.SSM_ERR_INVALID
    for out, other in (("y", "x"), ("y", "residual"), ("sum", "x")):
        passes(norm(lib, **{**a, out: a[other]}))
    for other in ("x", "dy", "dsum"):
        passes(norm_back(lib, **{**b, "dx": b[other]}))


def test_more_steps_than_a_device_holds(lib):
    d = dims(batch=1, seqlen=1 << 37, heads=1, groups=1, dk=1, dv=1)
    assert fwd(lib, d) == bwd(lib, d) == S.SSM_ERR_INVALID


def test_without_a_gpu_the_calls_fail_cleanly(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for rc in (fwd(lib), bwd(lib), step(lib), norm(lib), norm_back(lib)):
        assert rc in (S.SSM_ERR_CUDA, S.SSM_ERR_INVALID)
