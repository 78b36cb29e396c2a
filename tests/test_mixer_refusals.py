"""The refusals of the linear-attention and layer-norm entry points, one
changed argument at a time: the call as it stands gets as far as the device,
so that what is refused is refused for that argument (no GPU needed)."""
import ctypes

import pytest
import torch

import selective_state_space_51_b200 as S
from selective_state_space_51_b200 import build as B
from test_mixer_host import (BWD, FWD, NORM, NORM_BACK, bwd, dims, far, fwd,
                             norm, norm_back, step)

pytestmark = pytest.mark.skipif(
    torch.cuda.is_available(),
    reason="a GPU is present: these addresses are not its own")
STEP = ("q", "k", "v", "log_decay", "head", "state", "y")
CALLS = {"fwd": (fwd, FWD), "bwd": (bwd, BWD), "step": (step, STEP),
         "norm": (norm, NORM), "norm_back": (norm_back, NORM_BACK)}
PAST_THE_HOST = (S.SSM_ERR_CUDA, S.SSM_ERR_ARCH)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return S.library()


def run(lib, name, d=None, *, without=(), moved=None, **kw):
    call, names = CALLS[name]
    a = far(names)
    for n in without:
        a[n] = None
    for n, by in (moved or {}).items():
        a[n] += by
    if d is not None:
        kw["d"] = d
    return call(lib, **a, **kw)


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("dtype", [S.SSM_F32, S.SSM_BF16])
def test_the_call_itself_reaches_the_device(lib, name, dtype):
    assert run(lib, name, dtype=dtype) in PAST_THE_HOST


OPTIONAL = {"fwd": ["log_decay", "head", "lengths", "h0", "h_last", "ws"],
            "bwd": ["lengths", "h0", "dh_last", "dlog_decay", "dhead", "dh0",
                    "ws"],
            "step": ["log_decay", "head"],
            "norm": ["weight", "bias", "sum", "mean", "rstd"],
            "norm_back": ["weight", "dsum", "dweight", "dbias", "ws"]}


@pytest.mark.parametrize("name,arg", [
    (n, a) for n, (_, names) in sorted(CALLS.items()) for a in names])
def test_each_pointer_is_required_or_not(lib, name, arg):
    rc = run(lib, name, without=[arg])
    if arg in OPTIONAL[name]:
        assert rc in PAST_THE_HOST
    else:
        # (a decay may be left out with its gradient, a residual with its sum:
        # below)
        assert rc == S.SSM_ERR_INVALID


@pytest.mark.parametrize("name,pair", [
    ("bwd", ("log_decay", "dlog_decay")), ("bwd", ("head", "dhead")),
    ("norm", ("residual", "sum"))])
def test_what_may_be_left_out_together(lib, name, pair):
    assert run(lib, name, without=pair) in PAST_THE_HOST
    assert run(lib, name, without=pair[:1]) == S.SSM_ERR_INVALID


@pytest.mark.parametrize("name,arg", [
    (n, a) for n, (_, names) in sorted(CALLS.items()) for a in names
    if a != "ws"])
def test_each_pointer_has_its_alignment(lib, name, arg):
    assert run(lib, name, moved={arg: 2}) == S.SSM_ERR_ALIGN
    assert run(lib, name, moved={arg: 1},
               dtype=S.SSM_BF16) == S.SSM_ERR_ALIGN


BAD_DIMS = [dict(batch=0), dict(heads=0), dict(groups=0), dict(dk=0),
            dict(dv=-1), dict(heads=5), dict(groups=3), dict(q_stride=31),
            dict(k_stride=1), dict(v_stride=63), dict(batch=1 << 50)]


@pytest.mark.parametrize("name", ["fwd", "bwd", "step"])
@pytest.mark.parametrize("bad", BAD_DIMS)
def test_dims(lib, name, bad):
    one = dict(seqlen=1) if name == "step" else {}
    assert run(lib, name, dims(**one)) in PAST_THE_HOST
    assert run(lib, name, dims(**one, **bad)) == S.SSM_ERR_INVALID


@pytest.mark.parametrize("name", ["fwd", "bwd"])
@pytest.mark.parametrize("bad", [dict(seqlen=0), dict(seqlen=-3),
                                 dict(seqlen=1 << 52),
                                 dict(batch=1 << 40, seqlen=1 << 40)])
def test_lengths(lib, name, bad):
    assert run(lib, name, dims(**bad)) == S.SSM_ERR_INVALID


@pytest.mark.parametrize("name", ["fwd", "bwd"])
def test_more_steps_than_a_device_holds(lib, name):
    """Apart from the buffers, which would overlap: one element a step, and
    addresses that far apart."""
    call, names = CALLS[name]
    one = dict(batch=1, heads=1, groups=1, dk=1, dv=1)
    a = far(names, step=1 << 40)
    assert call(lib, dims(seqlen=1 << 36, **one), **a) in PAST_THE_HOST
    assert call(lib, dims(seqlen=(1 << 36) + 1, **one),
                **a) == S.SSM_ERR_INVALID


@pytest.mark.parametrize("name,most", [("fwd", 256), ("bwd", 128),
                                       ("step", 256)])
def test_sizes_that_are_built(lib, name, most):
    one = dict(seqlen=1) if name == "step" else {}
    assert run(lib, name, dims(dk=128, dv=most, **one)) in PAST_THE_HOST
    assert run(lib, name, dims(dk=129, **one)) == S.SSM_ERR_UNSUPPORTED
    assert run(lib, name, dims(dv=most + 1, **one)) == S.SSM_ERR_UNSUPPORTED
    assert run(lib, name, dims(**one), dtype=2) == S.SSM_ERR_UNSUPPORTED


def test_a_step_is_one_token(lib):
    assert run(lib, "step", dims(seqlen=1)) in PAST_THE_HOST
    assert run(lib, "step", dims(seqlen=2)) == S.SSM_ERR_INVALID


@pytest.mark.parametrize("name", ["norm", "norm_back"])
def test_norm_sizes(lib, name):
    assert run(lib, name, rows=7, dim=8192) in PAST_THE_HOST
    for bad in (dict(rows=0), dict(rows=-1), dict(dim=0), dict(dim=-1),
                dict(rows=(1 << 42) + 1)):
        assert run(lib, name, **bad) == S.SSM_ERR_INVALID
    assert run(lib, name, dim=8193) == S.SSM_ERR_UNSUPPORTED
    assert run(lib, name, dtype=5) == S.SSM_ERR_UNSUPPORTED


def test_devices(lib):
    """A device that is not there is refused by the calls themselves too."""
    a = far(FWD)
    for device in (-1, 64):
        rc = lib.ssm_linattn_fwd(
            device, a["q"], a["k"], a["v"], a["log_decay"], a["head"], 1.0,
            a["lengths"], a["h0"], a["y"], a["h_last"], a["ws"], 1 << 40,
            dims(), S.SSM_F32, None)
        assert rc == S.SSM_ERR_INVALID
        n = ctypes.c_size_t(7)
        assert lib.ssm_linattn_workspace(device, dims(), S.SSM_F32, 1,
                                         ctypes.byref(n)) == S.SSM_ERR_INVALID
        assert n.value == 0
