"""Linear attention and layer norm on another stream than the current one,
where the current one still has to make their inputs, and where these are
dropped as soon as the call returns."""
import pytest
import torch

import selective_state_space_51_b200 as S

pytestmark = pytest.mark.gpu
SLEEP = 100_000_000      # cycles: about 50 ms


def prompt(attn, norm, x, **kw):
    return list(attn(x, x, x, **kw))


def step(attn, norm, x, **kw):
    state = torch.zeros(1, 4, 32, 32, device="cuda")
    return [attn.step(x[:, 0], x[:, 1], x[:, 2], state, **kw)]


def backward(attn, norm, x, **kw):
    g = attn.backward(x, x, x, x, **kw)
    return [g[k] for k in ("dq", "dk", "dv", "dh0")]


def norm_forward(attn, norm, x, **kw):
    out = norm(x, weight=x.view(-1)[:32], residual=x, **kw)
    return [out[k] for k in ("y", "sum", "mean", "rstd")]


def norm_backward(attn, norm, x, **kw):
    rows = x.numel() // 32
    g = norm.backward(x, x, x.view(-1)[:rows], x.view(-1)[rows:2 * rows],
                      weight=x.view(-1)[:32], **kw)
    return [g["dx"], g["dweight"]]


CALLS = [prompt, step, backward, norm_forward, norm_backward]


@pytest.fixture(scope="module")
def ops():
    return S.LinearAttention(0), S.LayerNorm(0)


@pytest.fixture(scope="module")
def data():
    gen = torch.Generator(device="cuda").manual_seed(5)
    return torch.randn(1, 300, 4, 32, generator=gen, device="cuda")


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
@pytest.mark.parametrize("raw", [False, True])
def test_inputs_that_are_still_being_made(ops, data, call, raw):
    want = call(*ops, data)
    x, side = torch.zeros_like(data), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    x.copy_(data)
    got = call(*ops, x, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_inputs_that_are_dropped_at_once(ops, data, call):
    want = call(*ops, data)
    x, side = data.clone(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    got = call(*ops, x, stream=side)
    del x
    other = [torch.full_like(data, float("nan")) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del other


def test_captured_on_a_stream_of_its_own(ops, data):
    """A graph that is captured on `stream` alone, and one that forks to it."""
    want = prompt(*ops, data)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        got = prompt(*ops, data, stream=side)
        here.wait_stream(side)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    graph, lone = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(lone):
        graph.capture_begin()
        try:
            with torch.cuda.stream(torch.cuda.default_stream()):
                alone = prompt(*ops, data, stream=lone)
        finally:
            graph.capture_end()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, want))


def test_the_status_waits_for_its_own_stream(ops):
    """Not for the current one (unless that is the default stream, which the
    status word is read on)."""
    side, here = torch.cuda.Stream(), torch.cuda.Stream()
    done = torch.cuda.Event()
    assert ops[0].sync_status(stream=side) == S.SSM_OK    # (first use)
    torch.cuda.synchronize()
    with torch.cuda.stream(here):
        torch.cuda._sleep(10 * SLEEP)
        done.record()
        for s in (side, side.cuda_stream):
            assert ops[0].sync_status(stream=s) == S.SSM_OK
        assert not done.query()
        assert ops[0].sync_status() == S.SSM_OK
        assert done.query()
