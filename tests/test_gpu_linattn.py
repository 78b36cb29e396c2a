"""GPU parity of linear attention with a decay for each head (prompt, single
token, backward) with the 64-bit recurrence, within the bounds derived in
mixer_oracle."""
import numpy as np
import pytest
import torch

import mixer_oracle as M
import selective_state_space_51_b200 as S

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def attn():
    return S.LinearAttention(0)


class Case:
    """Inputs on the device and, as the device holds them, in 64 bits."""

    def __init__(self, dtype, b, L, H, G, dk, dv, gate="both", state=True,
                 lengths=None, seed=0, rate=0.1):
        rng = np.random.default_rng(seed + L * 7 + dk)
        self.dtype, self.ty = dtype, TYPES[dtype]
        act = M.bf16 if dtype == "bf16" else (
            lambda a: a.astype(np.float32).astype(np.float64))
        f32 = lambda a: a.astype(np.float32).astype(np.float64)  # noqa: E731
        self.q = act(rng.standard_normal((b, L, G, dk)))
        self.k = act(rng.standard_normal((b, L, G, dk)))
        self.v = act(rng.standard_normal((b, L, H, dv)))
        self.log_decay = (act(-rate * rng.exponential(size=(b, L, H)))
                          if gate in ("token", "both") else None)
        self.head = (f32(-rate * rng.exponential(size=H))
                     if gate in ("head", "both") else None)
        self.h0 = (f32(rng.standard_normal((b, H, dk, dv))) if state else None)
        self.dy = act(rng.standard_normal(self.v.shape))
        self.dh = f32(rng.standard_normal((b, H, dk, dv))) if state else None
        self.lengths = lengths
        self.scale = 0.25
        self.dims = (b, L, H, G, dk, dv)

    @property
    def g(self):
        g = np.zeros(self.v.shape[:3])
        if self.log_decay is not None:
            g = g + self.log_decay
        if self.head is not None:
            g = g + self.head
        return g

    def t(self, name):
        a = getattr(self, name)
        if a is None:
            return None
        if name == "lengths":
            return torch.tensor(a, dtype=torch.int32, device="cuda")
        ty = torch.float32 if name in ("head", "h0", "dh") else self.ty
        return torch.from_numpy(a).to("cuda", torch.float32).to(ty)

    def run(self, attn, q=None, k=None, v=None, **kw):
        return attn(self.t("q") if q is None else q,
                    self.t("k") if k is None else k,
                    self.t("v") if v is None else v,
                    log_decay=self.t("log_decay"),
                    head_log_decay=self.t("head"), scale=self.scale,
                    lengths=self.t("lengths"), h0=self.t("h0"), **kw)

    def run_back(self, attn, **kw):
        return attn.backward(self.t("q"), self.t("k"), self.t("v"),
                             self.t("dy"), log_decay=self.t("log_decay"),
                             head_log_decay=self.t("head"), scale=self.scale,
                             lengths=self.t("lengths"), h0=self.t("h0"),
                             dh_last=self.t("dh"), **kw)

    def check_forward(self, y, h):
        L = self.dims[1]
        a = (self.q, self.k, self.v, self.g, self.scale)
        ry, rh = M.forward(*a, self.h0, self.lengths)
        ab = [np.abs(x) for x in a[:3]]
        my, mh = M.forward(*ab, self.g, self.scale,
                           None if self.h0 is None else np.abs(self.h0),
                           self.lengths)
        M.check(host(y), ry, M.bound(ry, my, self.dtype, L), "y")
        M.check(host(h), rh, M.bound(rh, mh, self.dtype, L, True, "f32"),
                "h_last")

    def check_backward(self, g, exact=True):
        L = self.dims[1]
        ref = M.backward(self.q, self.k, self.v, self.g, self.scale, self.dy,
                         self.h0, self.dh, self.lengths)
        n = lambda x: None if x is None else np.abs(x)  # noqa: E731
        mag = M.backward(n(self.q), n(self.k), n(self.v), self.g, self.scale,
                         n(self.dy), n(self.h0), n(self.dh), self.lengths,
                         absolute=True)
        dt = self.dtype
        for name in ("dq", "dk", "dv"):
            M.check(host(g[name]), ref[name],
                    M.bound(ref[name], mag[name], dt, L,
                            exact and name != "dv"), name)
        M.check(host(g["dh0"]), ref["dh0"],
                M.bound(ref["dh0"], mag["dh0"], dt, L, True, "f32"), "dh0")
        if g["dlog_decay"] is not None:
            M.check(host(g["dlog_decay"]), ref["dg"],
                    M.bound(ref["dg"], mag["dg"], dt, L, True), "dlog_decay")
        if g["dhead_log_decay"] is not None:
            M.check(host(g["dhead_log_decay"]), ref["dhead"],
                    M.bound(ref["dhead"], mag["dg"].sum((0, 1)), dt, L, True,
                            "f32"), "dhead_log_decay")


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


SHAPES = {
    # name: b, L, H, G, dk, dv
    "one_token": (2, 1, 2, 2, 16, 16),
    "two_tokens_odd": (1, 2, 3, 1, 1, 1),
    "chunk_less_one": (1, 63, 2, 1, 64, 64),
    "chunk": (2, 64, 2, 2, 64, 64),
    "chunk_and_one": (1, 65, 2, 2, 128, 128),
    "odd_sizes": (2, 130, 3, 3, 77, 45),
    "narrow": (1, 100, 4, 2, 8, 8),
    "split": (1, 900, 1, 1, 32, 40),
    "split_wide": (1, 1200, 2, 1, 128, 128),
    "three_tiles": (1, 80, 2, 1, 20, 130),
}


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_prompt(attn, shape, dtype):
    c = Case(dtype, *SHAPES[shape])
    c.check_forward(*c.run(attn))


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("gate", ["token", "head", "none"])
@pytest.mark.parametrize("state", [False, True])
def test_prompt_options(attn, dtype, gate, state):
    c = Case(dtype, 2, 150, 4, 2, 24, 32, gate=gate, state=state, rate=0.5)
    c.check_forward(*c.run(attn))


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("shape", [s for s in sorted(SHAPES)
                                   if s != "three_tiles"])
def test_backward(attn, shape, dtype):
    c = Case(dtype, *SHAPES[shape])
    c.check_backward(c.run_back(attn))


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("gate", ["token", "head", "none"])
@pytest.mark.parametrize("state", [False, True])
def test_backward_options(attn, dtype, gate, state):
    c = Case(dtype, 2, 150, 4, 2, 24, 32, gate=gate, state=state, rate=0.5)
    c.check_backward(c.run_back(attn), exact=gate != "none")
    g = c.run_back(attn, decay_gradient=False)
    assert g["dlog_decay"] is None and g["dhead_log_decay"] is None
    c.check_backward(g, exact=False)


# around the ends of the 128-step chunks and the weighted slots inside them
@pytest.mark.parametrize("L", [31, 33, 80, 113, 127, 128, 129, 256, 300, 385])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128),
                                   (128, 128), (24, 96)])
def test_chunk_ends(attn, L, dk, dv):
    c = Case("bf16", 1, L, 2, 1, dk, dv, rate=0.3)
    c.check_forward(*c.run(attn))
    c.check_backward(c.run_back(attn))
    c.head = None       # the token's decay alone: the gradients' other kernel
    c.check_backward(c.run_back(attn))
    assert attn.sync_status() == S.SSM_OK


def test_more_heads_than_multiprocessors(attn):
    """The last, ill-filled round of heads runs cut into segments."""
    heads = torch.cuda.get_device_properties(0).multi_processor_count + 5
    c = Case("bf16", 1, 1100, heads, heads, 16, 16, gate="token")
    c.check_forward(*c.run(attn))
    c.lengths = [1061]
    c.check_forward(*c.run(attn))


LENGTHS = {"short_long": (200, [0, 1, 64, 200, 130]),
           "inside_a_chunk": (400, [399, 257, 255, 128, 100, 1]),
           "outside": (70, [-3, 90, 70, 69, 2]),
           "all_empty": (64, [0, 0]),
           "split": (1500, [1500, 700])}


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("name", sorted(LENGTHS))
def test_padded_batches(attn, name, dtype):
    """What stands behind a sequence is never read: NaN and infinity there
    change nothing, and the rows there come back as zeros."""
    L, lengths = LENGTHS[name]
    b = len(lengths)
    c = Case(dtype, b, L, 2, 1, 32, 24, lengths=lengths,
             gate="token" if dtype == "bf16" else "both")
    y0, h0 = c.run(attn)
    c.check_forward(y0, h0)
    g0 = c.run_back(attn)
    c.check_backward(g0)
    for i, n in enumerate(lengths):
        n = min(max(n, 0), L)
        for a in (c.q, c.k, c.v, c.log_decay, c.dy):
            a[i, n:] = np.nan
            a[i, n + 1:] = np.inf
    y1, h1 = c.run(attn)
    g1 = c.run_back(attn)
    assert torch.equal(y0, y1) and torch.equal(h0, h1)
    for k in g0:
        assert g0[k] is None or torch.equal(g0[k], g1[k]), k
    assert attn.sync_status() == S.SSM_OK
    for i, n in enumerate(lengths):
        n = min(max(n, 0), L)
        assert not y1[i, n:].any() and not g1["dv"][i, n:].any()
        assert not g1["dq"][i, n:].any() and not g1["dlog_decay"][i, n:].any()


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("value", [-np.inf, -100.0, -90.0])
def test_restarts(attn, dtype, value):
    """A decay of 0 starts the state anew, several times in one chunk, at its
    first and last step and at a segment's, whatever the state held."""
    c = Case(dtype, 2, 700, 2, 2, 16, 16, gate="token")
    for t in (0, 1, 10, 11, 40, 63, 64, 127, 128, 255, 256, 511, 699):
        c.log_decay[:, t] = value
    c.check_forward(*c.run(attn))
    c.check_backward(c.run_back(attn))
    c.h0 = c.h0 * np.inf     # infinities and NaN in the state in front
    y, h = c.run(attn)
    c.h0 = np.zeros_like(c.h0)
    c.check_forward(y, h)


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_a_restart_has_no_decay_gradient(attn, dtype):
    c = Case(dtype, 2, 300, 4, 2, 32, 16, gate="token")
    at = [0, 5, 63, 64, 128, 299]
    c.log_decay[:, at] = -np.inf
    g = c.run_back(attn)["dlog_decay"]
    assert not g[:, at].any() and bool(g.isfinite().all())


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_decay_extremes(attn, dtype):
    """Strong decays next to none: the differences of the sums stay exact."""
    c = Case(dtype, 1, 256, 2, 2, 16, 16, gate="token")
    c.log_decay[:, ::3] = -80.0
    c.log_decay[:, 1::3] = 0.0
    c.check_forward(*c.run(attn))
    c.check_backward(c.run_back(attn))
    c.log_decay[:] = M.bf16(np.full_like(c.log_decay, 0.01))   # it may grow
    c.check_forward(*c.run(attn))


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("pad", [8, 1])
def test_slices_of_a_wider_row(attn, dtype, pad):
    """q, k and v as columns of one projection, aligned and not."""
    c = Case(dtype, 2, 100, 4, 2, 32, 16)
    b, L, H, G, dk, dv = c.dims
    w = G * dk * 2 + H * dv + 2 * pad
    row = torch.full((b, L, w), float("nan"), dtype=c.ty, device="cuda")
    cuts = [pad, pad + G * dk, pad + 2 * G * dk]
    q = row[..., cuts[0]:cuts[1]].unflatten(-1, (G, dk))
    k = row[..., cuts[1]:cuts[2]].unflatten(-1, (G, dk))
    v = row[..., cuts[2]:cuts[2] + H * dv].unflatten(-1, (H, dv))
    for dst, name in ((q, "q"), (k, "k"), (v, "v")):
        dst.copy_(c.t(name))
    y, h = c.run(attn, q=q, k=k, v=v)
    c.check_forward(y, h)
    g = attn.backward(q, k, v, c.t("dy"), log_decay=c.t("log_decay"),
                      head_log_decay=c.t("head"), scale=c.scale,
                      h0=c.t("h0"), dh_last=c.t("dh"))
    c.check_backward(g)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("shape", [(1, 2, 1, 16, 16), (3, 4, 2, 77, 45),
                                   (5, 6, 3, 128, 128), (2, 2, 2, 1, 1),
                                   (4, 3, 1, 64, 200), (300, 8, 8, 64, 64)])
def test_steps_follow_the_prompt(attn, shape, dtype):
    """Token by token with the state in place: each step within its bound of
    the recurrence from the kernel's own state, the last state that of the
    prompt."""
    b, H, G, dk, dv = shape
    T = 4
    c = Case(dtype, b, T, H, G, dk, dv)
    state = c.t("h0")
    q, k, v, g = (c.t(n) for n in ("q", "k", "v", "log_decay"))
    for t in range(T):
        before = host(state)
        y = attn.step(q[:, t], k[:, t], v[:, t], state,
                      log_decay=g[:, t].contiguous(),
                      head_log_decay=c.t("head"), scale=c.scale)
        one = [x[:, t:t + 1] for x in (c.q, c.k, c.v, c.g)]
        ry, rs = M.forward(*one, c.scale, before)
        my, ms = M.forward(*[np.abs(x) for x in one[:3]], one[3], c.scale,
                           np.abs(before))
        # float32 sums of dk terms in some order, each factor exact
        u = M.U[dtype]
        M.check(host(y), ry[:, 0], u * np.abs(ry[:, 0])
                + (dk + 8) * 2.0 ** -23 * my[:, 0] + 1e-30, "y")
        M.check(host(state), rs, 2.0 ** -21 * ms + 1e-30, "state")
    y, h = c.run(attn)
    ms = M.forward(np.abs(c.q), np.abs(c.k), np.abs(c.v), c.g, c.scale,
                   np.abs(c.h0))[1]
    M.check(host(state), host(h), M.bound(host(h), ms, dtype, T, True, "f32")
            * 2, "state after the prompt")


def test_step_restarts_a_used_state(attn):
    state = torch.full((2, 2, 8, 8), float("nan"), device="cuda")
    q, k, v = (torch.ones(2, 2, 8, device="cuda") for _ in range(3))
    g = torch.full((2, 2), -float("inf"), device="cuda")
    y = attn.step(q, k, v, state, log_decay=g, scale=1.0)
    assert torch.equal(state, torch.ones_like(state))
    assert torch.equal(y, torch.full_like(y, 8.0))


def test_a_prompt_in_pieces(attn):
    """The state carries: two pieces give what the whole gives, in place."""
    c = Case("f32", 2, 333, 4, 2, 48, 32)
    b, L, H, G, dk, dv = c.dims
    y, h = c.run(attn)
    q, k, v, g = (c.t(n) for n in ("q", "k", "v", "log_decay"))
    state = c.t("h0")
    parts = []
    for s in (slice(0, 101), slice(101, L)):
        yp, hp = attn(q[:, s].contiguous(), k[:, s].contiguous(),
                      v[:, s].contiguous(), log_decay=g[:, s].contiguous(),
                      head_log_decay=c.t("head"), scale=c.scale, h0=state,
                      h_last=state)
        assert hp is state
        parts.append(yp)
    my, mh = M.forward(np.abs(c.q), np.abs(c.k), np.abs(c.v), c.g, c.scale,
                       np.abs(c.h0))
    M.check(host(torch.cat(parts, 1)), host(y),
            2 * M.bound(host(y), my, "f32", L), "y")
    M.check(host(state), host(h), 2 * M.bound(host(h), mh, "f32", L), "h")


def test_the_same_on_every_run_and_stream(attn):
    c = Case("bf16", 1, 1100, 4, 2, 64, 64)
    y, h = c.run(attn)
    g = c.run_back(attn)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:      # one object, several streams at once
        with torch.cuda.stream(s):
            got.append((c.run(attn), c.run_back(attn)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got.append((c.run(attn, stream=side), c.run_back(attn, stream=side)))
    torch.cuda.synchronize()
    for (y2, h2), g2 in got:
        assert torch.equal(y, y2) and torch.equal(h, h2)
        for k in g:
            assert torch.equal(g[k], g2[k]), k


def test_captured_calls_replay(attn):
    """Prompt, backward and steps captured in two graphs, replayed in turn
    with new inputs, against eager calls."""
    a, b = Case("bf16", 2, 700, 4, 2, 64, 64), Case("bf16", 2, 700, 4, 2, 64,
                                                    64, seed=9)
    ins = {n: a.t(n) for n in ("q", "k", "v", "log_decay", "head", "h0", "dy",
                               "dh")}
    c_state = a.t("h0")

    def calls():
        y, h = attn(ins["q"], ins["k"], ins["v"], log_decay=ins["log_decay"],
                    head_log_decay=ins["head"], h0=ins["h0"])
        g = attn.backward(ins["q"], ins["k"], ins["v"], ins["dy"],
                          log_decay=ins["log_decay"],
                          head_log_decay=ins["head"], h0=ins["h0"],
                          dh_last=ins["dh"])
        ys = attn.step(ins["q"][:, 0], ins["k"][:, 0], ins["v"][:, 0],
                       c_state, log_decay=ins["log_decay"][:, 0].contiguous())
        return [y, h, ys] + [g[k] for k in sorted(g)]

    graphs, outs = [], []
    calls()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(calls())
        graphs.append(graph)
    for case in (b, a):
        for n in ins:
            ins[n].copy_(case.t(n))
        c_state.copy_(case.t("h0"))
        want = [x.clone() for x in calls()]
        state = c_state.clone()
        for graph, out in zip(graphs, outs):
            c_state.copy_(case.t("h0"))
            graph.replay()
            torch.cuda.synchronize()
            for x, y in zip(out, want):
                assert torch.equal(x, y)
            assert torch.equal(c_state, state)


def test_raw_streams(attn):
    c = Case("bf16", 1, 300, 2, 2, 32, 32)
    y, h = c.run(attn)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (0, side.cuda_stream, side):
        y2, h2 = c.run(attn, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(h, h2)


FIRST = """
import torch
import selective_state_space_51_b200 as S
attn, norm = S.LinearAttention(), S.LayerNorm()
q = torch.randn(1, 300, 2, 32, device="cuda", dtype=torch.%s)
x = torch.randn(64, 96, device="cuda")
w = torch.ones(96, device="cuda")
state = torch.zeros(1, 2, 32, 32, device="cuda")

def calls():
    y, h = attn(q, q, q)
    g = attn.backward(q, q, q, q)
    state.zero_()
    s = attn.step(q[:, 0], q[:, 0], q[:, 0], state)
    f = norm(x, w)
    b = norm.backward(x, x, f["mean"], f["rstd"], w)
    return [y, h, s, f["y"], b["dx"], b["dweight"]] + [
        g[n] for n in ("dq", "dk", "dv", "dh0")]

graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(got, calls()):
    assert torch.equal(a, b)
print("same")
"""


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_the_first_call_of_a_process_is_captured(dtype):
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", FIRST % dtype], text=True,
                       capture_output=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_far_tokens(attn):
    """Offsets past 2^31 elements: the last sequence of a batch whose rows
    lie far apart gives what it gives alone."""
    b, L, H, d, stride = 2, 130, 1, 16, 9_000_000   # b L stride = 2.3e9
    row = torch.empty((b, L, stride), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (row[..., i * d:(i + 1) * d].unflatten(-1, (H, d))
               for i in range(3))
    for t in (q, k, v):
        t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
    y, h = attn(q, k, v)
    y1, h1 = attn(q[1:].contiguous(), k[1:].contiguous(), v[1:].contiguous())
    assert torch.equal(y[1:], y1) and torch.equal(h[1:], h1)


def test_refused_tensors(attn):
    q = torch.zeros(2, 8, 2, 16, device="cuda")
    v = torch.zeros(2, 8, 4, 16, device="cuda")
    ok = dict(q=q, k=q, v=v)
    attn(**ok)
    for bad in (dict(k=q.bfloat16()), dict(v=v.cpu()), dict(k=q[:, :4]),
                dict(v=v[:, :, :3]), dict(q=q.transpose(1, 2)),
                dict(q=q[:, :1].expand(2, 8, 2, 16)),
                dict(log_decay=torch.zeros(2, 8, 2, device="cuda")),
                dict(head_log_decay=torch.zeros(4, device="cuda").bfloat16()),
                dict(lengths=torch.zeros(2, device="cuda")),
                dict(h0=torch.zeros(2, 4, 16, 8, device="cuda")),
                dict(y=torch.zeros(2, 8, 4, 8, device="cuda"))):
        with pytest.raises(ValueError):
            attn(**{**ok, **bad})
    with pytest.raises(TypeError):
        attn(q.half(), q.half(), v.half())
    with pytest.raises(ValueError):
        attn.backward(q, q, v, None)
    for empty in (dict(q=q[..., :0], k=q[..., :0]), dict(q=q[:, :, :0]),
                  dict(v=v[:, :, :0]), dict(q=q[:, :0], k=q[:, :0],
                                            v=v[:, :0])):
        with pytest.raises(ValueError):
            attn(**{**ok, **empty})
    with pytest.raises(S.SsmScanError):
        attn(**ok, y=v)
    with pytest.raises(S.SsmScanError) as e:
        wide = torch.zeros(1, 4, 1, 130, device="cuda")
        attn(wide, wide, torch.zeros(1, 4, 1, 8, device="cuda"))
    assert e.value.status == S.SSM_ERR_UNSUPPORTED
