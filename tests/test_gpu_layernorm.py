"""GPU parity of layer norm (with the residual sum) and its backward pass
with the 64-bit formulas."""
import numpy as np
import pytest
import torch

import mixer_oracle as M
import selective_state_space_51_b200 as S

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
F32 = 2.0 ** -24


@pytest.fixture(scope="module")
def norm():
    return S.LayerNorm(0)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def dev(a, ty=torch.float32):
    return None if a is None else torch.from_numpy(
        np.ascontiguousarray(a)).to("cuda", torch.float32).to(ty)


def data(dtype, rows, dim, residual, affine, seed=0, offset=0.5, size=1.0):
    rng = np.random.default_rng(seed + rows * 3 + dim)
    f32 = lambda a: a.astype(np.float32).astype(np.float64)  # noqa: E731
    act = M.bf16 if dtype == "bf16" else f32
    d = dict(x=act(size * rng.standard_normal((rows, dim)) + offset),
             residual=act(rng.standard_normal((rows, dim)))
             if residual else None,
             weight=f32(1 + 0.3 * rng.standard_normal(dim))
             if affine else None,
             bias=f32(rng.standard_normal(dim)) if affine else None,
             dy=act(rng.standard_normal((rows, dim))),
             dsum=act(rng.standard_normal((rows, dim)))
             if residual else None)
    return d, act


def check(norm, dtype, rows, dim, residual, affine, **kw):
    """Bounds, with u = 2^-24 and n = dim terms to a sum: a float32 sum of n
    terms in a tree at most dim / 32 + 10 deep (a thread adds at most 64, then
    the lanes and warps) is off by (dim / 32 + 42) u of the terms' absolute
    sum at the very most; the statistics inherit that relative to the row's
    mean absolute value (mean) and relative to themselves (rstd: half of the
    variance's), and y and dx a few roundings of their own."""
    d, act = data(dtype, rows, dim, residual, affine, **kw)
    ty = TYPES[dtype]
    out = norm(dev(d["x"], ty), weight=dev(d["weight"]), bias=dev(d["bias"]),
               residual=dev(d["residual"], ty))
    s, mean, rstd, y = M.norm_forward(d["x"], d["residual"], d["weight"],
                                      d["bias"], 1e-5, act)
    n = (min(dim, 64) + 42) * F32
    u = M.U[dtype]
    if residual:
        np.testing.assert_array_equal(host(out["sum"]), s)
    else:
        assert out["sum"] is None
    avg = np.abs(s).mean(1)
    M.check(host(out["mean"]), mean, n * avg + 1e-30, "mean")
    # the variance is taken around the computed mean: off by n relative and by
    # the square of the mean's error
    dm = n * avg
    rel = n + (dm * rstd) ** 2 + 4 * F32
    M.check(host(out["rstd"]), rstd, rstd * rel, "rstd")
    w = 1.0 if d["weight"] is None else np.abs(d["weight"])
    hat = np.abs(s - mean[:, None]) * rstd[:, None]
    tol = (hat * (rel[:, None] + 4 * F32) + (dm * rstd)[:, None]) * w
    tol = tol + (u + 2 * F32) * (np.abs(y) + hat * w)
    if u == F32:
        tol = tol + 2 * F32 * (0 if d["bias"] is None else np.abs(d["bias"]))
    M.check(host(out["y"]), y, tol + 1e-30, "y")

    # backward from the kernel's statistics
    kmean, krstd = host(out["mean"]), host(out["rstd"])
    g = norm.backward(dev(d["dy"], ty), dev(s, ty), out["mean"], out["rstd"],
                      weight=dev(d["weight"]), bias=dev(d["bias"]),
                      dsum=dev(d["dsum"], ty))
    dx, dw, db = M.norm_backward(d["dy"], s, kmean, krstd, d["weight"],
                                 d["dsum"])
    # dx: the terms' absolute values, each with its sums' error
    up = np.abs(d["dy"]) * w
    khat = np.abs(s - kmean[:, None]) * krstd[:, None]
    # s - mean is rounded once: relative to |s| + |mean|, not to itself
    loose = (np.abs(s) + np.abs(kmean)[:, None]) * krstd[:, None] * F32
    mag = up + up.mean(1, keepdims=True) + khat * (up * khat).mean(
        1, keepdims=True)
    tol = krstd[:, None] * ((n + 8 * F32) * mag + loose * (up * khat).mean(
        1, keepdims=True) + khat * (up * loose).mean(1, keepdims=True))
    if d["dsum"] is not None:
        tol = tol + 2 * F32 * np.abs(d["dsum"])
    tol = tol + u * np.abs(dx) * (1 + 2.0 ** -7)
    M.check(host(g["dx"]), dx, tol + 1e-30, "dx")
    if not affine:
        assert g["dweight"] is None and g["dbias"] is None
        return
    # columns: a thread's running sums of at most rows terms, then the blocks'
    depth = min(rows, 64) + rows / 1000 + 200
    M.check(host(g["dweight"]), dw, depth * F32 * (np.abs(d["dy"]) * (
        khat + loose)).sum(0) + (np.abs(d["dy"]) * loose).sum(0) + 1e-30,
        "dweight")
    M.check(host(g["dbias"]), db, depth * F32 * np.abs(d["dy"]).sum(0)
            + 1e-30, "dbias")


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("dim", [1, 2, 7, 8, 16, 31, 32, 40, 64, 77, 96, 128,
                                 136, 256, 500, 511, 512, 768, 1000, 2560,
                                 4096, 5120, 8191, 8192])
def test_widths(norm, dtype, dim):
    check(norm, dtype, 37, dim, True, True)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("dim", [264, 768, 1280, 1792, 2304, 4104, 6144, 6152,
                                 8184])
def test_groups_a_thread(norm, dtype, dim):
    """Two to four 16-byte groups a thread, with and without idle lanes, and
    parameters beyond the small shared memory."""
    check(norm, dtype, 37, dim, True, True)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("dim", [768, 2304])
def test_many_rows_a_block(norm, dtype, dim):
    check(norm, dtype, 3000, dim, True, True)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("rows", [1, 2, 3, 255, 5000])
@pytest.mark.parametrize("dim", [24, 33, 320])
def test_rows(norm, dtype, rows, dim):
    check(norm, dtype, rows, dim, False, True)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("residual,affine", [(False, False), (True, False)])
def test_options(norm, dtype, residual, affine):
    check(norm, dtype, 50, 200, residual, affine)


def test_many_short_rows(norm):
    check(norm, "f32", 200_000, 16, False, True)


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_a_mean_far_from_zero(norm, dtype):
    check(norm, dtype, 20, 300, False, True, offset=1000.0)


def test_constant_rows(norm):
    """No variance: rstd = 1 / sqrt(eps), y = bias, finite gradients."""
    x = torch.full((5, 64), 3.0, device="cuda")
    w, b = torch.ones(64, device="cuda"), torch.arange(64.0, device="cuda")
    out = norm(x, weight=w, bias=b)
    assert torch.equal(out["y"], b.expand(5, 64))
    np.testing.assert_allclose(host(out["rstd"]), 1e-5 ** -0.5,
                               rtol=4 * F32 + 1e-8)
    g = norm.backward(torch.randn(5, 64, device="cuda"), x, out["mean"],
                      out["rstd"], weight=w, bias=b)
    assert torch.isfinite(g["dx"]).all() and not g["dweight"].any()


def test_a_bad_row_stays_alone(norm):
    """Infinity and NaN in one row reach no other row."""
    x = torch.randn(9, 100, device="cuda")
    a = norm(x)
    x[4, 3] = float("inf")
    x[7, 0] = float("nan")
    b = norm(x)
    keep = [0, 1, 2, 3, 5, 6, 8]
    assert torch.equal(a["y"][keep], b["y"][keep])
    assert torch.isnan(b["y"][7]).all()


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_unaligned_buffers(norm, dtype):
    """Rows that start off a 16-byte boundary give what aligned ones give up
    to the order of the sums."""
    d, _ = data(dtype, 40, 256, False, True)
    ty = TYPES[dtype]
    x = dev(d["x"], ty)
    far = torch.empty(40 * 256 + 1, dtype=ty, device="cuda")[1:].view(40, 256)
    far.copy_(x)
    a = norm(x, weight=dev(d["weight"]), bias=dev(d["bias"]))
    b = norm(far, weight=dev(d["weight"]), bias=dev(d["bias"]))
    u = M.U[dtype]
    tol = (2 * u + 300 * F32) * (np.abs(host(a["y"])) + 3)
    M.check(host(b["y"]), host(a["y"]), tol, "y")
    dy = dev(d["dy"], ty)
    ga = norm.backward(dy, x, a["mean"], a["rstd"], weight=dev(d["weight"]))
    gb = norm.backward(dy, far, a["mean"], a["rstd"],
                       weight=dev(d["weight"]))
    M.check(host(gb["dx"]), host(ga["dx"]),
            (2 * u + 600 * F32) * (np.abs(host(ga["dx"])) + 3), "dx")


def test_the_same_on_every_run_and_stream(norm):
    d, _ = data("bf16", 3000, 640, True, True)
    x, r, dy = (dev(d[k], torch.bfloat16) for k in ("x", "residual", "dy"))
    w, b = dev(d["weight"]), dev(d["bias"])

    def both(**kw):
        o = norm(x, weight=w, bias=b, residual=r, **kw)
        g = norm.backward(dy, o["sum"], o["mean"], o["rstd"], weight=w,
                          bias=b, **kw)
        return [o[k] for k in sorted(o)] + [g[k] for k in sorted(g)]

    want = both()
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(s):
            got.append(both())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got.append(both(stream=side))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    graph.replay()
    torch.cuda.synchronize()
    for g in got + [out]:
        for p, q in zip(want, g):
            assert torch.equal(p, q)


def test_in_place(norm):
    x = torch.randn(33, 128, device="cuda")
    want = norm(x)["y"]
    got = norm(x, y=x)["y"]
    assert got is x and torch.equal(want, got)


def test_refused_tensors(norm):
    x = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad in (dict(x=x.t()), dict(x=x.cpu()), dict(weight=w[:32]),
                dict(weight=w.bfloat16()), dict(residual=x.bfloat16()),
                dict(residual=x[:2]), dict(x=x[:0])):
        with pytest.raises(ValueError):
            norm(**{**dict(x=x, weight=w), **bad})
    with pytest.raises(TypeError):
        norm(x.half())
    with pytest.raises(ValueError):
        norm.backward(x, x, None, None)
    with pytest.raises(S.SsmScanError) as e:
        norm(torch.zeros(1, 8200, device="cuda"))
    assert e.value.status == S.SSM_ERR_UNSUPPORTED
