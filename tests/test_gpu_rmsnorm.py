"""The residual RMS norm with its 8-bit outputs, and its backward pass, against the fp64 definition.

Bounds.  u is half a step (fp32 2^-24, bf16 2^-8).  A sum of d squares goes through at most 32 additions in a thread,
5 in a warp and 15 across warps, plus the product and the division: its relative error is below 55 u, the square root
halves it, and 2 more roundings follow: rstd within 30 u.  y has two more products and the sum x + r (one rounding of
s, relative to |s|): 33 u |y|, and the output's own rounding.  An 8-bit value is within half a step of e4m3 (2^-4
relative, 2^-10 scale below its normal range) of y, its scale within 34 u.
Backward: the mean of n products is off by 60 u mean |gw xhat|; dx = ds + rstd (gw - xhat mean) adds four roundings of
its terms.  dw sums rows / parts products in a thread, then parts in the second kernel: (rows + 20) u of the sum of
magnitudes bounds both.
"""
import numpy as np
import pytest
import torch

import oracle.attn as oa
from attn_util import U, f64

pytestmark = pytest.mark.gpu
EPS = 1e-5
u = 2.0 ** -24


def lib():
    import gated_delta_rule_105_b200 as g
    return g


def draw(rows, d, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(rows, d, generator=g).to(dt), (3 * torch.randn(rows, d, generator=g)).to(dt),
            1 + 0.3 * torch.randn(d, generator=g)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out,group", [("same", 0), ("e4m3", 0), ("e4m3", 128)])
@pytest.mark.parametrize("rows,d", [(1, 8), (1, 128), (5, 256), (3, 1024), (2, 1032), (7, 1920), (2, 4096), (3, 5000),
                                    (2, 8192), (1, 16384), (700, 128)])
@pytest.mark.parametrize("residual", [True, False])
def test_forward(dt, out, group, rows, d, residual):
    if group and d % group:
        pytest.skip("128-channel scales need d to be a multiple of 128")
    x, r, w = draw(rows, d, dt, rows * d)
    r = r if residual else None
    got = lib().add_rmsnorm_fwd(x.cuda(), w.cuda(), None if r is None else r.cuda(), EPS,
                                torch.float8_e4m3fn if out == "e4m3" else dt, group)
    s, rstd, y = oa.add_rmsnorm(f64(x), None if r is None else f64(r), f64(w), EPS)
    assert np.all(np.abs(f64(got["s"]) - s) <= U[dt] * np.abs(s) * (1 if residual else 0))
    assert np.all(np.abs(f64(got["rstd"]) - rstd) <= 30 * u * rstd)
    if out == "same":
        assert got["scale"] is None
        assert np.all(np.abs(f64(got["y"]) - y) <= 33 * u * np.abs(y) + U[dt] * np.abs(y) * (1 + 33 * u))
        return
    parts = np.abs(y).reshape(rows, -1, group or d)
    scale = parts.max(-1) / 448
    gs = f64(got["scale"]).reshape(scale.shape)
    assert np.all(np.abs(gs - scale) <= 36 * u * scale)
    val = oa.e4m3_value(got["y"].cpu().view(torch.uint8).numpy()).reshape(parts.shape) * gs[..., None]
    ys = y.reshape(parts.shape)
    bound = np.maximum(2.0 ** -4 * np.abs(ys), 2.0 ** -10 * gs[..., None]) + 72 * u * np.abs(ys)
    assert np.all(np.abs(val - ys) <= bound)


def test_stream_updated_in_place_and_zero_and_nan_rows():
    g = lib()
    x, r, w = draw(4, 512, torch.bfloat16, 3)
    x[1], r[1] = 0, 0
    x[2, 7] = float("nan")
    rd = r.cuda()
    got = g.add_rmsnorm_fwd(x.cuda(), w.cuda(), rd, EPS, torch.float8_e4m3fn, 0, s=rd)
    assert got["s"].data_ptr() == rd.data_ptr()
    want = g.add_rmsnorm_fwd(x.cuda(), w.cuda(), r.cuda(), EPS, torch.float8_e4m3fn, 0)
    for k in ("s", "rstd", "scale"):
        assert torch.equal(torch.nan_to_num(got[k].float(), 7.0), torch.nan_to_num(want[k].float(), 7.0))
    assert torch.equal(got["y"].view(torch.uint8), want["y"].view(torch.uint8))
    y = got["y"].float()
    assert (y[1] == 0).all() and torch.isfinite(got["scale"][1])
    assert torch.isnan(y[2]).all() and torch.isnan(got["scale"][2])
    assert torch.isfinite(y[[0, 3]]).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", [(1, 8), (2, 128), (5, 1000), (300, 256), (7, 1032), (601, 2048), (3, 4096), (2, 16384)])
@pytest.mark.parametrize("with_ds", [True, False])
def test_backward(dt, rows, d, with_ds):
    g = lib()
    s, dy, w = draw(rows, d, dt, rows + d)
    ds = draw(rows, d, dt, 7 * rows + d)[0] if with_ds else None
    rstd = (1 / torch.sqrt(s.double().square().mean(-1) + EPS)).float()
    got = g.add_rmsnorm_bwd(dy.cuda(), s.cuda(), w.cuda(), rstd.cuda(), None if ds is None else ds.cuda())
    S, DY, W, R = f64(s), f64(dy), f64(w), f64(rstd)[:, None]
    dx, dw = oa.add_rmsnorm_grads(DY, S, W, R[:, 0], None if ds is None else f64(ds))
    xhat, gw = S * R, DY * W
    m = np.mean(np.abs(gw * xhat), -1, keepdims=True)
    terms = np.abs(R * gw) + np.abs(R * xhat) * m + (0 if ds is None else np.abs(f64(ds)))
    assert np.all(np.abs(f64(got["dx"]) - dx) <= 6 * u * terms + 60 * u * np.abs(R * xhat) * m + U[dt] * np.abs(dx) * (1 + 2.0 ** -7))
    assert np.all(np.abs(f64(got["dweight"]) - dw) <= (rows + 20) * u * np.sum(np.abs(DY * xhat), 0))


def test_backward_in_place_repeats_to_the_bit_and_of_no_rows():
    g = lib()
    s, dy, w = draw(400, 640, torch.bfloat16, 1)
    ds = draw(400, 640, torch.bfloat16, 2)[0]
    rstd = torch.rsqrt(s.float().square().mean(-1) + EPS)
    dev = [t.cuda() for t in (dy, s, w, rstd)]
    a = g.add_rmsnorm_bwd(*dev, ds.cuda())
    for target in ("dy", "ds"):
        d2, s2 = dy.cuda(), ds.cuda()
        b = g.add_rmsnorm_bwd(d2, *dev[1:], s2, dx=d2 if target == "dy" else s2)
        assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])
    none = g.add_rmsnorm_bwd(dev[0][:0], dev[1][:0], dev[2], dev[3][:0])
    assert none["dx"].shape == (0, 640) and (none["dweight"] == 0).all()


def test_gradients_agree_with_differences():
    """Through the forward kernel itself, in fp32: directional differences of <dy, y> + <ds, s>."""
    g = lib()
    x, r, w = draw(6, 384, torch.float32, 5)
    dy, ds, dirs = draw(6, 384, torch.float32, 6)[0], draw(6, 384, torch.float32, 7)[0], draw(6, 384, torch.float32, 8)
    dw_dir = draw(1, 384, torch.float32, 9)[0][0]

    def loss(x, r, w):
        o = g.add_rmsnorm_fwd(x.cuda(), w.cuda(), r.cuda(), EPS)
        return float((o["y"].double().cpu() * dy.double()).sum() + (o["s"].double().cpu() * ds.double()).sum()), o

    _, o = loss(x, r, w)
    got = g.add_rmsnorm_bwd(dy.cuda(), o["s"], w.cuda(), o["rstd"], ds.cuda())
    # a step of 2^-6: the difference's own error is its third derivative (relative ~2^-12), and the losses' fp32
    # roundings, 2304 terms of ~2^-22 in quadrature over 2^-5, are below 1e-3
    h = 2.0 ** -6
    for dx, dr, dw in ((dirs[0], 0, 0), (0, dirs[0], 0), (0, 0, dw_dir)):
        num = (loss(x + h * dx, r + h * dr, w + h * dw)[0] - loss(x - h * dx, r - h * dr, w - h * dw)[0]) / (2 * h)
        want = float((got["dx"].double().cpu() * (torch.as_tensor(dx) + torch.as_tensor(dr)).double()).sum()
                     + (got["dweight"].double().cpu() * torch.as_tensor(dw).double()).sum())
        size = float((got["dx"].double().cpu().abs() * (torch.as_tensor(dx).abs() + torch.as_tensor(dr).abs()).double()).sum()
                     + (got["dweight"].double().cpu().abs() * torch.as_tensor(dw).abs().double()).sum())
        assert abs(num - want) <= 2e-3 + 2.0 ** -11 * size


@pytest.mark.parametrize("out", [None, torch.float8_e4m3fn])
def test_forward_and_backward_captured_and_on_another_stream(out):
    """One graph of both passes, replayed on new values beside an eager call on another stream."""
    g = lib()
    x, r, w = (t.cuda() for t in draw(700, 1024, torch.bfloat16, 11))
    dy = draw(700, 1024, torch.bfloat16, 12)[0].cuda()
    ws = torch.empty(g.add_rmsnorm_bwd_workspace_bytes(700, 1024), dtype=torch.uint8, device="cuda")

    def both(x, ws):
        o = g.add_rmsnorm_fwd(x, w, r, EPS, out, 128 if out else 0)
        return {**o, **g.add_rmsnorm_bwd(dy, o["s"], w, o["rstd"], None, workspace=ws)}

    both(x, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(x, ws)
    other = torch.cuda.Stream()
    for seed in (21, 22, 23):
        x.copy_(draw(700, 1024, torch.bfloat16, seed)[0])
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            want = both(x, None)
        torch.cuda.synchronize()
        for k, t in want.items():
            assert t is None or torch.equal(t.view(torch.uint8), got[k].view(torch.uint8)), k


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [0, 128])
def test_8_bit_scales_over_fp32_s_range(dt, group):
    """Weights whose outputs come close to fp32's largest number, and to its smallest normal one."""
    x, _, w = draw(5, 256, dt, 13)
    for size in (5e37, 1e-24):
        got = lib().add_rmsnorm_fwd(x.cuda(), (w * size).cuda(), None, EPS, torch.float8_e4m3fn, group)
        y = oa.add_rmsnorm(f64(x), None, f64(w * size), EPS)[2]
        gs = f64(got["scale"]).repeat(group or 256, -1)
        val = oa.e4m3_value(got["y"].cpu().view(torch.uint8).numpy()) * gs
        assert np.all(np.abs(val - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * gs) + 72 * u * np.abs(y))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("d", [256, 1024, 4096])
def test_8_bit_scales_are_the_largest_output_over_448(dt, group, d):
    """Given rstd, every step to a scale has one fp32 value: (s rstd) w, the largest magnitude, and its quotient by 448,
    rounded once each.  The scales are those, to the bit."""
    x, r, w = draw(200, d, dt, 17)
    got = lib().add_rmsnorm_fwd(x.cuda(), w.cuda(), r.cuda(), EPS, torch.float8_e4m3fn, group)
    s = x.float().numpy() + r.float().numpy()
    y = (s * got["rstd"].cpu().numpy()[:, None]) * w.numpy()
    assert y.dtype == np.float32
    want = np.abs(y).reshape(200, -1, group or d).max(-1) / np.float32(448)
    assert np.array_equal(got["scale"].cpu().numpy().reshape(want.shape), want)


def test_gradients_agree_with_differences_where_the_mean_counts():
    """Through the forward kernel, in fp32: differences of <dy, y> along the normed rows themselves (and along the weight), with
    a dy that goes with them.  y does not change along its own row, so dx . xhat is all but 0, and only because the mean
    term takes away rstd sum gw xhat, some 130 per row.

    The bound: what the difference quotient of the fp64 definition misses of its derivative; the kernel's error in y, within
    34 u |y| at either end of a step 2 h; and that of the gradients (see the head of the file)."""
    g = lib()
    h = 2.0 ** -4
    x, r, w = draw(6, 384, torch.float32, 5)
    W = f64(w)
    S, R, _ = oa.add_rmsnorm(f64(x), f64(r), W, EPS)
    xhat = torch.from_numpy(S * R[:, None]).float()
    dy = xhat * w
    DY, XH = f64(dy), f64(xhat)

    def both(x, r, w):  # <dy, y> of the kernel and of the definition, and the kernel's outputs
        o = g.add_rmsnorm_fwd(x.cuda(), w.cuda(), r.cuda(), EPS)
        return float((f64(o["y"]) * DY).sum()), float((oa.add_rmsnorm(f64(x), f64(r), f64(w), EPS)[2] * DY).sum()), o

    o = both(x, r, w)[2]
    got = g.add_rmsnorm_bwd(dy.cuda(), o["s"], w.cuda(), o["rstd"])
    dx, dw = oa.add_rmsnorm_grads(DY, S, W, R)
    gw, xh, rs = DY * W, S * R[:, None], R[:, None]
    m = np.mean(np.abs(gw * xh), -1, keepdims=True)
    e_dx = (64 * u * (np.abs(rs * gw) + np.abs(rs * xh) * m) + 60 * u * np.abs(rs * xh) * m)  # with rstd's and s's own errors
    e_dw = (6 + 20 + 34) * u * np.sum(np.abs(DY * xh), 0)
    for a, b, c in ((xhat, 0, 0), (0, xhat, 0), (0, 0, w)):
        (n1, d1, _), (n0, d0, _) = both(x + h * a, r + h * b, w + h * c), both(x - h * a, r - h * b, w - h * c)
        num, num64 = (n1 - n0) / (2 * h), (d1 - d0) / (2 * h)
        along = f64(torch.as_tensor(a)) + f64(torch.as_tensor(b))
        exact = float((dx * along).sum() + (dw * f64(torch.as_tensor(c))).sum())
        want = float((f64(got["dx"]) * along).sum() + (f64(got["dweight"]) * f64(torch.as_tensor(c))).sum())
        size = float(np.sum(np.abs(DY * xh * W)) * (1 + h))
        tol = abs(num64 - exact) + 34 * u * size / h + float(np.sum(e_dx * np.abs(along)) + np.sum(e_dw * np.abs(f64(torch.as_tensor(c)))))
        assert tol < 1.0 and abs(num - want) <= tol, (num, want, tol)
        if c is not w:  # gradients whose mean term is missing, halved, doubled or turned round are far outside
            for factor in (0.0, 0.5, 2.0, -1.0):
                wrong = rs * gw - factor * rs * xh * np.mean(gw * xh, -1, keepdims=True)
                assert abs(num - float((wrong * along).sum())) > 100 * tol
