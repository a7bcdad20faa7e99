"""Layer norm on the GPU, forward and backward, against the float64 oracle.

Allowed errors, with e = 2^-24 (half a step of fp32), n = d: the sums of a row go through
at most 8 additions in a thread's pack per pack it holds, five of a warp's and 32 of a
CTA's warps; S = 120 bounds that for every width here.  With M = max|x| of a row and
s = 1/rstd, mean is off by S e mean|x|; x - mean by 2 e M more; rstd by (S + 8) e
relative, and by what an error of mean does (second order).  An output stored in bf16 is
off by 2^-8 of itself besides."""
import numpy as np
import pytest
import torch

import chunkwise_linear_rnn_fwd_b200 as pkg
from oracle import layernorm as oracle

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
E = 2.0 ** -24
S = 120
HALF = {BF16: 2.0 ** -8, F32: E}

WIDTHS = [1, 2, 7, 64, 200, 256, 264, 1000, 1001, 1024, 1032, 2048, 2050, 4096, 4104, 8192, 9000, 16384]


def inputs(rows, d, dtype, seed=0, offset=0.5, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, d, generator=g) * scale + offset).to(dtype)
    dy = torch.randn(rows, d, generator=g).to(dtype)
    w = 1 + 0.3 * torch.randn(d, generator=g)
    b = 0.3 * torch.randn(d, generator=g)
    return x, dy, w, b


def n64(t):
    return t.detach().double().cpu().numpy()


def check_fwd(x, w, b, got, eps=1e-5):
    y, mean, rstd = (n64(t) for t in got)
    X = n64(x)
    W = np.ones(X.shape[1]) if w is None else n64(w)
    ry, rm, rr = oracle.fwd(X, W, None if b is None else n64(b), eps)
    M = np.abs(X).max(1)
    dm = S * E * np.abs(X).mean(1) + E * np.abs(rm)
    assert np.all(np.abs(mean - rm) <= dm + 1e-30)
    dr = (S + 8) * E + 0.5 * (dm * rr) ** 2 + 4 * E * M * rr  # relative
    assert np.all(np.abs(rstd - rr) <= dr * rr)
    c = np.abs(X - rm[:, None]) * rr[:, None]
    tol = np.abs(W) * (c * (dr + 4 * E)[:, None] + ((dm + 2 * E * M) * rr)[:, None]) * 1.01
    tol = tol + 2 * E * np.abs(ry) + (0 if b is None else E * np.abs(n64(b)))
    tol = tol + HALF[x.dtype] * (np.abs(ry) + tol) + 1e-30
    assert np.all(np.abs(y - ry) <= tol), float(np.max(np.abs(y - ry) / tol))


def check_bwd(x, dy, mean, rstd, w, got):
    dx, dw, db = (None if t is None else n64(t) for t in got)
    X, DY, m, r = n64(x), n64(dy), n64(mean), n64(rstd)
    W = np.ones(X.shape[1]) if w is None else n64(w)
    rdx, rdw, rdb = oracle.bwd(X, DY, m, r, W)
    xh = np.abs(X - m[:, None]) * r[:, None]
    dxh = 3 * E * xh + E * (np.abs(m) * r)[:, None]
    g = np.abs(DY * W)
    s1 = (S + 4) * E * g.mean(1, keepdims=True)
    s2 = (S + 8) * E * (g * xh).mean(1, keepdims=True) + (g * dxh).mean(1, keepdims=True)
    B2 = np.abs((DY * W * (X - m[:, None]) * r[:, None]).mean(1, keepdims=True))
    tol = r[:, None] * (6 * E * (g + np.abs((DY * W).mean(1, keepdims=True)) + xh * B2) + s1 + xh * s2 + dxh * B2)
    tol = tol + HALF[x.dtype] * (np.abs(rdx) + tol) + 1e-30
    assert np.all(np.abs(dx - rdx) <= tol), float(np.max(np.abs(dx - rdx) / tol))
    if dw is None:
        return
    # a CTA's chain over its rows, then the fixed-order sum of the partial ones
    n = X.shape[0] // 128 + 80
    A = (np.abs(DY) * xh).sum(0)
    assert np.all(np.abs(dw - rdw) <= n * E * A + (np.abs(DY) * dxh).sum(0) * 2 + 1e-30)
    assert np.all(np.abs(db - rdb) <= n * E * np.abs(DY).sum(0) + 1e-30)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("rows", [1, 5, 700])
def test_widths(dtype, d, rows):
    x, dy, w, b = inputs(rows, d, dtype, seed=d)
    dev = [t.cuda() for t in (x, dy, w, b)]
    got = pkg.gla_layernorm_fwd(dev[0], dev[2], dev[3])
    check_fwd(x, w, b, got)
    check_bwd(x, dy, got[1], got[2], w, pkg.gla_layernorm_bwd(dev[0], dev[1], got[1], got[2], dev[2]))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_without_weight_bias_or_sums(dtype):
    x, dy, _, _ = inputs(33, 320, dtype, seed=1)
    got = pkg.gla_layernorm_fwd(x.cuda(), eps=1e-3)
    check_fwd(x, None, None, got, eps=1e-3)
    out = pkg.gla_layernorm_bwd(x.cuda(), dy.cuda(), got[1], got[2], want_dwb=False)
    assert out[1] is None and out[2] is None
    check_bwd(x, dy, got[1], got[2], None, out)
    y, mean, rstd = pkg.gla_layernorm_fwd(x.cuda(), eps=1e-3, want_stats=False)
    assert mean is None and rstd is None and torch.equal(y, got[0])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,start", [(512, 64), (512, 3), (77, 1), (2048, 8)])
def test_rows_of_a_wider_matrix(dtype, d, start):
    """Rows a distance apart, and starting anywhere: what lies between them stays."""
    x, dy, w, b = inputs(19, d, dtype, seed=2)
    big = torch.full((3, 19, d + 70), 7.0, dtype=dtype, device="cuda")
    vx, vg, vo = (big[i, :, start:start + d] for i in range(3))
    vx.copy_(x)
    vg.copy_(dy)
    y, mean, rstd = pkg.gla_layernorm_fwd(vx, w.cuda(), b.cuda(), y=vo)
    check_fwd(x, w, b, (vo, mean, rstd))
    out = pkg.gla_layernorm_bwd(vx, vg, mean, rstd, w.cuda(), dx=vo)
    check_bwd(x, dy, mean, rstd, w, out)
    assert bool((big[:, :, :start] == 7).all()) and bool((big[:, :, start + d:] == 7).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [96, 1536, 5000])
def test_in_place(dtype, d):
    x, dy, w, b = (t.cuda() for t in inputs(50, d, dtype, seed=3))
    y, mean, rstd = pkg.gla_layernorm_fwd(x, w, b)
    z = x.clone()
    assert torch.equal(pkg.gla_layernorm_fwd(z, w, b, y=z)[0], y) and torch.equal(z, y)
    dx, dw, db = pkg.gla_layernorm_bwd(x, dy, mean, rstd, w)
    g = dy.clone()
    out = pkg.gla_layernorm_bwd(x, g, mean, rstd, w, dx=g)
    assert torch.equal(g, dx) and torch.equal(out[1], dw) and torch.equal(out[2], db)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offset,scale", [(1000.0, 1.0), (0.0, 1e-6), (-3.0, 0.0), (0.0, 1e15)])
def test_large_means_and_constant_rows(dtype, offset, scale):
    """A mean far larger than the spread, rows below eps, constant rows, large values."""
    x, dy, w, b = inputs(9, 520, dtype, seed=4, offset=offset, scale=scale)
    got = pkg.gla_layernorm_fwd(x.cuda(), w.cuda(), b.cuda())
    check_fwd(x, w, b, got)
    check_bwd(x, dy, got[1], got[2], w, pkg.gla_layernorm_bwd(x.cuda(), dy.cuda(), got[1], got[2], w.cuda()))


def test_a_row_that_is_not_finite_keeps_to_itself():
    x, dy, w, b = (t.cuda() for t in inputs(6, 300, F32, seed=5))
    bad = x.clone()
    bad[2, 7], bad[4, 0] = float("nan"), float("inf")
    y, mean, rstd = pkg.gla_layernorm_fwd(x, w, b)
    z, m2, r2 = pkg.gla_layernorm_fwd(bad, w, b)
    keep = [0, 1, 3, 5]
    assert torch.equal(z[keep], y[keep]) and torch.equal(m2[keep], mean[keep]) and torch.equal(r2[keep], rstd[keep])
    assert bool(z[2].isnan().all()) and bool(z[4].isnan().all())
    assert torch.equal(pkg.gla_layernorm_bwd(bad, dy, m2, r2, w)[0][keep], pkg.gla_layernorm_bwd(x, dy, mean, rstd, w)[0][keep])


def test_bits_streams_and_graphs():
    x, dy, w, b = (t.cuda() for t in inputs(3000, 1024, BF16, seed=6))
    y, mean, rstd = pkg.gla_layernorm_fwd(x, w, b)
    one = pkg.gla_layernorm_bwd(x, dy, mean, rstd, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    two = pkg.gla_layernorm_bwd(x, dy, mean, rstd, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    xs, gs = x.clone(), dy.clone()
    with torch.cuda.graph(g):
        yc, mc, rc = pkg.gla_layernorm_fwd(xs, w, b)
        three = pkg.gla_layernorm_bwd(xs, gs, mc, rc, w)
    xs.zero_()
    g.replay()
    xs.copy_(x)
    g.replay()
    assert torch.equal(yc, y)
    for a, c, e in zip(one, two, three):
        assert torch.equal(a, c) and torch.equal(a, e)


def test_refusals():
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    m = torch.zeros(4, device="cuda")
    w = torch.ones(64, device="cuda")
    for call in (lambda: pkg.gla_layernorm_fwd(x.half()), lambda: pkg.gla_layernorm_fwd(x, w.bfloat16()),
                 lambda: pkg.gla_layernorm_fwd(x, w[:63]), lambda: pkg.gla_layernorm_fwd(x, w.cpu()),
                 lambda: pkg.gla_layernorm_fwd(x, y=x.float()), lambda: pkg.gla_layernorm_fwd(x.t()),
                 lambda: pkg.gla_layernorm_bwd(x, x[:3], m, m), lambda: pkg.gla_layernorm_bwd(x, x, m[:3], m),
                 lambda: pkg.gla_layernorm_bwd(x, x, m, m.double())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: pkg.gla_layernorm_fwd(x, eps=0.0), lambda: pkg.gla_layernorm_fwd(x[:0]),
                 lambda: pkg.gla_layernorm_bwd(x, x, m, m, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(pkg.GLAError):
            call()
