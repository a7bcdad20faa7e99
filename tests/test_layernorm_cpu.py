"""Layer norm without a GPU: the oracle against differences, and the refusals of the calls."""
import ctypes

import numpy as np
import pytest
import torch

import chunkwise_linear_rnn_fwd_b200 as pkg
from oracle import layernorm as oracle

ARG, SHAPE, MIS, WS = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    from chunkwise_linear_rnn_fwd_b200 import build
    build.build()
    return pkg.load()


def test_oracle_gradients_against_differences():
    rng = np.random.default_rng(0)
    x, dy, w, b = rng.standard_normal((5, 7)), rng.standard_normal((5, 7)), rng.standard_normal(7), rng.standard_normal(7)
    loss = lambda x, w, b: (oracle.fwd(x, w, b)[0] * dy).sum()  # noqa: E731
    _, mean, rstd = oracle.fwd(x, w, b)
    g = oracle.bwd(x, dy, mean, rstd, w)
    for i, a in enumerate((x, w, b)):
        u, e = rng.standard_normal(a.shape), 1e-5
        hi, lo = (loss(*(c + s * e * u if j == i else c for j, c in enumerate((x, w, b)))) for s in (1, -1))
        # the third derivative's term, and the rounding of the losses over 2 e
        assert abs((hi - lo) / (2 * e) - (g[i] * u).sum()) <= 1e-8 + 1e-15 * (abs(hi) + abs(lo)) / e


def test_bad_arguments_enqueue_nothing(lib):
    a, mis = 4096, 4098

    def fwd(dtype=0, rows=4, d=64, x=a, ldx=64, w=a, b=a, eps=1e-5, y=a, ldy=64, mean=a, rstd=a):
        return lib.gla_layernorm_fwd(dtype, rows, d, x, ldx, w, b, eps, y, ldy, mean, rstd, None)

    assert fwd(dtype=2) == ARG and fwd(rows=0) == ARG and fwd(d=0) == ARG
    assert fwd(d=16385, ldx=16385, ldy=16385) == SHAPE and fwd(rows=1 << 31) == SHAPE
    assert fwd(x=None) == ARG and fwd(y=None) == ARG and fwd(ldx=63) == ARG and fwd(ldy=0) == ARG
    assert fwd(x=4097) == MIS and fwd(w=mis) == MIS and fwd(b=mis) == MIS and fwd(mean=mis) == MIS and fwd(rstd=mis) == MIS
    assert fwd(dtype=1, x=mis) == MIS
    for eps in (0.0, -1e-5, 1.0, float("nan")):
        assert fwd(eps=eps) == ARG

    def bwd(rows=4, d=64, x=a, dy=a, lddy=64, mean=a, rstd=a, w=a, dx=a, lddx=64, dw=a, db=a, ws=1 << 20, n=1 << 30):
        return lib.gla_layernorm_bwd(0, rows, d, x, 64, dy, lddy, mean, rstd, w, dx, lddx, dw, db, ws, n, None)

    assert bwd(rows=0) == ARG and bwd(d=0) == ARG
    assert bwd(x=None) == ARG and bwd(dy=None) == ARG and bwd(dx=None) == ARG and bwd(mean=None) == ARG
    assert bwd(rstd=None) == ARG and bwd(lddy=63) == ARG and bwd(lddx=63) == ARG
    assert bwd(dy=4097) == MIS and bwd(dx=4097) == MIS and bwd(dw=mis) == MIS and bwd(db=mis) == MIS and bwd(mean=mis) == MIS
    assert bwd(ws=None) == ARG and bwd(ws=(1 << 20) + 8) == MIS
    assert bwd(n=lib.gla_layernorm_workspace_size(4, 64) - 1) == WS
    assert bwd(ws=None, db=None) == ARG


def test_workspace_size(lib):
    size = lib.gla_layernorm_workspace_size
    assert size(0, 64) == 0 and size(4, 0) == 0 and size(4, 16385) == 0
    assert size(1, 64) == 512 and size(10**6, 64) >= size(10**5, 64) > size(4, 64)
    with pytest.raises(pkg.GLAError):
        pkg.layernorm_workspace_size(4, 20000)


def test_tensors_of_the_host_are_refused():
    x = torch.zeros(3, 8)
    with pytest.raises(ValueError):
        pkg.gla_layernorm_fwd(x)
    with pytest.raises(ValueError):
        pkg.gla_layernorm_bwd(x, x, x[:, 0], x[:, 0])
