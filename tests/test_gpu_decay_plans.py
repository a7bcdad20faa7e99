"""Gradients and prompts of decay attention where the batch fills about one or two CTAs an SM,
so that the plan just splits its walks or just does not, with a workspace of exactly the size
that the library asks for: against float64, and nothing written behind the workspace."""
import pytest
import torch

import chunkwise_linear_rnn_fwd_b200 as pkg
from tests.decay_cases import Batch, check, packing, reference, rows, views

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
OK = 0


def on_tc(b):
    return b.dtype == BF16 and b.dk % 8 == 0 and b.dv % 8 == 0


def workspace(*args, **kw):
    """A workspace of the size asked for, and the 64 KB behind it."""
    n = pkg.decay_workspace_size(*args, **kw)
    ws = pkg.alloc_decay_workspace(n + (1 << 16), "cuda")
    ws[n:] = 0xA5
    return ws[:n], ws[n:]


# sequences, heads, tokens, dk, dv: 74 to 444 CTAs for 64 columns, a last piece of a
# contraction of 1, 44 and 64 channels among them
PLANS = [(F32, 20, 4, 128, 64, 320), (F32, 20, 4, 100, 64, 320), (F32, 25, 4, 128, 64, 257), (F32, 5, 4, 65, 256, 320),
         (F32, 37, 2, 200, 40, 576), (F32, 19, 4, 130, 16, 300), (BF16, 20, 4, 128, 33, 300), (BF16, 25, 3, 100, 64, 321),
         (F32, 20, 4, 200, 64, 64), (F32, 37, 2, 200, 64, 64), (F32, 37, 4, 130, 64, 64), (F32, 12, 4, 150, 128, 64),
         (BF16, 20, 4, 400, 64, 64), (BF16, 10, 4, 500, 128, 256), (BF16, 19, 4, 520, 128, 64), (BF16, 10, 4, 400, 64, 512),
         (BF16, 37, 4, 300, 64, 64)]


# equal lengths and falling ones in turn, the first plans with both
@pytest.mark.parametrize("dtype,n,H,T,dk,dv,layout", [
    (*p, x) for i, p in enumerate(PLANS) for j, x in enumerate(("dense", "tokens")) if i < 2 or i % 2 == j])
def test_gradients(dtype, n, H, T, dk, dv, layout):
    lens = [T] * n if layout == "dense" else [max(1, T - 17 * i) for i in range(n)]
    b = Batch(lens, H, dk, dv, dtype, seed=n + dk + dv)
    x = views(b, ("q", "k", "v", "do"), layout)
    p = packing(b, layout)
    ws, behind = workspace(n, H, T if layout == "dense" else b.rows, dk, dv, dtype, True, max_len=p.get("max_len", 0))
    dq, dk_, dv_, dh0 = pkg.gla_decay_bwd(x["q"], x["k"], x["v"], b.ld.cuda(), x["do"], h0=b.h0.cuda(),
                                          dh_final=b.dh.cuda(), workspace=ws, **p)
    assert pkg.poll_status(ws) == OK
    check({"dq": rows(dq), "dk": rows(dk_), "dv": rows(dv_), "dh0": dh0}, reference(b, bwd=True), b, on_tc(b))
    assert bool((behind == 0xA5).all())


@pytest.mark.parametrize("dtype,n,H,T,dk,dv", PLANS[::3])
def test_prompts(dtype, n, H, T, dk, dv):
    b = Batch([max(1, T - 17 * i) for i in range(n)], H, dk, dv, dtype, seed=n + dk + dv)
    x = views(b, ("q", "k", "v"), "tokens")
    p = packing(b, "tokens")
    ws, behind = workspace(n, H, b.rows, dk, dv, dtype, max_len=p["max_len"])
    o, hT = pkg.gla_decay_fwd(x["q"], x["k"], x["v"], b.ld.cuda(), h0=b.h0.cuda(), workspace=ws, **p)
    assert pkg.poll_status(ws) == OK
    check({"o": rows(o), "h_final": hT}, reference(b), b, on_tc(b))
    assert bool((behind == 0xA5).all())
