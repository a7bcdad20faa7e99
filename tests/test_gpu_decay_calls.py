"""How the decay and layer-norm calls are made on the GPU: arguments by keyword, outputs and
workspaces that the call makes or is given, states that many chunks and tokens pass on."""
import ctypes

import pytest
import torch

import chunkwise_linear_rnn_fwd_b200 as pkg
from tests.decay_cases import Batch, packing, views

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def same(one, two):
    for s, t in zip(one, two):
        assert (s is None and t is None) or torch.equal(s, t)


def test_keywords_give_what_positions_give():
    b = Batch([70, 9], 2, 64, 72, BF16, seed=1)
    x, p, ld = views(b, ("q", "k", "v", "do"), "tokens"), packing(b, "tokens"), b.ld.cuda()
    q, k, v, do = (x[n] for n in ("q", "k", "v", "do"))
    same(pkg.gla_decay_fwd(q=q, k=k, v=v, log_decay=ld, **p), pkg.gla_decay_fwd(q, k, v, ld, **p))
    same(pkg.gla_decay_bwd(q=q, k=k, v=v, log_decay=ld, do=do, **p), pkg.gla_decay_bwd(q, k, v, ld, do, **p))
    tok = [t[0, :, :3].transpose(0, 1) for t in (q, k, v)]
    s, t = (torch.zeros(3, 2, 64, 72, device="cuda") for _ in range(2))
    same([pkg.gla_decay_step(q=tok[0], k=tok[1], v=tok[2], log_decay=ld, state=s), s],
         [pkg.gla_decay_step(*tok, ld, t), t])
    r = b.q[:, 0].cuda()
    fwd = pkg.gla_layernorm_fwd(x=r)
    same(fwd, pkg.gla_layernorm_fwd(r))
    same(pkg.gla_layernorm_bwd(x=r, dy=r, mean=fwd[1], rstd=fwd[2]), pkg.gla_layernorm_bwd(r, r, *fwd[1:]))


def poison(nbytes):
    """Leaves NaN in the memory that the next allocations of this size get."""
    x = torch.full((nbytes // 4,), float("nan"), device="cuda")
    torch.cuda.synchronize()
    del x


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (F32, 64), (BF16, 33)])
@pytest.mark.parametrize("given", [(), ("dk",)])
def test_rows_of_no_sequence_are_zero_in_outputs_the_call_makes(dtype, d, given):
    """Rows before the first sequence, behind the last one, and those of a sequence that is
    refused; whatever the memory held."""
    b = Batch([40, 700, 30], 2, d, d, dtype, seed=3, spare=300)
    x, ld = views(b, ("q", "k", "v", "do"), "tokens"), b.ld.cuda()
    q, k, v, do = (x[n] for n in ("q", "k", "v", "do"))
    cu = torch.tensor([7, 40, 740, 770], dtype=torch.int32, device="cuda")
    nobody = torch.ones(b.rows, dtype=torch.bool, device="cuda")
    nobody[7:40] = nobody[740:770] = False  # the second sequence is longer than max_len
    p = {"cu_seqlens": cu, "max_len": 300}
    poison(q.numel() * q.element_size())
    o, _ = pkg.gla_decay_fwd(q, k, v, ld, want_final=False, **p)
    for _ in range(3):
        poison(q.numel() * q.element_size())
    mine = {n: torch.full_like(q, 7.0) for n in given}
    g = dict(zip(("dq", "dk", "dv"), pkg.gla_decay_bwd(q, k, v, ld, do, want_dh0=False, **mine, **p)))
    for name, t in {"o": o, **g}.items():
        assert bool((t[0][:, nobody] == (7.0 if name in given else 0.0)).all()), name
        assert bool(torch.isfinite(t).all()) and bool((t[0][:, ~nobody] != 0.0).any())


def test_workspaces_of_the_host_or_with_gaps_are_refused():
    b = Batch([20], 2, 64, 64, BF16, seed=4)
    x, ld, p = views(b, ("q", "k", "v"), "tokens"), b.ld.cuda(), packing(b, "tokens")
    q, k, v = (x[n] for n in ("q", "k", "v"))
    tok = [t[0, :, :1].transpose(0, 1) for t in (q, k, v)]
    r = b.q[:, 0].cuda()
    _, mean, rstd = pkg.gla_layernorm_fwd(r)
    calls = [lambda ws: pkg.gla_decay_fwd(q, k, v, ld, workspace=ws, **p),
             lambda ws: pkg.gla_decay_bwd(q, k, v, ld, v, workspace=ws, **p),
             lambda ws: pkg.gla_decay_step(*tok, ld, torch.zeros(1, 2, 64, 64, device="cuda"), workspace=ws),
             lambda ws: pkg.gla_layernorm_bwd(r, r, mean, rstd, workspace=ws)]
    for call in calls:
        call(pkg.alloc_decay_workspace(1 << 20, "cuda"))
        for bad in (torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(1 << 21, dtype=torch.uint8, device="cuda")[::2]):
            with pytest.raises(ValueError, match="workspace"):
                call(bad)


def carried(state, h0, ld, tokens):
    """The mean relative error of states [H,..] that only decayed, for each head."""
    want = h0.double() * torch.exp(ld.double() * tokens).view(-1, *[1] * (h0.dim() - 1))
    return ((state.double() / want - 1).flatten(1).mean(1)).abs()


def mean_bound(updates, values):
    """What rounding may leave of the mean: each update rounds a value by at most 2^-24 of it, an
    error of mean zero and at most 2^-24 / sqrt(3) standard deviation.  The errors of one value's
    updates may all be alike (a value hardly changes from one to the next), those of different
    values are independent.  Ten standard deviations."""
    return 10 * 2.0 ** -24 * updates / (3 * values) ** 0.5


# rates whose lambda^64 (first) and lambda^128 lie 0.5 steps of fp32 off the next number
SLOW = (-1.082700009646942e-06, -2.684299943211954e-06)


def test_a_slow_head_decays_right_over_a_long_fp32_sequence():
    """2048 chunks without new tokens: a factor that is off in its last bit would be off the
    same way in each of them, 6e-5 in all."""
    T, dk, dv = 131072, 128, 256
    ld = torch.tensor(SLOW, device="cuda")
    h0 = 1 + torch.rand(1, 2, dk, dv, generator=torch.Generator().manual_seed(5)).cuda()
    k, v = torch.zeros(1, 1, T, dk, device="cuda").expand(1, 2, T, dk), torch.zeros(1, 1, T, dv, device="cuda").expand(1, 2, T, dv)
    o = torch.empty(1, 2, T, dv, device="cuda")
    _, hT = pkg.gla_decay_fwd(k, k, v, ld, h0=h0, o=o, segments=1)
    assert bool((carried(hT[0], h0[0], ld, T) <= mean_bound(T // 64, dk * dv)).all())


def test_a_slow_head_decays_right_token_by_token():
    n, dk, dv = 2000, 128, 256
    ld = torch.tensor([-2.652400098668295e-06], device="cuda")  # lambda lies half a step of fp32 off
    h0 = 1 + torch.rand(1, 1, dk, dv, generator=torch.Generator().manual_seed(6)).cuda()
    k, v, state = torch.zeros(1, 1, dk, device="cuda"), torch.zeros(1, 1, dv, device="cuda"), h0.clone()
    for _ in range(n):
        pkg.gla_decay_step(k, k, v, ld, state)
    assert bool((carried(state[0], h0[0], ld, n) <= mean_bound(n, dk * dv)).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_slow_head_decays_right_across_segments(dtype):
    """32 segments of 128 tokens: a start state passes 30 joins and at most four chunks."""
    T, n, dk, dv = 4096, 8, 128, 256
    ld = torch.tensor(SLOW, device="cuda")
    h0 = 1 + torch.rand(n, 2, dk, dv, generator=torch.Generator().manual_seed(7)).cuda()
    k, v = torch.zeros(n, 2, T, dk, dtype=dtype, device="cuda"), torch.zeros(n, 2, T, dv, dtype=dtype, device="cuda")
    _, hT = pkg.gla_decay_fwd(k, k, v, ld, h0=h0, segments=32)
    off = carried(hT.transpose(0, 1), h0.transpose(0, 1), ld, T)
    assert bool((off <= mean_bound(34, n * dk * dv)).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_entries_of_a_pool_that_is_not_given_are_not_reported(dtype):
    """slots0 and slots1 count the entries of pools that are given; without one they mean nothing."""
    from chunkwise_linear_rnn_fwd_b200 import gla as G
    b = Batch([20], 2, 64, 64, dtype, seed=8)
    x, ld = views(b, ("q", "k", "v"), "heads"), b.ld.cuda()
    o, ws = torch.empty_like(x["v"]), pkg.alloc_decay_workspace(1 << 20, "cuda")
    d = G._decay_desc(1, 2, 20, 0, 64, 64, dtype, -7, -7, 0, ws, 0)
    shape = x["q"].shape
    keep, p = G._views(dtype, 0, *((t, "", shape) for t in (x["q"], x["k"], x["v"], o)))
    r = pkg.load().gla_decay_fwd(ctypes.byref(d), p, p + 32, p + 64, ld.data_ptr(), None, None, None, p + 96, None, None,
                                 torch.cuda.current_stream().cuda_stream)
    assert r == 0 and pkg.poll_status(ws) == 0
    assert torch.equal(o, pkg.gla_decay_fwd(x["q"], x["k"], x["v"], ld)[0])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_batch_of_empty_sequences_passes_its_states_on(dtype):
    """The longest of no tokens at all is zero."""
    q = torch.full((1, 2, 6, 64), float("nan"), dtype=dtype, device="cuda")
    ld, cu = torch.full((2,), -0.5, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    h = torch.randn(3, 2, 64, 64, generator=torch.Generator().manual_seed(9)).cuda()
    ws = pkg.alloc_decay_workspace(1 << 20, "cuda")
    kw = {"cu_seqlens": cu, "max_len": 0, "workspace": ws}
    o, hT = pkg.gla_decay_fwd(q, q, q, ld, h0=h, **kw)
    *g, dh0 = pkg.gla_decay_bwd(q, q, q, ld, q, h0=h, dh_final=h, **kw)
    assert torch.equal(hT, h) and torch.equal(dh0, h) and pkg.poll_status(ws) == 0
    assert not any(bool(t.any()) for t in (o, *g))
