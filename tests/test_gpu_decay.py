"""Decay attention on the GPU against the float64 recurrence: the chunked pass and its
gradients over dense and packed batches, the recurrent step, pools of states, and what a
batch may hold besides (empty sequences, rows of nobody, bad bounds and indexes)."""
import numpy as np
import pytest
import torch

import chunkwise_linear_rnn_fwd_b200 as pkg
from oracle import decay as oracle
from tests.decay_cases import Batch, check, packing, reference, rows, views

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
OK, INDEX, GATE = 0, -9, -7


def on_tc(b):
    return b.dtype == BF16 and b.dk % 8 == 0 and b.dv % 8 == 0


def run_fwd(b, layout, with_h0=True, segments=0):
    x = views(b, ("q", "k", "v"), layout)
    ws = pkg.alloc_decay_workspace(1 << 26, "cuda")
    o, hT = pkg.gla_decay_fwd(x["q"], x["k"], x["v"], b.ld.cuda(), h0=b.h0.cuda() if with_h0 else None,
                              segments=segments, workspace=ws, **packing(b, layout))
    assert pkg.poll_status(ws) == OK
    return {"o": rows(o), "h_final": hT}


SIZES = [(64, 64), (128, 128), (128, 256), (256, 512), (256, 64), (40, 24), (96, 200), (8, 8), (33, 17), (1, 1), (200, 5)]
LENS = {"one": [1], "chunk": [128], "ragged": [129, 0, 1, 127, 255], "long": [1100]}


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("lens", LENS)
def test_fwd(dtype, dk, dv, lens):
    b = Batch(LENS[lens], 3 if lens != "long" else 2, dk, dv, dtype, seed=dk + dv)
    layout = {"one": "heads", "chunk": "dense", "ragged": "fused", "long": "tokens"}[lens]
    check(run_fwd(b, layout), reference(b), b, on_tc(b))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("segments", [1, 2, 5, 32])
def test_fwd_segments(dtype, segments):
    """Any split of the sequences gives the same function, shorter sequences included."""
    b = Batch([1300, 70, 0, 640], 2, 64, 72, dtype, seed=segments)
    check(run_fwd(b, "tokens", segments=segments), reference(b), b, on_tc(b))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["dense", "dense_tokens"])
def test_dense_layouts_without_start_states(dtype, layout):
    b = Batch([190, 190, 190], 2, 64, 64, dtype, seed=3)
    check(run_fwd(b, layout, with_h0=False), reference(b, with_h0=False), b, on_tc(b))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", [0.0, -1e-4, -1.0, -60.0, -np.inf])
def test_decays_from_none_to_everything(dtype, kind):
    """No decay rescales anything: also one that leaves nothing of the token before."""
    b = Batch([300, 2], 1, 64, 64, dtype, seed=5, kind=kind)
    check(run_fwd(b, "tokens", segments=2), reference(b), b, on_tc(b))
    x = views(b, ("q", "k", "v", "do"), "tokens")
    dq, dk, dv, dh0 = pkg.gla_decay_bwd(x["q"], x["k"], x["v"], b.ld.cuda(), x["do"], h0=b.h0.cuda(),
                                        dh_final=b.dh.cuda(), segments=2, **packing(b, "tokens"))
    check({"dq": rows(dq), "dk": rows(dk), "dv": rows(dv), "dh0": dh0}, reference(b, bwd=True), b, on_tc(b))


def test_a_decay_above_one_is_reported():
    b = Batch([40], 3, 64, 64, BF16, seed=6)
    ld = b.ld.clone()
    x = views(b, ("q", "k", "v"), "tokens")
    ws = pkg.alloc_decay_workspace(1 << 20, "cuda")
    for bad in (0.5, float("nan")):
        ld[1] = bad
        o, _ = pkg.gla_decay_fwd(x["q"], x["k"], x["v"], ld.cuda(), workspace=ws, **packing(b, "tokens"))
        assert pkg.poll_status(ws) == GATE
        b.ld = torch.where(torch.arange(3) == 1, 0.0, ld)  # taken as no decay
        check({"o": rows(o)}, reference(b, with_h0=False), b, True)
    assert pkg.poll_status(ws) == OK


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 256), (256, 320), (96, 200), (33, 17), (16, 520)])
@pytest.mark.parametrize("lens", ["one", "ragged", "long"])
def test_bwd(dtype, dk, dv, lens):
    b = Batch(LENS[lens], 2, dk, dv, dtype, seed=dk * dv)
    layout = {"one": "heads", "ragged": "fused", "long": "tokens"}[lens]
    x = views(b, ("q", "k", "v", "do"), layout)
    p = packing(b, layout)
    ws = pkg.alloc_decay_workspace(pkg.decay_workspace_size(len(b.lens), b.H, b.rows, dk, dv, dtype, True,
                                                            max_len=p["max_len"]), "cuda")
    dq, dk_, dv_, dh0 = pkg.gla_decay_bwd(x["q"], x["k"], x["v"], b.ld.cuda(), x["do"], h0=b.h0.cuda(),
                                          dh_final=b.dh.cuda(), workspace=ws, **p)
    assert pkg.poll_status(ws) == OK
    check({"dq": rows(dq), "dk": rows(dk_), "dv": rows(dv_), "dh0": dh0}, reference(b, bwd=True), b, on_tc(b))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bwd_dense_without_states(dtype):
    b = Batch([257, 257], 2, 64, 96, dtype, seed=8)
    x = views(b, ("q", "k", "v", "do"), "dense")
    dq, dk, dv, dh0 = pkg.gla_decay_bwd(x["q"], x["k"], x["v"], b.ld.cuda(), x["do"], want_dh0=False)
    assert dh0 is None
    want = reference(b, with_h0=False, bwd=True, with_dh=False)
    check({"dq": rows(dq), "dk": rows(dk), "dv": rows(dv)}, want, b, on_tc(b))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("what", ["heads", "sequences", "tokens"])
def test_inputs_shared_by_heads_sequences_or_tokens(dtype, packed, what):
    """An expanded input (distance zero) is the input written out, and each of those that
    share it gets its own gradient."""
    if packed and what == "sequences":
        pytest.skip("packed sequences share no rows")
    n, H, T = 2, 3, 150
    b = Batch([T] * n, H, 64, 72, dtype, seed=21)
    for name in ("k", "v"):
        x = getattr(b, name).view(n, T, H, -1)
        x = {"heads": x[:, :, :1], "sequences": x[:1], "tokens": x[:, :1]}[what]
        setattr(b, name, x.expand(n, T, H, -1).reshape(n * T, H, -1))
    x = views(b, ("q", "k", "v", "do"), "tokens" if packed else "dense_tokens")
    axis = {"heads": 1, "sequences": 0, "tokens": 2}[what]
    if packed and what == "tokens":  # one row for the tokens of both sequences
        b.k[:], b.v[:] = b.k[:1].clone(), b.v[:1].clone()
    for name in ("k", "v"):
        x[name] = (views(b, (name,), "tokens" if packed else "dense_tokens")[name].narrow(axis, 0, 1).expand(x[name].shape))
        assert x[name].stride(axis) == 0
    p = packing(b, "tokens" if packed else "dense")
    o, hT = pkg.gla_decay_fwd(x["q"], x["k"], x["v"], b.ld.cuda(), h0=b.h0.cuda(), **p)
    dq, dk, dv, dh0 = pkg.gla_decay_bwd(x["q"], x["k"], x["v"], b.ld.cuda(), x["do"], h0=b.h0.cuda(),
                                        dh_final=b.dh.cuda(), **p)
    on = on_tc(b) and what != "tokens"
    check({"o": rows(o), "h_final": hT}, reference(b), b, on)
    check({"dq": rows(dq), "dk": rows(dk), "dv": rows(dv), "dh0": dh0}, reference(b, bwd=True), b, on)


@pytest.mark.parametrize("segments", [1, 4])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_nobody(dtype, segments):
    """Rows outside the sequences, and other sequences, hold infinities and NaN: none of it
    arrives, and the rows behind the last sequence keep what was in the output."""
    b = Batch([130, 600, 3], 2, 64, 64, dtype, seed=9, spare=70)
    x = views(b, ("q", "k", "v", "do"), "tokens")
    ld, cu = b.ld.cuda(), torch.tensor(b.cu, dtype=torch.int32, device="cuda")
    for poisoned in (0, 2):
        bad = {n: t.clone(memory_format=torch.preserve_format) for n, t in x.items()}
        for n, t in bad.items():
            t[0, :, b.cu[poisoned]:b.cu[poisoned + 1]] = float("nan")
            t[0, :, b.cu[-1]:] = float("inf")
        o = torch.full((b.rows, b.H, b.dv), 7.0, dtype=dtype, device="cuda").transpose(0, 1)[None]
        _, hT = pkg.gla_decay_fwd(bad["q"], bad["k"], bad["v"], ld, cu_seqlens=cu, max_len=600, h0=b.h0.cuda(), o=o,
                                  segments=segments)
        g = pkg.gla_decay_bwd(bad["q"], bad["k"], bad["v"], ld, bad["do"], cu_seqlens=cu, max_len=600,
                              h0=b.h0.cuda(), dh_final=b.dh.cuda(), segments=segments,
                              **{n: torch.full_like(x[m], 7.0) for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"))})
        for y in (o, *g[:3]):
            assert bool((y[0, :, b.cu[-1]:] == 7.0).all())
        want, wantb = reference(b), reference(b, bwd=True)
        keep = [i for i in range(3) if i != poisoned]
        s = Batch([b.lens[i] for i in keep], b.H, b.dk, b.dv, dtype)
        take = torch.cat([torch.arange(b.cu[i], b.cu[i + 1]) for i in keep]).cuda()
        check({"o": rows(o)[take], "h_final": hT[keep]}, [want[i] for i in keep], s, on_tc(b))
        check({"dq": rows(g[0])[take], "dk": rows(g[1])[take], "dv": rows(g[2])[take], "dh0": g[3][keep]},
              [wantb[i] for i in keep], s, on_tc(b))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("segments", [1, 3])
def test_pool_in_place(dtype, segments):
    """States are read from and written to the named entries of one pool, a new request
    starts from zero, one without an entry leaves none, and the other entries stay."""
    b = Batch([500, 130, 0, 260], 2, 64, 48, dtype, seed=11)
    x = views(b, ("q", "k", "v"), "fused")
    pool = torch.randn(7, 2, 64, 48, generator=torch.Generator().manual_seed(1)).cuda()
    before = pool.clone()
    read, write = [5, -1, 2, 6], [5, 3, 2, -1]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = pkg.alloc_decay_workspace(1 << 26, "cuda")
    o, out = pkg.gla_decay_fwd(x["q"], x["k"], x["v"], b.ld.cuda(), h0=pool, h0_index=i32(read), h_final=pool,
                               h_final_index=i32(write), segments=segments, workspace=ws, **packing(b, "fused"))
    assert out is pool and pkg.poll_status(ws) == OK
    b.h0 = torch.stack([before[r].cpu() if r >= 0 else torch.zeros_like(before[0]).cpu() for r in read])
    want = reference(b)
    check({"o": rows(o)}, want, b, on_tc(b))
    for i, w in enumerate(write):
        if w >= 0:
            check({"h_final": pool[w:w + 1]}, [want[i]], Batch([b.lens[i]], 2, 64, 48, dtype), on_tc(b))
    for e in (0, 1, 4, 6):
        assert torch.equal(pool[e], before[e])
    assert torch.equal(pool[2], before[2])  # an empty sequence passes its state on


@pytest.mark.parametrize("offset", [4, 8])
def test_pools_aligned_to_16_or_32_bytes(offset):
    """States are moved 32 bytes at a time where their address allows, 16 elsewhere."""
    b = Batch([200, 31], 2, 64, 72, BF16, seed=71)
    x = views(b, ("q", "k", "v"), "tokens")
    h0, hT = (torch.full((b.h0.numel() + 64,), 7.0, device="cuda") for _ in range(2))
    h0v, hTv = (t[offset:offset + b.h0.numel()].view(b.h0.shape) for t in (h0, hT))
    assert h0v.data_ptr() % 32 == (4 * offset) % 32
    h0v.copy_(b.h0)
    o, _ = pkg.gla_decay_fwd(x["q"], x["k"], x["v"], b.ld.cuda(), h0=h0v, h_final=hTv, **packing(b, "tokens"))
    check({"o": rows(o), "h_final": hTv}, reference(b), b, True)
    assert torch.all(hT[:offset] == 7) and torch.all(hT[offset + b.h0.numel():] == 7)


def test_pool_conflicts_are_reported():
    """One entry named twice, another sequence's entry read, an entry past the pool."""
    b = Batch([150, 40, 20], 1, 64, 64, BF16, seed=12)
    x = views(b, ("q", "k", "v"), "tokens")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = pkg.alloc_decay_workspace(1 << 22, "cuda")
    start = torch.randn(4, 1, 64, 64, generator=torch.Generator().manual_seed(2))
    for read, write, begins, ends in (([-1, -1, -1], [1, 1, 2], [-1, -1, -1], [1, -1, 2]),
                                      ([0, 1, 2], [1, 0, 2], [-1, -1, 2], [1, 0, 2]),
                                      ([0, 9, 1], [0, 1, 7], [0, -1, -1], [0, 1, -1])):
        pool = start.clone().cuda()
        o, _ = pkg.gla_decay_fwd(x["q"], x["k"], x["v"], b.ld.cuda(), h0=pool, h0_index=i32(read), h_final=pool,
                                 h_final_index=i32(write), workspace=ws, **packing(b, "tokens"))
        assert pkg.poll_status(ws) == INDEX and pkg.poll_status(ws) == OK
        b.h0 = torch.stack([start[r] if r >= 0 else torch.zeros_like(start[0]) for r in begins])
        want = reference(b)
        check({"o": rows(o)}, want, b, True)
        for i, e in enumerate(ends):
            if e >= 0:
                check({"h_final": pool[e:e + 1]}, [want[i]], Batch([b.lens[i]], 1, 64, 64, BF16), True)
        for e in set(range(4)) - set(ends):
            assert torch.equal(pool[e].cpu(), start[e])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bad_bounds_are_reported(dtype):
    """Bounds outside the rows, decreasing ones and a sequence longer than max_len: such a
    sequence is treated as empty, the others are computed."""
    b = Batch([60, 60, 60], 2, 64, 64, dtype, seed=13)
    x = views(b, ("q", "k", "v"), "tokens")
    ws = pkg.alloc_decay_workspace(1 << 22, "cuda")
    want = reference(b, with_h0=False)
    for cu, max_len, good in (([0, 60, 120, 181], 70, (0, 1)), ([-60, 0, 60, 120], 60, (0, 1)), ([0, 60, 0, 180], 60, (0,)),
                              ([0, 60, 180, 180], 60, (0,))):
        o = torch.zeros(180, 2, 64, dtype=dtype, device="cuda").transpose(0, 1)[None]
        pkg.gla_decay_fwd(x["q"], x["k"], x["v"], b.ld.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                          max_len=max_len, o=o, workspace=ws)
        assert pkg.poll_status(ws) == INDEX
        s = Batch([60] * len(good), 2, 64, 64, dtype)
        take = torch.cat([torch.arange(60 * i, 60 * i + 60) for i in good] or [torch.arange(0)]).cuda()
        check({"o": rows(o)[take]}, [want[i] for i in good], s, on_tc(b))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 64, 64), (3, 4, 128, 256), (5, 2, 256, 512), (2, 3, 33, 17), (4, 1, 1, 1),
                                       (9, 2, 40, 100), (1, 2, 8, 4)])
def test_step(dtype, B, H, dk, dv):
    b = Batch([1] * B, H, dk, dv, dtype, seed=B + dv)
    x = torch.cat([b.q, b.k, b.v], -1).cuda()
    q, k, v = x.split([dk, dk, dv], -1)
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(B))[:B]
    pool = torch.randn(B + 3, H, dk, dv, generator=torch.Generator().manual_seed(1))
    b.h0 = pool[slots]
    state = pool.cuda()
    ws = pkg.alloc_decay_workspace(256, "cuda")
    o = pkg.gla_decay_step(q, k, v, b.ld.cuda(), state, slots.int().cuda(), workspace=ws)
    assert pkg.poll_status(ws) == OK
    check({"o": o, "h_final": state[slots.cuda()]}, reference(b), b, False)
    rest = [e for e in range(B + 3) if e not in slots.tolist()]
    assert torch.equal(state[rest].cpu(), pool[rest])
    dense = b.h0.cuda()
    assert torch.equal(pkg.gla_decay_step(q, k, v, b.ld.cuda(), dense), o)
    assert torch.equal(dense, state[slots.cuda()])


def test_step_padding_and_conflicts():
    B, H, d = 6, 2, 64
    b = Batch([1] * B, H, d, d, BF16, seed=21)
    for n in ("q", "k", "v"):
        getattr(b, n)[2] = float("nan")  # a padding row's tokens are not read
    pool = torch.randn(4, H, d, d, generator=torch.Generator().manual_seed(3))
    state, o = pool.cuda(), torch.full((B, H, d), 7.0, dtype=BF16, device="cuda")
    index = torch.tensor([3, 0, -1, 3, 4, 1], dtype=torch.int32, device="cuda")
    ws = pkg.alloc_decay_workspace(256, "cuda")
    pkg.gla_decay_step(b.q.cuda(), b.k.cuda(), b.v.cuda(), b.ld.cuda(), state, index, o=o, workspace=ws)
    assert pkg.poll_status(ws) == INDEX
    for i in (2, 3, 4):
        assert bool((o[i] == 7.0).all())
    live, entry = [0, 1, 5], [3, 0, 1]
    for i, e in zip(live, entry):
        ro, rS = oracle.fwd(b.seq("q", i), b.seq("k", i), b.seq("v", i), b.ld.double().numpy(), pool[e].double().numpy())
        assert np.abs(o[i].double().cpu().numpy() - ro[:, 0]).max() <= 2.0 ** -7 * np.abs(ro).max()
        assert np.abs(state[e].double().cpu().numpy() - rS).max() <= 2.0 ** -21 * np.abs(rS).max()
    assert torch.equal(state[2].cpu(), pool[2])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_then_steps(dtype):
    """A prompt into the pool, then single tokens from it, is one longer sequence."""
    n, more = 200, 5
    b = Batch([n + more] * 2, 2, 64, 64, dtype, seed=31)
    x = {m: getattr(b, m).view(2, n + more, 2, 64).transpose(1, 2).cuda() for m in ("q", "k", "v")}
    ld, pool = b.ld.cuda(), torch.zeros(3, 2, 64, 64, device="cuda")
    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    o, _ = pkg.gla_decay_fwd(*(x[m][:, :, :n] for m in ("q", "k", "v")), ld, h_final=pool, h_final_index=slots)
    outs = [pkg.gla_decay_step(*(x[m][:, :, t] for m in ("q", "k", "v")), ld, pool, slots) for t in range(n, n + more)]
    y = torch.cat([o, torch.stack(outs, 2)], 2)
    check({"o": rows(y), "h_final": pool[slots.long()]}, reference(b, with_h0=False), b, on_tc(b))
    assert not bool(pool[1].any())


def test_two_calls_give_the_same_bits():
    b = Batch([700, 90], 2, 128, 128, BF16, seed=41)
    x = views(b, ("q", "k", "v", "do"), "tokens")
    kw = dict(h0=b.h0.cuda(), segments=3, **packing(b, "tokens"))
    one, two = ([*pkg.gla_decay_fwd(x["q"], x["k"], x["v"], b.ld.cuda(), **kw),
                 *pkg.gla_decay_bwd(x["q"], x["k"], x["v"], b.ld.cuda(), x["do"], **kw)] for _ in range(2))
    for s, t in zip(one, two):
        assert torch.equal(s, t)


def test_streams_and_graphs():
    """On another stream, and captured into a graph that is replayed with other inputs."""
    b = Batch([300, 50], 2, 64, 64, BF16, seed=51)
    c = Batch([300, 50], 2, 64, 64, BF16, seed=52)
    x = views(b, ("q", "k", "v"), "tokens")
    ld, p, h0 = b.ld.cuda(), packing(b, "tokens"), b.h0.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, hT = pkg.gla_decay_fwd(x["q"], x["k"], x["v"], ld, h0=h0, stream=s, **p)
    torch.cuda.current_stream().wait_stream(s)
    check({"o": rows(o), "h_final": hT}, reference(b), b, True)
    ws = pkg.alloc_decay_workspace(1 << 22, "cuda")
    tok = [t[0, :, 0].unsqueeze(0).clone() for t in x.values()]
    state = h0.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        o, hT = pkg.gla_decay_fwd(x["q"], x["k"], x["v"], ld, h0=h0, workspace=ws, **p)
        os = pkg.gla_decay_step(*tok, ld, state[:1], workspace=ws)
    y = views(c, ("q", "k", "v"), "tokens")
    for n in x:
        x[n].copy_(y[n])
    h0.copy_(c.h0)
    for t, n in zip(tok, x):
        t.copy_(x[n][0, :, 0])
    state.copy_(h0)
    g.replay()
    check({"o": rows(o), "h_final": hT}, reference(c), c, True)
    assert pkg.poll_status(ws) == OK
    f = Batch([1], 2, 64, 64, BF16)
    f.q, f.k, f.v, f.ld, f.h0 = c.q[:1], c.k[:1], c.v[:1], c.ld, c.h0[:1]
    check({"o": os, "h_final": state[:1]}, reference(f), f, False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("segments", [0, 3])
@pytest.mark.parametrize("graph", [False, True])
def test_what_follows_finds_the_call_complete(dtype, segments, graph):
    """Walks of a call start before the kernel ahead of them ends; what the stream does next
    (outputs copied, inputs, states and workspace overwritten) still comes after all of them."""
    b = Batch([900, 40, 513], 3, 64, 128, dtype, seed=61)
    x = views(b, ("q", "k", "v", "do"), "tokens")
    ld, p, h0, dh = b.ld.cuda(), packing(b, "tokens"), b.h0.cuda(), b.dh.cuda()
    keep = {n: t.clone() for n, t in x.items()}
    ws = pkg.alloc_decay_workspace(pkg.decay_workspace_size(3, 3, b.rows, 64, 128, dtype, True, max_len=p["max_len"],
                                                            segments=segments), "cuda")

    def run():
        for n in x:
            x[n].copy_(keep[n])
        out = []
        for _ in range(2):
            o, hT = pkg.gla_decay_fwd(x["q"], x["k"], x["v"], ld, h0=h0, segments=segments, workspace=ws, **p)
            g = pkg.gla_decay_bwd(x["q"], x["k"], x["v"], ld, x["do"], h0=h0, dh_final=dh, segments=segments,
                                  workspace=ws, **p)
            out.append([t.clone() for t in (o, hT, *g)])
            ws[256:].fill_(255)
        for t in x.values():
            t.fill_(float("nan"))
        return out

    if graph:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        for _ in range(3):
            g.replay()
    else:
        out = run()
    want, wantg = reference(b), reference(b, bwd=True)
    for o, hT, dq, dk, dv, dh0 in out:
        check({"o": rows(o), "h_final": hT}, want, b, on_tc(b))
        check({"dq": rows(dq), "dk": rows(dk), "dv": rows(dv), "dh0": dh0}, wantg, b, on_tc(b))
    assert pkg.poll_status(ws) == OK


def test_offsets_past_32_bits():
    """A pool and rows whose far end lies more than 2^31 elements from the start."""
    H, d = 1, 64
    slots = (1 << 31) // (d * d) + 3
    pool = torch.zeros(slots, H, d, d, device="cuda")
    b = Batch([130], H, d, d, BF16, seed=61)
    big = torch.zeros((1 << 31) // 512 + 400, 512, dtype=BF16, device="cuda")
    at = big.shape[0] - 200
    q, k, v = (big[:, i * d:(i + 1) * d].unsqueeze(0).unsqueeze(0) for i in range(3))
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        t[0, 0, at:at + 130] = getattr(b, n)[:, 0].cuda()
    cu = torch.tensor([at, at + 130], dtype=torch.int32, device="cuda")
    slot = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    pool[slots - 1] = b.h0[0].cuda()
    o = big[:, 3 * d:4 * d].unsqueeze(0).unsqueeze(0)
    pkg.gla_decay_fwd(q, k, v, b.ld.cuda(), cu_seqlens=cu, max_len=130, h0=pool, h0_index=slot, h_final=pool,
                      h_final_index=slot, o=o)
    want = reference(b)
    check({"o": o[0, 0, at:at + 130].unsqueeze(1), "h_final": pool[slots - 1:]}, want, b, True)
    tok = (x[0, :, at:at + 1].transpose(0, 1) for x in (q, k, v))
    pool[slots - 1] = b.h0[0].cuda()
    y = pkg.gla_decay_step(*tok, b.ld.cuda(), pool, slot)
    f = Batch([1], H, d, d, BF16)
    f.q, f.k, f.v, f.ld, f.h0 = b.q[:1], b.k[:1], b.v[:1], b.ld, b.h0
    check({"o": y, "h_final": pool[slots - 1:]}, reference(f), f, False)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_against_differences(dtype):
    """The gradients of the loss sum(o do) + sum(S_T dS) along random directions against
    central differences of the GPU's own forward in fp32 (the loss is linear in each input,
    so a difference is off by the forward's rounding alone)."""
    b = Batch([150, 40], 2, 32, 40, F32, seed=71)
    x = {n: t for n, t in views(b, ("q", "k", "v", "do"), "tokens").items()}
    p, ld, h0, dh = packing(b, "tokens"), b.ld.cuda(), b.h0.cuda(), b.dh.cuda()

    def loss(q, k, v, h):
        o, hT = pkg.gla_decay_fwd(q, k, v, ld, h0=h, **p)
        return float((o.double() * x["do"].double()).sum() + (hT.double() * dh.double()).sum())

    y = {n: t.to(dtype) for n, t in x.items()}
    g = pkg.gla_decay_bwd(y["q"], y["k"], y["v"], ld, y["do"], h0=h0, dh_final=dh, **p)
    args = [x["q"], x["k"], x["v"], h0]
    for i, grad in enumerate(g):
        u = torch.randn(args[i].shape, generator=torch.Generator("cuda").manual_seed(i), device="cuda")
        hi, lo = (loss(*(a + s * u if j == i else a for j, a in enumerate(args))) for s in (1.0, -1.0))
        along = float((grad.double() * u.double()).sum())
        size = float(grad.double().norm() * u.double().norm())
        # inputs, products and outputs rounded to bf16: five roundings of 2^-8; in fp32 the
        # two losses' own rounding, of at most 2^-23 * 400 of sums as large as `size`
        allowed = (5 * 2.0 ** -8 if dtype == BF16 else 400 * 2.0 ** -23) * size
        assert abs((hi - lo) / 2 - along) <= allowed, (i, (hi - lo) / 2, along, size)
