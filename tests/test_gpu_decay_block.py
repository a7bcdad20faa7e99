"""A linear-attention block put together from the library's calls, as a model would use
them: layer norm, projections, decay attention, the gated output epilogue; prompts and then
single tokens over a pool of states, and a training step's gradients by the chain of backward
calls, all against the same block in float64."""
import pytest
import torch

import chunkwise_linear_rnn_fwd_b200 as pkg

pytestmark = pytest.mark.gpu

H, DK, DV, D = 2, 64, 96, 128
# Six stages (norm, projection, attention, norm, gate, projection), each a chain of at most
# 300 fp32 additions rounded by 2^-24: 6 * 300 * 2^-24 = 1.1e-4 of the terms' sizes.
TOL = 1.1e-4


def weights(seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, scale: torch.randn(*s, generator=g) * scale  # noqa: E731
    return {"nw": 1 + r(D, scale=0.1), "nb": r(D, scale=0.1), "wq": r(D, H * DK, scale=D ** -0.5),
            "wk": r(D, H * DK, scale=D ** -0.5 * DK ** -0.5), "wv": r(D, H * DV, scale=D ** -0.5),
            "wr": r(D, H * DV, scale=D ** -0.5), "ow": 1 + r(DV, scale=0.1), "ob": r(DV, scale=0.1),
            "wo": r(H * DV, D, scale=(H * DV) ** -0.5)}


LD = torch.tensor([-0.3, -0.004])


def plain(x, p, s0):
    """One sequence x [T,D] in float64: (y [T,D], last state)."""
    n = torch.nn.functional.layer_norm(x, (D,), p["nw"], p["nb"], 1e-5)
    q, k, v, r = ((n @ p[m]).view(len(x), H, -1) for m in ("wq", "wk", "wv", "wr"))
    lam, S, outs = torch.exp(LD.double()).view(H, 1, 1), s0, []
    for t in range(len(x)):
        S = lam * S + k[t, :, :, None] * v[t, :, None, :]
        outs.append((q[t, :, None, :] @ S)[:, 0])
    o = torch.nn.functional.layer_norm(torch.stack(outs), (DV,), p["ow"], p["ob"], 1e-5) * r * torch.sigmoid(r)
    return x + o.reshape(len(x), H * DV) @ p["wo"], S


def close(a, b, tol=TOL):
    a, b = a.double().cpu(), b.double().cpu()
    off = float((a - b).norm() / b.norm())
    assert off <= tol, off


def test_prompts_then_tokens():
    p64 = {n: w.double() for n, w in weights().items()}
    p = {n: w.cuda() for n, w in weights().items()}
    lens, more, slots = [150, 1, 37], 4, [4, 0, 2]
    g = torch.Generator().manual_seed(1)
    xs = [torch.randn(n + more, D, generator=g) for n in lens]
    want = [plain(x.double(), p64, torch.zeros(H, DK, DV, dtype=torch.float64)) for x in xs]
    cu = torch.tensor([0, 150, 151, 188], dtype=torch.int32, device="cuda")
    index = torch.tensor(slots, dtype=torch.int32, device="cuda")
    pool = torch.zeros(5, H, DK, DV, device="cuda")
    ld = LD.cuda()
    proj = torch.cat([p["wq"].view(D, H, DK), p["wk"].view(D, H, DK), p["wv"].view(D, H, DV), p["wr"].view(D, H, DV)], 2)
    proj = proj.flatten(1)

    def front(x):  # one fused projection; q, k, v are views of its rows
        n, _, _ = pkg.gla_layernorm_fwd(x, p["nw"], p["nb"], want_stats=False)
        return (n @ proj).view(len(x), H, -1).split([DK, DK, DV, DV], 2)

    def back(x, o, r):  # [N,H,DV]
        o, r = o[None, None].reshape(1, 1, -1, DV).contiguous(), r.reshape(1, 1, -1, DV).contiguous()
        y = pkg.gla_epilogue_fwd(o, r, p["ow"], p["ob"])
        return x + y.view(len(x), H * DV) @ p["wo"]

    x = torch.cat([x[:n] for x, n in zip(xs, lens)]).cuda()
    q, k, v, r = front(x)
    o, _ = pkg.gla_decay_fwd(*(t.transpose(0, 1)[None] for t in (q, k, v)), ld, cu_seqlens=cu, max_len=150,
                             h_final=pool, h_final_index=index)
    y = back(x, o[0].transpose(0, 1).contiguous(), r).split(lens)
    for a, (b, _), n in zip(y, want, lens):
        close(a, b[:n])
    for t in range(more):
        x = torch.stack([x[n + t] for x, n in zip(xs, lens)]).cuda()
        q, k, v, r = front(x)
        y = back(x, pkg.gla_decay_step(q, k, v, ld, pool, index), r)
        for i, n in enumerate(lens):
            close(y[i], want[i][0][n + t])
    for s, (_, S) in zip(slots, want):
        close(pool[s], S)


def test_training_step_gradients():
    lens = [70, 200]
    T = sum(lens)
    g = torch.Generator().manual_seed(2)
    x, up = torch.randn(T, D, generator=g), torch.randn(T, D, generator=g)
    p64 = {n: w.double().requires_grad_() for n, w in weights().items()}
    x64 = x.double().requires_grad_()
    ys = [plain(s, p64, torch.zeros(H, DK, DV, dtype=torch.float64))[0] for s in x64.split(lens)]
    (torch.cat(ys) * up.double()).sum().backward()

    p, x, up, ld = {n: w.cuda() for n, w in weights().items()}, x.cuda(), up.cuda(), LD.cuda()
    cu = {"cu_seqlens": torch.tensor([0, 70, 270], dtype=torch.int32, device="cuda"), "max_len": 200}
    heads = lambda t: t.view(T, H, -1).transpose(0, 1)[None]  # noqa: E731
    rows = lambda t: t[0].transpose(0, 1).reshape(T, -1)  # noqa: E731
    n, mean, rstd = pkg.gla_layernorm_fwd(x, p["nw"], p["nb"])
    q, k, v = (heads(n @ p[m]) for m in ("wq", "wk", "wv"))
    r = heads(n @ p["wr"]).contiguous()
    o, _ = pkg.gla_decay_fwd(q, k, v, ld, want_final=False, **cu)
    a = pkg.gla_epilogue_fwd(o.contiguous(), r, p["ow"], p["ob"])
    close(x + rows(a) @ p["wo"], torch.cat(ys).detach())

    grads = {"wo": rows(a).t() @ up}
    do, dr, grads["ow"], grads["ob"] = pkg.gla_epilogue_bwd(o, r, heads(up @ p["wo"].t()).contiguous(), p["ow"], p["ob"])
    dq, dk, dv, _ = pkg.gla_decay_bwd(q, k, v, ld, do, want_dh0=False, **cu)
    dn = torch.zeros_like(n)
    for m, d in (("wq", dq), ("wk", dk), ("wv", dv), ("wr", dr)):
        grads[m] = n.t() @ rows(d)
        dn += rows(d) @ p[m].t()
    dx, grads["nw"], grads["nb"] = pkg.gla_layernorm_bwd(x, dn, mean, rstd, p["nw"])
    close(dx + up, x64.grad, 2 * TOL)  # the backward's six stages behind the forward's
    for m, w in p64.items():
        close(grads[m], w.grad, 2 * TOL)
