"""Measured cases of the decay-attention and layer-norm operators.

Five operators of a linear-attention block whose heads forget at a constant rate:

  prompt  the chunked pass over a batch of prompts packed row after row, reading and
          writing states in a pool (gla_decay_fwd)
  step    one recurrent token for each running request, states in a pool (gla_decay_step)
  grad    the gradients of the chunked pass, for training (gla_decay_bwd)
  norm    the layer norm in front of the block (gla_layernorm_fwd)
  dnorm   its gradients, with the sums over rows for weight and bias (gla_layernorm_bwd)

With lambda_h = exp(log_decay_h), per sequence and head:
  S_t = lambda_h S_{t-1} + k_t^T v_t ,   o_t = q_t S_t .
"""
import math
import random

import torch

own = False  # False: the operators in their plain form; True: the framework's calls

CHUNK = 128  # tokens of a chunk of the plain form
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a single short request joins: launch latency
        {"name": "prompt one short", "op": "prompt", "dtype": "bf16", "nseq": 1, "lo": 100, "hi": 100, "empty": 0,
         "spare": 0, "H": 4, "dk": 64, "dv": 64},
        # a scheduler's batch: many prompts of very different lengths, one of them empty, rows padded to a bucket
        {"name": "prompt ragged batch", "op": "prompt", "dtype": "bf16", "nseq": 24, "lo": 1, "hi": 2048, "empty": 1,
         "spare": 201, "H": 16, "dk": 128, "dv": 128},
        # two long documents at the widest heads (32768 tokens, 4 heads of 256 x 512)
        {"name": "prompt long", "op": "prompt", "dtype": "bf16", "nseq": 2, "lo": 16384, "hi": 16384, "empty": 0,
         "spare": 0, "H": 4, "dk": 256, "dv": 512},
        # a model kept in 32 bits
        {"name": "prompt fp32", "op": "prompt", "dtype": "fp32", "nseq": 3, "lo": 33, "hi": 700, "empty": 0,
         "spare": 7, "H": 4, "dk": 64, "dv": 64},
        # one user's chat: a single token
        {"name": "step one", "op": "step", "dtype": "bf16", "B": 1, "slots": 4, "H": 4, "dk": 128, "dv": 256},
        # a full serving batch, some of its rows padding, out of a larger pool
        {"name": "step batch", "op": "step", "dtype": "bf16", "B": 256, "slots": 300, "H": 16, "dk": 128, "dv": 128},
        # a training layer: batch 8, 2048 tokens, 4 heads of 128 x 256
        {"name": "grad layer", "op": "grad", "dtype": "bf16", "nseq": 8, "lo": 2048, "hi": 2048, "empty": 0,
         "dense": True, "H": 4, "dk": 128, "dv": 256},
        # fine-tuning on packed short documents, odd head sizes
        {"name": "grad packed", "op": "grad", "dtype": "bf16", "nseq": 6, "lo": 20, "hi": 700, "empty": 0,
         "dense": False, "H": 3, "dk": 64, "dv": 96},
        # the norm in front of a single decoded token
        {"name": "norm one row", "op": "norm", "dtype": "bf16", "rows": 1, "d": 1024},
        # and in front of a training batch (8 x 2048 tokens, width 2048)
        {"name": "norm batch", "op": "norm", "dtype": "bf16", "rows": 16384, "d": 2048},
        # its gradients
        {"name": "dnorm batch", "op": "dnorm", "dtype": "bf16", "rows": 16384, "d": 2048},
        # an odd width, in 32 bits
        {"name": "dnorm odd", "op": "dnorm", "dtype": "fp32", "rows": 777, "d": 1001},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "step", "grad", "norm", "dnorm"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("norm", "dnorm"):
        d = _log_int(rng, 32, 8192)
        rows = _log_int(rng, 1, max(2, min(65536, 16384 * 2048 // (2 * d))))
        return {"op": op, "dtype": dtype, "rows": rows, "d": d}
    H = rng.randint(1, 16)
    if op == "step":
        dk, dv = 8 * rng.randint(2, 32), 8 * rng.randint(2, 64)
        B = _log_int(rng, 1, max(2, min(256, 256 * 16 * 128 * 128 // (H * dk * dv))))
        return {"op": op, "dtype": dtype, "B": B, "slots": B + rng.randint(0, 40), "H": H, "dk": dk, "dv": dv}
    dk, dv = 8 * rng.randint(4, 32), 8 * rng.randint(4, 32)
    hi = _log_int(rng, 1, 8192)
    most = 32768 * 4 * 768 // (H * (dk + dv))  # rows of the largest listed case, by bytes
    if dtype == "fp32":
        most, hi = most // 16, min(hi, 2048)
    if op == "grad":
        most //= 8
    nseq = _log_int(rng, 1, max(2, min(64, most // hi)))
    hi = min(hi, max(1, most // nseq))
    c = {"op": op, "dtype": dtype, "nseq": nseq, "lo": max(1, hi // rng.choice([1, 4, 64])), "hi": hi,
         "empty": rng.choice([0, 0, 1]), "H": H, "dk": dk, "dv": dv}
    if op == "prompt":
        c["spare"] = rng.choice([0, 0, 5, 130])
    else:
        c["dense"] = c["lo"] == hi and not c["empty"]
    return c


def lengths(case):
    """The lengths of the case's sequences: spread over their logarithm, the `empty` first of a shuffle at zero."""
    r = random.Random("%(nseq)d %(lo)d %(hi)d %(empty)d" % case)
    n = [min(case["hi"], max(case["lo"], _log_int(r, case["lo"], case["hi"]))) for _ in range(case["nseq"])]
    for b in r.sample(range(case["nseq"]), min(case["empty"], case["nseq"] - 1)):
        n[b] = 0
    return n


def _width(case):
    return 4 if case["dtype"] == "fp32" else 2


def work(case):
    """Inputs read once, outputs written once; products of the recurrence."""
    s = _width(case)
    if case["op"] in ("norm", "dnorm"):
        rows, d = case["rows"], case["d"]
        if case["op"] == "norm":
            return {"bytes": 2 * rows * d * s + 8 * rows + 8 * d, "flops": 8 * rows * d}
        return {"bytes": 3 * rows * d * s + 8 * rows + 12 * d, "flops": 14 * rows * d}
    H, dk, dv = case["H"], case["dk"], case["dv"]
    if case["op"] == "step":
        B = len([i for i in _slots(case) if i >= 0])
        return {"bytes": B * H * (8 * dk * dv + 2 * (dk + dv) * s), "flops": 5 * B * H * dk * dv}
    n = sum(lengths(case))
    states = case["nseq"] * H * dk * dv * 4
    if case["op"] == "prompt":
        return {"bytes": n * H * 2 * (dk + dv) * s + 2 * states, "flops": 4 * n * H * dk * dv}
    return {"bytes": n * H * (4 * dk + 3 * dv) * s + 3 * states, "flops": 10 * n * H * dk * dv}


# ---------------------------------------------------------------- inputs

def _slots(case):
    """The pool slot of each running request; -1: a padding row of the batch."""
    r = random.Random("%(B)d %(slots)d" % case)
    s = r.sample(range(case["slots"]), case["B"])
    for b in range(case["B"] // 16):
        s[-1 - b] = -1
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    st = {"case": dict(case)}
    if case["op"] in ("norm", "dnorm"):
        rows, d = case["rows"], case["d"]
        st["x"] = randn(rows, d) * 2 + 0.5
        st["w"] = 1 + randn(d, scale=0.1, dtype=torch.float32)
        st["b"] = randn(d, scale=0.1, dtype=torch.float32)
        st["y"] = torch.empty_like(st["x"])
        if case["op"] == "dnorm":
            st["dy"] = randn(rows, d)
            x = st["x"].double()  # what the forward pass left for the backward
            mean = x.mean(1)
            st["mean"] = mean.float()
            st["rstd"] = torch.rsqrt((x - mean[:, None]).square().mean(1) + 1e-5).float()
        return st
    H, dk, dv = case["H"], case["dk"], case["dv"]
    # heads from fast to slow forgetting: lambda = 1 - 2^-(3 .. 9)
    st["log_decay"] = torch.log1p(-torch.exp2(-3 - 6 * torch.arange(H, device="cuda") / max(1, H - 1)))
    if case["op"] == "step":
        B = case["B"]
        qkv = randn(B, H, 2 * dk + dv)  # one fused projection's output
        qkv[..., dk:2 * dk] *= dk ** -0.5
        st["q"], st["k"], st["v"] = qkv.split([dk, dk, dv], -1)
        st["state"] = randn(case["slots"], H, dk, dv, scale=dk ** -0.5, dtype=torch.float32)
        st["index"] = torch.tensor(_slots(case), dtype=torch.int32, device="cuda")
        st["o"] = torch.zeros(B, H, dv, dtype=dt, device="cuda")
        return st
    lens = lengths(case)
    n, nseq = sum(lens), len(lens)
    st["max_len"] = max(lens)
    st["n_chunks"] = sum(-(-x // CHUNK) for x in lens)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if case["op"] == "prompt":
        n += case["spare"]
        qkv = randn(n, H, 2 * dk + dv)  # token-major, one fused projection's output
        qkv[..., dk:2 * dk] *= dk ** -0.5
        st["q"], st["k"], st["v"] = (x.transpose(0, 1)[None] for x in qkv.split([dk, dk, dv], -1))
        st["o"] = torch.zeros(n, H, dv, dtype=dt, device="cuda").transpose(0, 1)[None]
        r = random.Random(nseq)
        slot = r.sample(range(nseq + 2), nseq)
        # every other request is new; the others continue from the state in their slot
        st["h0_index"] = torch.tensor([s if i % 2 else -1 for i, s in enumerate(slot)], dtype=torch.int32, device="cuda")
        st["index"] = torch.tensor(slot, dtype=torch.int32, device="cuda")
        st["state"] = randn(nseq + 2, H, dk, dv, scale=dk ** -0.5, dtype=torch.float32)
        return st
    if case["dense"]:
        shape = (nseq, H, case["hi"])
        st["q"], st["k"] = randn(*shape, dk), randn(*shape, dk, scale=dk ** -0.5)
        st["v"], st["do"] = randn(*shape, dv), randn(*shape, dv)
    else:
        st["q"], st["k"] = (randn(n, H, dk, scale=x).transpose(0, 1)[None] for x in (1.0, dk ** -0.5))
        st["v"], st["do"] = (randn(n, H, dv).transpose(0, 1)[None] for _ in range(2))
    st["h0"] = randn(nseq, H, dk, dv, scale=dk ** -0.5, dtype=torch.float32)
    st["dh_final"] = randn(nseq, H, dk, dv, scale=0.1, dtype=torch.float32)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import chunkwise_linear_rnn_fwd_b200 as pkg

    op = st["case"]["op"]
    if op == "prompt":
        o, state = pkg.gla_decay_fwd(st["q"], st["k"], st["v"], st["log_decay"], cu_seqlens=st["cu"],
                                     max_len=st["max_len"], h0=st["state"], h0_index=st["h0_index"],
                                     h_final=st["state"], h_final_index=st["index"], o=st["o"])
        return {"o": o, "state": state}
    if op == "step":
        o = pkg.gla_decay_step(st["q"], st["k"], st["v"], st["log_decay"], st["state"], st["index"], o=st["o"])
        return {"o": o, "state": st["state"]}
    if op == "grad":
        packed = {} if st["case"]["dense"] else {"cu_seqlens": st["cu"], "max_len": st["max_len"]}
        dq, dk, dv, dh0 = pkg.gla_decay_bwd(st["q"], st["k"], st["v"], st["log_decay"], st["do"], h0=st["h0"],
                                            dh_final=st["dh_final"], **packed)
        return {"dq": dq, "dk": dk, "dv": dv, "dh0": dh0}
    if op == "norm":
        y, mean, rstd = pkg.gla_layernorm_fwd(st["x"], st["w"], st["b"], eps=1e-5, y=st["y"])
        return {"y": y, "mean": mean, "rstd": rstd}
    dx, dw, db = pkg.gla_layernorm_bwd(st["x"], st["dy"], st["mean"], st["rstd"], st["w"])
    return {"dx": dx, "dw": dw, "db": db}


def _pow(log_decay, n):
    """lambda_h^n as [H, *n.shape], the exponent formed in 64 bits."""
    return torch.exp(log_decay.double().view(-1, *[1] * n.dim()) * n).float()


def _chunked(q, k, v, log_decay, cu, n_chunks, s0, reverse=False):
    """The recurrence over packed rows in chunks: q, k [H,N,dk], v [H,N,dv], s0 [nseq,H,dk,dv], all in 32 bits.
    Returns o for the rows of a sequence (the other rows are zero) and the final states. reverse: the adjoint
    recurrence from each sequence's last row to its first, s0 entering
    the last row undecayed, and the final state decayed once more."""
    H, N, dv = v.shape
    dev = q.device
    lead, tail = (0, 1) if reverse else (1, 0)
    cu = cu.long()
    lens = cu[1:] - cu[:-1]
    nch = (lens + CHUNK - 1) // CHUNK
    seq = torch.repeat_interleave(torch.arange(len(lens), device=dev), nch, output_size=n_chunks)
    p0 = CHUNK * (torch.arange(n_chunks, device=dev) - (nch.cumsum(0) - nch)[seq])
    m = (lens[seq] - p0).clamp(max=CHUNK)
    i = torch.arange(CHUNK, device=dev)
    pos = p0[:, None] + i
    live = i < m[:, None]
    tok = cu[seq][:, None] + ((lens[seq][:, None] - 1 - pos) if reverse else pos)
    tok = torch.where(live, tok, N)  # row N: a row of zeros to read, a spare row to write
    qc, kc, vc = (torch.nn.functional.pad(x, (0, 0, 0, 1))[:, tok] for x in (q, k, v))
    d = i[:, None] - i
    decay = torch.where(d >= 0, _pow(log_decay, d.clamp(min=0)), 0.0)
    o = (qc @ kc.transpose(-1, -2) * decay[:, None]) @ vc
    end = p0 + m
    u = (kc * _pow(log_decay, (m[:, None] - 1 - i).clamp(min=0))[..., None]).transpose(-1, -2) @ vc
    gap = p0[:, None] - end + 1  # from chunk to chunk of one sequence
    carry = torch.where((seq[:, None] == seq) & (gap > 0), _pow(log_decay, gap.clamp(min=0)), 0.0)
    flat = u.flatten(2)
    s0 = s0.transpose(0, 1)
    start = (carry @ flat).view_as(u) + _pow(log_decay, p0 + lead)[..., None, None] * s0[:, seq]
    o = o + _pow(log_decay, i)[:, None, :, None] * (qc @ start)
    out = torch.zeros(H, N + 1, dv, device=dev)
    out[:, tok.flatten()] = o.flatten(1, 2)
    b = torch.arange(len(lens), device=dev)
    left = lens[:, None] - end + tail
    last = torch.where(seq == b[:, None], _pow(log_decay, left.clamp(min=0)), 0.0)
    final = (last @ flat).view(H, len(lens), *u.shape[2:]) + _pow(log_decay, lens)[..., None, None] * s0
    return out[:, :N], final.transpose(0, 1)


def _rows(x):
    """[B,H,T,d] as packed rows [H,B*T,d] in 32 bits."""
    return x.transpose(0, 1).flatten(1, 2).float()


def _run_plain(st):
    op = st["case"]["op"]
    if op == "prompt":
        begin = st["h0_index"].long()
        s0 = torch.where((begin >= 0).view(-1, 1, 1, 1), st["state"][begin.clamp(min=0)], 0.0)
        o, final = _chunked(_rows(st["q"]), _rows(st["k"]), _rows(st["v"]), st["log_decay"], st["cu"],
                                  st["n_chunks"], s0)
        n = torch.arange(o.shape[1], device=o.device)
        st["o"][0] = torch.where((n < st["cu"][-1])[:, None], o.to(st["o"].dtype), st["o"][0])
        st["state"][st["index"].long()] = final
        return {"o": st["o"], "state": st["state"]}
    if op == "step":
        live = (st["index"] >= 0).view(-1, 1, 1)
        # a padding row reads some slot and writes it nowhere
        pool = torch.cat([st["state"], st["state"][:1]])
        at = torch.where(st["index"] >= 0, st["index"], len(st["state"])).long()
        q, k, v = (st[n].float() for n in "qkv")
        s = torch.exp(st["log_decay"])[:, None, None] * pool[at] + k[..., :, None] * v[..., None, :]
        o = (q[..., None, :] @ s)[..., 0, :]
        pool[at] = s
        st["state"].copy_(pool[:-1])
        st["o"].copy_(torch.where(live, o.to(st["o"].dtype), st["o"]))
        return {"o": st["o"], "state": st["state"]}
    if op == "grad":
        q, k, v, do = (_rows(st[n]) for n in ("q", "k", "v", "do"))
        dq, _ = _chunked(do, v, k, st["log_decay"], st["cu"], st["n_chunks"], st["h0"].transpose(-1, -2))
        dk, _ = _chunked(v, do, q, st["log_decay"], st["cu"], st["n_chunks"], st["dh_final"].transpose(-1, -2), True)
        dv, dh0 = _chunked(k, q, do, st["log_decay"], st["cu"], st["n_chunks"], st["dh_final"], True)
        out = {}
        for name, x, like in (("dq", dq, st["q"]), ("dk", dk, st["k"]), ("dv", dv, st["v"])):
            B, H, T, d = like.shape
            out[name] = x.view(H, B, T, d).transpose(0, 1).to(like.dtype)
        return {**out, "dh0": dh0}
    x = st["x"].float()
    if op == "norm":
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = torch.rsqrt(c.square().mean(1) + 1e-5)
        st["y"].copy_(c * rstd[:, None] * st["w"] + st["b"])
        return {"y": st["y"], "mean": mean, "rstd": rstd}
    dy = st["dy"].float()
    rstd = st["rstd"][:, None]
    xh = (x - st["mean"][:, None]) * rstd
    gy = dy * st["w"]
    dx = rstd * (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True))
    return {"dx": dx.to(st["x"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


# ---------------------------------------------------------------- 64 bits

def _padded(st, name, lens):
    """[B,H,T,d] or packed rows as [T,nseq,H,d] in 64 bits, zeros behind each sequence."""
    x = st[name].double()
    if x.shape[0] == len(lens) and (len(lens) > 1 or x.shape[2] == max(lens)):
        return x.permute(2, 0, 1, 3)
    out = torch.zeros(max(lens), len(lens), x.shape[1], x.shape[3], dtype=torch.float64, device=x.device)
    at = 0
    for b, n in enumerate(lens):
        out[:n, b] = x[0, :, at:at + n].transpose(0, 1)
        at += n
    return out


def _unpadded(y, like, lens, fill=None):
    """[T,nseq,H,d] laid out as `like`; rows of no sequence as in `fill`."""
    if like.shape[0] == len(lens) and (len(lens) > 1 or like.shape[2] == max(lens)):
        return y.permute(1, 2, 0, 3).contiguous()
    out = torch.zeros(like.shape, dtype=torch.float64, device=y.device) if fill is None else fill.double().clone()
    at = 0
    for b, n in enumerate(lens):
        out[0, :, at:at + n] = y[:n, b].transpose(0, 1)
        at += n
    return out


def exact(case, seed):
    """From the definitions, token by token, in 64 bits."""
    st = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "dnorm"):
        x, w, b = st["x"].double(), st["w"].double(), st["b"].double()
        if op == "norm":
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = (var + 1e-5) ** -0.5
            return {"y": (x - mean[:, None]) * rstd[:, None] * w + b, "mean": mean, "rstd": rstd}
        dy, mean, rstd = st["dy"].double(), st["mean"].double()[:, None], st["rstd"].double()[:, None]
        xh = (x - mean) * rstd
        d = x.shape[1]
        s1, s2 = (dy @ w)[:, None] / d, ((dy * xh) @ w)[:, None] / d
        return {"dx": rstd * (dy * w - s1 - xh * s2), "dw": torch.einsum("nd,nd->d", dy, xh), "db": dy.sum(0)}
    lam = torch.exp(st["log_decay"].double())[:, None, None]
    if op == "step":
        q, k, v = (st[n].double() for n in "qkv")
        state, o = st["state"].double(), st["o"].double()
        for b, i in enumerate(_slots(case)):
            if i >= 0:
                state[i] = lam * state[i] + torch.einsum("hk,hv->hkv", k[b], v[b])
                o[b] = torch.einsum("hk,hkv->hv", q[b], state[i])
        return {"o": o, "state": state}
    lens = lengths(case)
    T = max(lens)
    left = torch.tensor(lens, device="cuda")
    q, k, v = (_padded(st, n, lens) for n in "qkv")
    alive = torch.arange(T, device="cuda")[:, None] < left
    keep = torch.where(alive[:, :, None, None, None], lam, 1.0)  # a sequence that has ended keeps its state
    if op == "prompt":
        begin = st["h0_index"].long()
        S = torch.where((begin >= 0).view(-1, 1, 1, 1), st["state"][begin.clamp(min=0)], 0.0).double()
        o = torch.empty_like(v)
        for t in range(T):
            S = S * keep[t] + k[t][..., :, None] * v[t][..., None, :]
            o[t] = torch.einsum("bhk,bhkv->bhv", q[t], S)
        state = st["state"].double()
        state[st["index"].long()] = S
        return {"o": _unpadded(o, st["o"], lens, st["o"]), "state": state}
    do = _padded(st, "do", lens)
    S, R = st["h0"].double(), st["dh_final"].double()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(T):
        S = S * keep[t] + k[t][..., :, None] * v[t][..., None, :]
        dq[t] = torch.einsum("bhv,bhkv->bhk", do[t], S)
    for t in reversed(range(T)):  # R: the loss's derivative by S_t
        R = R + q[t][..., :, None] * do[t][..., None, :]
        dk[t] = torch.einsum("bhv,bhkv->bhk", v[t], R)
        dv[t] = torch.einsum("bhk,bhkv->bhv", k[t], R)
        R = R * keep[t]
    return {"dq": _unpadded(dq, st["q"], lens), "dk": _unpadded(dk, st["k"], lens), "dv": _unpadded(dv, st["v"], lens),
            "dh0": R}
