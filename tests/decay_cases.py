"""Shared by the decay-attention tests: seeded batches of sequences, the float64 oracle
over them, and the error that the arithmetic of a path allows.

The allowed error of every output element is derived from the roundings that the path
makes.  With A the same quantity computed from absolute values (the sum of the absolute
values of all its terms), h = 2^-8 the half step of bf16:
  fp32 arithmetic: a term passes at most n additions and products, n the length of the
    dot products and of the chain of chunk updates, each off by at most 2^-23 (rounded or
    truncated) of what it adds up: n 2^-23 A.
  bf16 on tensor cores: a term of o passes one operand rounded to bf16, its score or the
    state it comes from: h (1 + h) A more.  The states take k and v exactly, and
    the weight times v as the exact sum of three bf16 numbers.
  an output stored in bf16: h (|r| + the error so far).
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import decay as oracle

H8 = 2.0 ** -8


def rates(H, kind="mixed"):
    if kind == "mixed":  # from fast to slow forgetting, the last head forgets nothing
        r = np.log1p(-np.exp2(-1 - 8 * np.arange(H) / max(1, H - 1)))
        if H > 1:
            r[-1] = 0.0
        return torch.tensor(r, dtype=torch.float32)
    return torch.full((H,), float(kind), dtype=torch.float32)


class Batch:
    """lens sequences; name -> [sum(lens) + spare, H, d] token-major double tensors whose
    values are exact in `dtype`; states [n,H,dk,dv] fp32."""

    def __init__(self, lens, H, dk, dv, dtype, seed=0, spare=0, kind="mixed"):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.dk, self.dv, self.dtype = list(lens), H, dk, dv, dtype
        self.cu = [0]
        for x in lens:
            self.cu.append(self.cu[-1] + x)
        self.rows = self.cu[-1] + spare

        def randn(d, scale=1.0):
            return (torch.randn(self.rows, H, d, generator=g, dtype=torch.float64) * scale).to(dtype)

        self.q, self.k, self.v, self.do = randn(dk), randn(dk, dk ** -0.5), randn(dv), randn(dv)
        self.ld = rates(H, kind)
        n = len(lens)
        self.h0 = torch.randn(n, H, dk, dv, generator=g) * dk ** -0.5
        self.dh = torch.randn(n, H, dk, dv, generator=g) * 0.3

    def seq(self, name, i, absolute=False):
        x = getattr(self, name)
        x = x[self.cu[i]:self.cu[i + 1]].transpose(0, 1) if x.dim() == 3 else x[i]
        x = x.double().numpy()
        return np.abs(x) if absolute else x


def steps(b, dk, dv, length):
    """Additions and products a term passes: dot products of dk, dv and of two chunks of at
    most 128 tokens, and three operations for each of the chain's chunks (of at least 32)."""
    return dk + dv + 2 * 128 + 3 * (length // 32 + 1) + 40


def tolerance(name, ref, A, b, tensor_cores, length):
    e = steps(b, b.dk, b.dv, length) * 2.0 ** -23 * A
    state = name in ("h_final", "dh0")
    if tensor_cores:
        e = e + (0.0 if state else H8 * (1 + H8) * A)
    if b.dtype == torch.bfloat16 and not state:
        e = e + H8 * (np.abs(ref) + e)
    return e + 1e-30


def reference(b, with_h0=True, bwd=False, with_dh=True):
    """[{name: (ref, A)}] per sequence."""
    out = []
    ld = b.ld.double().numpy()
    for i in range(len(b.lens)):
        r = []
        for a in (False, True):
            g = lambda n: b.seq(n, i, a)  # noqa: E731
            h0 = g("h0") if with_h0 else None
            if bwd:
                r.append(oracle.bwd(g("q"), g("k"), g("v"), ld, g("do"), h0, g("dh") if with_dh else None))
            else:
                r.append(oracle.fwd(g("q"), g("k"), g("v"), ld, h0))
        names = ("dq", "dk", "dv", "dh0") if bwd else ("o", "h_final")
        out.append({n: (x, y) for n, x, y in zip(names, *r)})
    return out


def check(got, want, b, tensor_cores):
    """got: {name: [rows,H,d] or [n,H,dk,dv] tensor}; every element within its tolerance."""
    for name, x in got.items():
        x = x.detach().double().cpu()
        for i, w in enumerate(want):
            ref, A = w[name]
            y = x[b.cu[i]:b.cu[i + 1]].transpose(0, 1) if x.dim() == 3 else x[i]
            off = np.abs(y.numpy() - ref)
            tol = tolerance(name, ref, A, b, tensor_cores, b.lens[i])
            assert np.all(np.isfinite(y.numpy())), f"{name} of sequence {i} is not finite"
            worst = float(np.max(off / tol)) if off.size else 0.0
            assert worst <= 1.0, f"{name} of sequence {i} (length {b.lens[i]}): {worst:.2f} of what the arithmetic allows"


def views(b, names, layout, device="cuda"):
    """The batch's tensors on the device as the calls take them.
    tokens: packed [1,H,rows,d] views of token-major rows; fused: slices of one matrix;
    heads: packed, contiguous [1,H,rows,d]; dense / dense_tokens: [n,H,T,d] contiguous, or
    views of [n,T,H,d] (equal lengths)."""
    xs = {n: getattr(b, n).to(device) for n in names}
    if layout == "fused":
        big = torch.cat([xs[n] for n in names], -1)
        return {n: x.transpose(0, 1)[None] for n, x in zip(names, big.split([xs[n].shape[-1] for n in names], -1))}
    if layout == "tokens":
        return {n: x.transpose(0, 1)[None] for n, x in xs.items()}
    if layout == "heads":
        return {n: x.transpose(0, 1).contiguous()[None] for n, x in xs.items()}
    n_seq, T = len(b.lens), b.lens[0]
    out = {n: x.view(n_seq, T, b.H, -1).transpose(1, 2) for n, x in xs.items()}
    return {n: x.contiguous() for n, x in out.items()} if layout == "dense" else out


def rows(x):
    """[B,H,T,d] back to [B*T,H,d]."""
    return x.transpose(1, 2).flatten(0, 1)


def packing(b, layout, device="cuda"):
    if layout.startswith("dense"):
        return {}
    return {"cu_seqlens": torch.tensor(b.cu, dtype=torch.int32, device=device), "max_len": max(1, max(b.lens))}
