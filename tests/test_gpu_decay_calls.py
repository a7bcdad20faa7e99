"""How the decay and layer-norm calls are made on the GPU: arguments by keyword, outputs and
workspaces that the call makes or is given, states that many chunks and tokens pass on."""
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
