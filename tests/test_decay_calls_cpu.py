"""How the decay and layer-norm calls take their arguments, without a GPU."""
import pytest
import torch

import chunkwise_linear_rnn_fwd_b200 as pkg


def test_every_argument_by_keyword():
    """As with the other entry points: the tensor's place is what is refused here, not the spelling."""
    x, ld, row = torch.zeros(1, 2, 8, 16), torch.zeros(2), torch.zeros(3, 8)
    with pytest.raises(ValueError, match="CUDA device"):
        pkg.gla_decay_fwd(q=x, k=x, v=x, log_decay=ld)
    with pytest.raises(ValueError, match="CUDA device"):
        pkg.gla_decay_bwd(q=x, k=x, v=x, log_decay=ld, do=x)
    with pytest.raises(ValueError, match="CUDA device"):
        pkg.gla_decay_step(q=x[:, :, 0], k=x[:, :, 0], v=x[:, :, 0], log_decay=ld, state=torch.zeros(1, 2, 16, 16))
    with pytest.raises(ValueError, match="CUDA device"):
        pkg.gla_layernorm_fwd(x=row)
    with pytest.raises(ValueError, match="CUDA device"):
        pkg.gla_layernorm_bwd(x=row, dy=row, mean=row[:, 0], rstd=row[:, 0])


def test_a_missing_argument_is_named():
    with pytest.raises(TypeError, match="'q'"):
        pkg.gla_decay_fwd()
    with pytest.raises(TypeError, match="'log_decay'"):
        pkg.gla_decay_step(k=torch.zeros(1), v=torch.zeros(1), state=torch.zeros(1))


def test_a_workspace_of_another_device_is_refused():
    """Its address would go to the kernels of cuda:0."""
    from chunkwise_linear_rnn_fwd_b200 import gla as G
    ws = torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace"):
        G._decay_desc(1, 1, 8, 0, 16, 16, torch.bfloat16, workspace=ws)
