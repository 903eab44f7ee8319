"""The group norm over a sequence where its numbers leave the ordinary range, and tighter bounds on its
statistics."""

import pytest
import torch

from mlstm_chunkwise_attention_b200 import binding, block

pytestmark = pytest.mark.gpu

SEQ = block.SCOPE_SEQUENCE


# groups that a cluster holds, and larger ones, whose blocks of 2048 channels leave warps without any
@pytest.mark.parametrize("T,NH,d", [(40, 2, 64), (3, 2, 2056), (2, 3, 1100), (300, 1, 4096)])
def test_norm_of_values_scaled_by_a_power_of_two(T, NH, d):
    """x 2^56 with eps 2^112 has the very outputs and gradients of x with eps (dx 2^-56): every operation
    scales exactly.  The values lie near 2^68, whose squares fp32 does not hold; their distances from the
    mean, near 2^56, it does."""
    g = torch.Generator().manual_seed(T + d)
    x = (4096.0 + torch.randn(1, T, NH * d, generator=g)).cuda()
    dy = torch.randn(1, T, NH * d, generator=g).cuda()
    res = []
    for p in (0, 56):
        s = x * 2.0 ** p
        y, stats = block.group_norm_forward(s, groups=NH, scope=SEQ, eps=1e-5 * 2.0 ** (2 * p))
        dx = block.group_norm_backward(s, None, None, dy, stats, groups=NH, scope=SEQ)["dx"]
        res.append((y, dx * 2.0 ** p, stats * torch.tensor([2.0 ** -p, 2.0 ** p], device="cuda")))
    binding.check_device()
    for a, b in zip(*res):
        assert torch.isfinite(a).all() and torch.equal(a, b)
