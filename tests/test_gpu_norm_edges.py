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


@pytest.mark.parametrize("d", [64, 2056])
def test_statistics_of_values_far_from_zero_and_from_each_other(d):
    """Group 0: one vector 2^12 from the rest.  Group 1: all values near 2^12.  The statistics against 64 bits:

    - the mean is joined in 64 bits and rounded once, 2^-24 of itself, from sums whose terms are distances
      (at most 300 additions in a row: 300 2^-24 of their mean size);
    - the squared distances are sums of at most 300 positive terms, 2^-16 of the variance and half of it of
      1 / deviation; but for d = 2056 a warp takes distances from one of its vectors, of which it has 512
      at most, so where that vector is the far one (group 0) 512 times that, 2^-8.

    y differs by 1 / deviation times the mean's error, that of 1 / deviation, and four roundings."""
    B, T, NH = 1, 200, 2
    g = torch.Generator().manual_seed(12)
    x = torch.randn(B, T, NH * d, generator=g)
    x[:, 0, :8] += 4096.0
    x[:, :, d:] += 4096.0
    y, stats = block.group_norm_forward(x.cuda(), groups=NH, scope=SEQ)
    binding.check_device()
    v = x.double().view(T, NH, d)
    mean = v.mean((0, 2))
    size = (v - mean[:, None]).abs().mean((0, 2))
    rstd = 1 / torch.sqrt(((v - mean[:, None]) ** 2).mean((0, 2)) + 1e-5)
    got = stats.double().cpu()[0]
    off = 2.0 ** -24 * (mean.abs() + 300 * size)
    rel = torch.tensor([2.0 ** -8 if d > 2048 else 2.0 ** -17, 2.0 ** -17], dtype=torch.float64) + 2.0 ** -22
    assert ((got[:, 0] - mean).abs() <= off).all(), (got[:, 0] - mean, off)
    assert ((got[:, 1] - rstd).abs() <= rel * rstd).all(), (got[:, 1] / rstd - 1, rel)
    xhat = (v - mean[:, None]) * rstd[:, None]
    bound = (rstd * off)[:, None] + (rel[:, None] + 2.0 ** -22) * (xhat.abs() + (rstd * off)[:, None])
    err = (y.double().cpu().view(T, NH, d) - xhat).abs()
    assert (err <= bound).all(), float((err - bound).max())


@pytest.mark.parametrize("T,d", [(40, 64), (3, 2056), (300, 4096)])
def test_norm_of_squares_beyond_the_range_of_fp32(T, d):
    """Distances from the mean near 2^66: the variance is infinite in fp32 and 1 / deviation 0, in the kernel
    for large groups as in the one for small ones, and the output is the bias."""
    x = torch.full((1, T, d), 2.0 ** 66, device="cuda")
    x[:, 0, :8] = 0.0  # the vector from which a warp takes its distances
    x[:, T // 2:, ::2] = 0.0
    b = torch.linspace(-1, 1, d, device="cuda")
    y, stats = block.group_norm_forward(x, None, b, groups=1, scope=SEQ)
    binding.check_device()
    assert float(stats[0, 0, 1]) == 0.0 and torch.equal(y, b.expand_as(y))
