"""The failure report of the kernels around the recurrence whose CTAs wait for one another, on the GPU,
without a fault: mlstm_block_selftest_timeout enqueues one kernel whose wait (on a word that nothing raises)
runs out after 2 s.  Each failure is reported once, replays of one captured launch among them: every
replay waits anew, and its failure is news although the launch is the same."""

import time

import pytest
import torch

from mlstm_chunkwise_attention_b200 import binding, block

pytestmark = pytest.mark.gpu

TIMEOUT = 5  # MLSTM_ERR_TIMEOUT
FAMILIES = {"scan_fwd": 0, "scan_bwd": 1, "norm": 2}


def status():
    return binding.mlstm_device_status(torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("family", FAMILIES)
def test_every_failure_of_a_replayed_launch_is_reported(family):
    binding.check_device()  # nothing pending before the test
    words = torch.ones(2, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert binding.load().mlstm_block_selftest_timeout(
            FAMILIES[family], words.data_ptr(), 8, torch.cuda.current_stream().cuda_stream) == 0
    for _ in range(2):
        torch.cuda.synchronize()
        began = time.monotonic()
        graph.replay()
        assert status() == TIMEOUT
        assert time.monotonic() - began > 1.5, "a replay gave up before its wait was over"
        assert status() == 0, "reported once"
    # what a failure sets is its own launch's: a call behind it has the bits of one before it
    x = torch.randn(2, 70, 128, device="cuda")
    y, _ = block.group_norm_forward(x, groups=2, scope=block.SCOPE_SEQUENCE)
    graph.replay()
    again, _ = block.group_norm_forward(x, groups=2, scope=block.SCOPE_SEQUENCE)
    assert status() == TIMEOUT and torch.equal(y, again)
