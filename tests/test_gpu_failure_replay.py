"""A captured launch whose wait ran out is replayed: the report of the first failure must not hide the next.
mlstm_selftest_timeout stands for a tensor-core kernel's launch (one wait, 2 s, no fault)."""

import time

import pytest
import torch

from mlstm_chunkwise_attention_b200 import binding

pytestmark = pytest.mark.gpu

TIMEOUT = 5  # MLSTM_ERR_TIMEOUT


def test_every_reported_failure_of_a_replayed_launch_is_news():
    binding.check_device()  # nothing pending before the test
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        assert binding.mlstm_selftest_timeout(torch.cuda.current_stream().cuda_stream) == 0
    status = lambda: binding.mlstm_device_status(torch.cuda.current_stream().cuda_stream)
    for _ in range(2):
        torch.cuda.synchronize()
        began = time.monotonic()
        graph.replay()
        assert status() == TIMEOUT
        assert time.monotonic() - began > 1.5, "a replay gave up before its wait was over"
        assert status() == 0, "reported once"
