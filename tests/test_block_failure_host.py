"""The waits' self-test refuses on the host what it cannot run (no GPU)."""

import os

import pytest

from mlstm_chunkwise_attention_b200 import binding as B

FAKE = 0x100000  # an aligned address that no call dereferences: every one of these returns before a launch


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from mlstm_chunkwise_attention_b200 import _build
        _build.build()
    return B.load()


@pytest.mark.parametrize("args,status", [
    ((-1, FAKE, 8), 1), ((3, FAKE, 8), 1), ((0, FAKE + 2, 8), 1), ((1, None, 8), 3), ((2, FAKE, 7), 3),
])
def test_selftest_argument_errors(lib, args, status):
    assert lib.mlstm_block_selftest_timeout(*args, None) == status
