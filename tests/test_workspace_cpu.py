"""The binding's check of scratch tensors, on the host."""

import pytest
import torch

from selected_token_logprob_gb300 import _args


@pytest.mark.parametrize("ws", [torch.empty(1, dtype=torch.uint8).expand(1 << 20), torch.empty(1 << 12)[::2],
                                torch.empty(64, 64).t()])
def test_scratch_that_does_not_own_its_bytes_is_refused(ws):
    with pytest.raises(ValueError, match="contiguous"):
        _args._workspace(ws)


def test_host_memory_is_refused():
    with pytest.raises(ValueError, match="CUDA"):
        _args._workspace(torch.empty(64, dtype=torch.uint8))
