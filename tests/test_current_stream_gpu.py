"""A call without a stream goes to torch's current one."""
import pytest
import torch

import moe_token_permute_gb300 as mp


@pytest.mark.gpu
def test_current_stream_is_torchs():
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            assert mp._stream(None) == s.cuda_stream == mp._stream(s)
