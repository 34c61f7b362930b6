"""The operators' choice of a stream, without a device."""
import pytest
import torch

import kv_cache_compression_c128_gb300 as kvc


class _Stream:
    def __init__(self, index):
        self.device = torch.device("cuda", index)
        self.cuda_stream = 0x1234


def test_a_stream_of_another_device_is_refused():
    kvc._load_torch()
    called = []
    with pytest.raises(ValueError, match="stream must be one of cuda:0, got one of cuda:1"):
        kvc._run(called.append, 0, _Stream(1))
    assert not called
