"""Refusals of the step operators' binding that host tensors reach (no GPU needed): tensors pass for
device 0's, and every call fails a check before the library is entered."""
import pytest

import fp8_kv_cache_gb300 as P


def test_a_cache_without_heads(monkeypatch):
    """A ValueError, as every wrong shape."""
    import torch
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    kv, sc = torch.zeros(4, 16, 0, 256, dtype=torch.int8), torch.zeros(4, 1, 0)
    q, i2 = torch.zeros(2, 4, 256, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(2, 2, dtype=torch.int32)
    for call in (lambda: P.paged_gqa_decode_scaled(q, kv, kv, sc, sc, table, i2, 16, 1.0),
                 lambda: P.paged_gqa_sparse_prefill_scaled(q, kv, kv, sc, sc, i2, 32, table, i2, 16, 1.0)):
        with pytest.raises(ValueError, match="a multiple of the cache's heads"):
            call()
