"""Paged attention at the ends of its ranges, on the GPU."""
import numpy as np
import pytest
import torch

import attention_harness as H

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_len", [0, 1, 40])
@pytest.mark.parametrize("requests", [0, 3, 200])
def test_pad_rows_alone(requests, max_len):
    """No request has a new token, or there is none: nothing to share out, and every row is zero."""
    from gated_deltanet_layer_gb300 import PagedAttention
    h = PagedAttention(8, 2, 128, 16, max_tokens=40, max_seqs=200)
    kv = torch.full((160, 2, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = torch.full((40, 1024), float("nan"), dtype=torch.bfloat16, device="cuda")
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    for _ in range(3):
        out = h.attend(q, kv, kv.clone(), ints(requests, 4), ints(requests + 1), ints(requests), max_len=max_len)
        assert (out == 0).all()
    assert h.check() == (0, 0)
