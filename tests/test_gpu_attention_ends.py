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


@pytest.mark.parametrize("heads,d,block", [((8, 2), 64, 16), ((8, 2), 128, 32), ((12, 3), 256, 16)])
def test_pieces_and_boxes_in_turn(heads, d, block):
    """Many short requests a CTA, whose last keys come in pieces and the others in boxes: each place of the ring has both in
    turn. Every call has the first one's bits."""
    rng = np.random.default_rng(d)
    p = H.Pages(heads, d, block, [(int(c), 1) for c in rng.integers(0, 700, 400)], seed=d)
    h = p.handle()
    outs = [p.call(h) for _ in range(10)]
    assert h.check() == (0, 0)
    H.check(outs[0], *p.reference())
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
