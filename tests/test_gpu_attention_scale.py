"""Paged attention with other scales than the usual one, on the GPU, against a 64-bit
implementation: the same handle's calls of one token, a few, and chunks."""
import numpy as np
import pytest
import torch

import attention_harness as H

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0.0, -0.0, -0.1, 2.0, 1e-4, -1e-40, 1e-40])
@pytest.mark.parametrize("heads,d,requests", [((8, 2), 64, [(130, 1), (5, 1), (700, 1)]), ((8, 2), 128, [(100, 60), (0, 130)]),
                                              ((10, 2), 128, [(900, 5), (33, 5)]), ((6, 1), 256, [(70, 90), (300, 2)])])
def test_scales(heads, d, requests, scale):
    p = H.Pages(heads, d, 16, requests, seed=d, gate=True)
    h = p.handle(scale=scale)
    out = p.call(h)
    # scale q . k = |scale| (-q) . k
    p.scale = abs(scale)
    if scale < 0:
        p.q = -p.q
    assert h.check() == (0, 0)
    H.check(out, *p.reference())
