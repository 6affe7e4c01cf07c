"""Paged attention where neighbouring tasks are each shared by more CTAs than are joined at once, on
the GPU, against a 64-bit implementation."""
import numpy as np
import pytest
import torch

import attention_harness as H

pytestmark = pytest.mark.gpu


def counters(h):
    """The words that the parts of tasks are counted in, behind the error word's 256 bytes."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return h.workspace[256:256 + 8 * sms].view(torch.int32)


@pytest.mark.parametrize("heads,d,block,requests", [
    ((8, 1), 128, 32, [(32768, 1)] * 8),
    ((8, 1), 128, 32, [(17952, 1)] * 8),
    ((6, 1), 128, 24, [(18949, 1)] * 5),
    ((4, 1), 64, 16, [(65536, 1)] * 5),
    ((16, 8), 128, 64, [(33400, 1)]),
    ((24, 4), 256, 64, [(29500, 1), (32768, 1)])])
def test_long_neighbours(heads, d, block, requests):
    """Many calls of one handle beside another handle's on a second stream, which take the SMs out of step: every one has the
    first one's bits and leaves its counters at zero, and a call of another form after them is right."""
    p = H.Pages(heads, d, block, requests, seed=d + len(requests))
    want = p.reference()
    h, outs = p.handle(), []
    side = H.Pages((8, 2), 128, 16, [(900, 60), (0, 77)], seed=2)
    other, beside = side.handle(), torch.cuda.Stream()
    beside.wait_stream(torch.cuda.current_stream())
    for i in range(24):
        with torch.cuda.stream(beside):
            side.call(other)
        outs.append(torch.full_like(p.q, 7.0))
        p.call(h, out=outs[-1])
    torch.cuda.synchronize()
    assert h.check() == (0, 0) and other.check() == (0, 0)
    assert (counters(h) == 0).all()
    H.check(outs[0], *want)
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
    short = H.Pages(heads, d, block, [(40 + i, 1) for i in range(len(requests))], seed=5)
    H.check(short.call(h), *short.reference())


@pytest.mark.parametrize("heads,d,requests", [((16, 4), 64, [(60 * i, 150 + 7 * i) for i in range(10)]),
                                              ((12, 6), 128, [(200 - 20 * i, 90 + 31 * i) for i in range(8)]),
                                              ((20, 4), 128, [(500 + 90 * i, 4) for i in range(16)]),
                                              ((24, 4), 256, [(30 * i, 40 + 13 * i) for i in range(10)])])
def test_hidden_values_in_many_parts(heads, d, requests):
    """Values that are not finite and that later tokens alone see, in about half of many parts of tasks, one right after the
    other in each pair of CTAs: no part has another's."""
    p = H.Pages(heads, d, 16, requests, seed=d)
    rng = np.random.default_rng(d)
    for s in range(p.S):
        at, n = p.slots(s), int(p.new[s])
        for head in range(p.Hkv):
            for row in rng.integers(1, n, 2):
                if rng.random() < 0.5:
                    p.v[int(at[len(at) - int(row)]), head, int(rng.integers(0, d))] = float(rng.choice([np.nan, np.inf, -np.inf]))
    want, tol = p.reference()
    ok = np.isfinite(want)
    assert ok.any() and not ok.all()
    h = p.handle()
    outs = [p.call(h) for _ in range(12)]
    assert h.check() == (0, 0)
    got = H.f64(outs[0])
    assert not np.isfinite(got[~ok]).any()
    assert np.isfinite(got[ok]).all() and (np.abs(got[ok] - want[ok]) <= tol[ok]).all()
    assert all(torch.equal(o.view(torch.int16), outs[0].view(torch.int16)) for o in outs[1:])
