"""The rotary op writes rows of every layout that do not overlap, and nothing between them."""

import numpy as np
import pytest
import torch

from gpu_util import bits, ready
from invariant_vd_step_gb300 import vd
from test_rotary_rows import layouts

pytestmark = pytest.mark.gpu


def test_rows_that_do_not_overlap():
    ready()
    L, hd = vd.lib(), 6
    rope = vd.Rope(hd, theta=100.0)
    x = torch.randn((5, 4, hd), device="cuda")
    pos = torch.tensor([3, 70, 1, 0, 12345], dtype=torch.int32, device="cuda")
    want = rope.apply(x, pos)
    size, jobs = 1200, []
    for T, H, st, sh, overlap in layouts():
        if overlap:
            continue
        for a, b in ((1, 1), (-1, 1), (1, -1)):
            y = torch.full((size,), 9.0, device="cuda")
            base = 600  # elements before and behind every row of every layout
            assert L.vd_op_rotary(rope.h, x.data_ptr(), y.data_ptr() + 4 * base, T, H, 4 * hd, hd, a * st, b * sh, 2,
                                  pos.data_ptr(), 0, None) == vd.VD_OK, (T, H, st, sh)
            jobs.append((T, H, a * st, b * sh, y))
    torch.cuda.synchronize()
    assert len(jobs) > 500
    w = bits(want)
    for T, H, st, sh, y in jobs:
        ref = np.full(size, bits(torch.full((1,), 9.0))[0])
        for t in range(T):
            for h in range(H):
                at = 600 + t * st + h * sh
                ref[at:at + hd] = w[t, h]
        np.testing.assert_array_equal(bits(y), ref)


def test_heads_interleaved_with_tokens():
    """Head stride 256, token stride 384, head dim 128: two heads of a token around a head of the next one."""
    ready()
    rope, x = vd.Rope(128), torch.randn((40, 2, 128), device="cuda").bfloat16()
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    y = torch.zeros(40 * 384 + 512, dtype=torch.bfloat16, device="cuda")
    view = y.as_strided((40, 2, 128), (384, 256, 1))
    rope.apply(x, pos, view)
    assert torch.equal(view, rope.apply(x, pos))
    with pytest.raises(vd.VDError):
        rope.apply(x, pos, y.as_strided((40, 2, 128), (384, 300, 1)))
