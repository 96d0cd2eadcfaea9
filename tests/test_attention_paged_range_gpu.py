"""fp16 values at the end of their range: an average of them stays inside it, although the rounded
weights can sum to 1 + 2^-11 times the sum they are divided by.  Tolerances as in
test_attention_paged_gpu.py."""

import math

import pytest
import torch

from .test_attention_paged_gpu import Case

pytestmark = pytest.mark.gpu


# A weight just behind the middle of two fp16 values next to 1/2: 1/2 (1 + 1.05 2^-11) rounds to
# 1/2 (1 + 2^-10), 0.95 2^-11 more of itself, and 65504 (1 + 2^-12) rounds to an infinity.
SCALE = -math.log(0.5 * (1 + 1.05 * 2.0 ** -11))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows,ctx,nq,nkv", [
    ([1] * 40, [60 + k % 5 for k in range(40)], 8, 2),  # whole items of the few-row kernel
    ([1, 1], [3000, 500], 8, 2),                        # its shared items
    ([60, 33], [50, 40], 8, 2),                         # whole items on tcgen05
    ([9, 40, 300], [2500, 700, 90], 4, 1),              # shared ones, one and two query tiles
])
def test_the_largest_fp16_values(rows, ctx, nq, nkv, hd):
    c = Case(91 + hd, rows, ctx, nq, nkv, hd, "f16", 16)
    c.q.zero_()
    c.q[..., 0] = 1
    # scores 0 for every 16th key and -SCALE for all others
    c.kp.copy_(torch.where(torch.isnan(c.kp), c.kp, torch.zeros_like(c.kp)))
    for r, t in enumerate(c.len):
        for key in range(int(t)):
            if key % 16:
                c.kp[c.tab[r, key // 16], :, key % 16, 0] = -1
    sign = torch.where(torch.arange(hd, device="cuda") % 3 == 0, -1.0, 1.0)
    c.vp.copy_(torch.where(torch.isnan(c.vp), c.vp, (65504.0 * sign).half()))
    for causal, window in ((True, 0), (False, 50)):
        out, lse = c.run(causal, window, scale=SCALE)
        assert torch.isfinite(out).all()
        c.check(out, lse, causal, window, scale=SCALE)


def test_infinities_that_rows_see_stay_infinite():
    for rows in ([2], [70]):
        c = Case(93, rows, [30], 4, 2, 64, "f16", 16)
        c.vp[c.tab[0, 0], :, 3, 5] = float("inf")
        c.vp[c.tab[0, 0], :, 4, 6] = float("-inf")
        out, lse = c.run()
        assert (out[..., 5] == float("inf")).all() and (out[..., 6] == float("-inf")).all()
        c.check(out, lse)
